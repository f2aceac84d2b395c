// paged_index.cuh -- index arithmetic of the paged key/value cache, shared by the kernels
// and the host: which cached tokens a query sees, where a token lives. Plain C++ (no CUDA
// types), so that it can be checked on the CPU.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define G2_HD __host__ __device__ __forceinline__
#else
#define G2_HD inline
#endif

namespace g2 {

// The work of one attention call is cut into tiles of PAT_TILE keys at positions 16 i ... 16 i +
// 15: with pages of 16 tokens or more a tile lies in one page.
constexpr int PAT_TILE = 16;

// The tokens that the newest of `len` tokens sees: positions below `sink` and lo .. len - 1; and
// the tiles that hold them: the first `sink_tiles`, then those from `first` on, `tiles` in all.
struct PagedVisible {
  int len, lo, sink, sink_tiles, first, tiles;
};

// len tokens cached, of which the newest has just been appended; window <= 0: all of them
// are visible; otherwise the newest `window`, and the first `sinks` besides.
G2_HD PagedVisible paged_visible(int len, int window, int sinks) {
  PagedVisible v;
  v.len = len;
  v.lo = window > 0 && len > window ? len - window : 0;
  v.sink = sinks < v.lo ? sinks : v.lo;
  v.sink_tiles = v.sink / PAT_TILE + (v.sink % PAT_TILE != 0);
  const int at = v.lo / PAT_TILE;
  v.first = at > v.sink_tiles ? at : v.sink_tiles;
  v.tiles = len > 0 ? v.sink_tiles + (len - 1) / PAT_TILE - v.first + 1 : 0;
  return v;
}

// The position of the first key of tile `t` (0 <= t < tiles), and which of its 16 keys are seen.
G2_HD int paged_tile_pos(const PagedVisible& v, int t) {
  return (t < v.sink_tiles ? t : t - v.sink_tiles + v.first) * PAT_TILE;
}
G2_HD uint32_t paged_below(int n) {  // bits 0 .. n - 1 of 16
  return n <= 0 ? 0u : n >= PAT_TILE ? 0xffffu : (1u << n) - 1;
}
G2_HD uint32_t paged_tile_mask(const PagedVisible& v, int pos) {
  return (paged_below(v.len - pos) & ~paged_below(v.lo - pos)) | paged_below(v.sink - pos);
}

// A sequence length as read from device memory, brought into [0, capacity]; *bad is set when
// it was outside.
G2_HD int paged_length(int len, int capacity, int* bad) {
  if (len < 0 || len > capacity) {
    *bad = 1;
    return len < 0 ? 0 : capacity;
  }
  return len;
}

// The tiles of all items (a sequence, a key head and a tile of its query heads) are laid end to
// end: sequence by sequence, item by item. Worker w takes tiles [w * share, (w + 1) * share).
G2_HD int64_t paged_div(int64_t x, int64_t d) {  // 0 <= x, 1 <= d; nearly always 32-bit numbers
  return ((x | d) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)d) : x / d;
}
// x / d for 0 <= x < 2^31 with inverse = (2^32 - 1) / d: the high product is at most one too small.
G2_HD int paged_div_by(int x, int d, uint32_t inverse) {
  const int q = (int)(((uint64_t)(uint32_t)x * inverse) >> 32);
  return q + (x - q * d >= d);
}
// The share of each of `workers`: total / workers, rounded up; `inverse` as in paged_div_by.
G2_HD int64_t paged_share(int64_t total, int workers, uint32_t inverse) {
  const int64_t x = total + workers - 1;
  const int64_t s = x >> 31 ? x / workers : paged_div_by((int)x, workers, inverse);
  return s < 1 ? 1 : s;
}

// A place in that order: tile `tile` (of `tiles`) of item `item` (of `items`) of sequence
// `seq`. `before` holds the number of tiles per item of all earlier sequences ([n_seqs + 1]).
struct PagedCursor {
  int seq, item, tile, tiles;
};

// The place of tile u, which is one of sequence `seq`'s.
G2_HD PagedCursor paged_place(const int* before, int seq, int items, int64_t u) {
  PagedCursor c;
  c.seq = seq;
  c.tiles = before[seq + 1] - before[seq];
  const int64_t v = u - (int64_t)before[seq] * items;
  c.item = (int)paged_div(v, c.tiles);
  c.tile = (int)(v - (int64_t)c.item * c.tiles);
  return c;
}

// The next place (only when there is one); true when the sequence changed.
G2_HD bool paged_next(PagedCursor& c, const int* before, int items) {
  if (++c.tile < c.tiles) return false;
  c.tile = 0;
  if (++c.item < items) return false;
  c.item = 0;
  do {
    ++c.seq;
    c.tiles = before[c.seq + 1] - before[c.seq];
  } while (c.tiles == 0);
  return true;
}

// n rows of `wa` elements at 0, lda, 2 lda ... and n of `wb` at d, d + ldb ... (host; 0 < wa <= lda
// and 0 < wb <= ldb of any size): whether no element belongs to a row of each. in_place: a row may
// also be the other's of the same index, exactly.
inline bool paged_rows_apart(int64_t lda, int64_t wa, int64_t d, int64_t ldb, int64_t wb, int64_t n, bool in_place) {
  typedef __int128 wide;
  if (d >= (wide)lda * (n - 1) + wa || d + (wide)ldb * (n - 1) + wb <= 0) return true;
  if (in_place && d == 0 && wa == wb && (lda == ldb || n == 1)) return true;
  if (lda == ldb) {
    // row i and row i + m of the other overlap when -wb < d + m ld < wa: two values of m can
    int64_t m = -(d / lda), r = d % lda;
    if (r < 0) r += lda, ++m;  // d + m ld = r
    return !(r < wa && m > -n && m < n) && !(r > lda - wb && m - 1 > -n && m - 1 < n);
  }
  for (int64_t i = 0, j = 0; i < n && j < n;) {  // in the order of their places
    const wide a = (wide)lda * i, b = d + (wide)ldb * j;
    if (a + wa <= b) {
      ++i;
    } else if (b + wb <= a) {
      ++j;
    } else if (in_place && i == j && a == b && wa == wb) {
      ++i, ++j;
    } else {
      return false;
    }
  }
  return true;
}

}  // namespace g2
