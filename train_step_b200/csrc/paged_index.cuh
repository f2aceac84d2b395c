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

// The tokens that the newest of `len` tokens sees, as positions: the first `sink`, then the
// contiguous range that ends at len - 1. The i-th visible token (0 <= i < count) is at
// position i for i < sink and i + shift otherwise.
struct PagedVisible {
  int sink, shift, count;
};

// len tokens cached, of which the newest has just been appended; window <= 0: all of them
// are visible; otherwise the newest `window`, and the first `sinks` besides.
G2_HD PagedVisible paged_visible(int len, int window, int sinks) {
  PagedVisible v;
  const int lo = window > 0 && len > window ? len - window : 0;
  v.sink = sinks < lo ? sinks : lo;
  v.shift = lo - v.sink;
  v.count = len - v.shift;
  return v;
}

G2_HD int paged_position(const PagedVisible& v, int i) { return i < v.sink ? i : i + v.shift; }

// A sequence length as read from device memory, brought into [0, capacity]; *bad is set when
// it was outside.
G2_HD int paged_length(int len, int capacity, int* bad) {
  if (len < 0 || len > capacity) {
    *bad = 1;
    return len < 0 ? 0 : capacity;
  }
  return len;
}

// The work of one attention call is cut into tiles of PAT_TILE visible keys of one item (a
// sequence, a key head and a tile of its query heads), laid end to end: sequence by sequence,
// item by item. Worker w takes tiles [w * share, (w + 1) * share).
constexpr int PAT_TILE = 16;
G2_HD int paged_tiles(int count) { return (count + PAT_TILE - 1) / PAT_TILE; }
G2_HD int64_t paged_share(int64_t total, int workers, int least) {
  const int64_t s = (total + workers - 1) / workers;
  return s < least ? least : s;
}

// A place in that order: tile `tile` (of `tiles`) of item `item` (of `items`) of sequence
// `seq`. `before` holds the number of tiles per item of all earlier sequences ([n_seqs + 1]).
struct PagedCursor {
  int seq, item, tile, tiles;
};

// The place of tile u of the whole order, 0 <= u < items * before[n_seqs].
G2_HD PagedCursor paged_locate(const int* before, int n_seqs, int items, int64_t u) {
  const int r = (int)(u / items);  // the sequence with before[seq] <= r < before[seq + 1]
  int lo = 0, hi = n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= r)
      lo = mid;
    else
      hi = mid - 1;
  }
  PagedCursor c;
  c.seq = lo;
  c.tiles = before[lo + 1] - before[lo];
  const int64_t v = u - (int64_t)before[lo] * items;
  c.item = (int)(v / c.tiles);
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

}  // namespace g2
