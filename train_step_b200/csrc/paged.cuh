// paged.cuh -- the paged key/value cache: appending new tokens' keys and values (with the
// position rotation of keys and queries), and the attention of one new token per sequence
// over the cache.
//
// A cache is a pool of n_pages pages of page_size (a power of two) tokens; token slot s of
// page p holds, for each of NKV heads, hd contiguous elements at
// p * page_stride + s * row_stride + h * head_stride. Sequence b's token t is in page
// table[b * table_stride + t / page_size], slot t % page_size. Page ids are checked where
// they are read: one outside [0, n_pages) raises the status word and the access is skipped.
#pragma once
#include "common.cuh"
#include "decode.cuh"
#include "paged_index.cuh"

namespace g2 {

struct PagedView {
  void *k, *v;
  int64_t page_stride, row_stride, head_stride;  // elements
  const int* table;
  int64_t table_stride;
  int* status;  // nullable
  int n_pages, log2_page, max_pages, n_seqs, nkv, hd;
};

// The page that holds position `pos` (0 <= pos < max_pages * page_size) of sequence `seq`, or
// -1 for a bad id in the table.
__device__ __forceinline__ int paged_page(const PagedView& c, int seq, int pos) {
  const int page = c.table[seq * c.table_stride + (pos >> c.log2_page)];
  return (unsigned)page < (unsigned)c.n_pages ? page : -1;
}

// Bits of the status word, set by kernels.
constexpr int PAGED_OUTSIDE = 1;  // a page id, sequence, position or length outside the cache
constexpr int PAGED_TIMEOUT = 2;  // a bounded wait gave up: results are void, whatever else was met

__device__ __forceinline__ void raise_paged_status(int* status, int bit) {
  if (status) atomicOr(status, bit);
}

// Clears the bits that were read, so that one which a call on another stream sets meanwhile is
// reported the next time.
__global__ void paged_clear_status_kernel(int* status, int bits) { atomicAnd(status, ~bits); }

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
constexpr int PKV_THREADS = 256;
constexpr int PKV_BLOCKS = 8;  // per SM

struct PagedAppendArgs {
  PagedView c;
  const void *k, *v, *q;  // rows of nkv (nh) heads of hd contiguous elements; q nullable
  void* q_out;
  int64_t ldk, ldv, ldq, ldqo;
  int nh;  // query heads (0 without q)
  int rows;
  const int* positions;
  const int* seqs;  // nullable: row n belongs to sequence n
  const float* cos_sin;
  int n_positions, rot;
  int tasks, tasks_per_row;
  uint32_t per_row, per_head;  // inverses of the tasks of a row and of a head, for paged_div_by
};

__device__ __forceinline__ void pkv_unpack(const uint4& r, float (&f)[8], bf16) {
  const float2 a = unpack_bf16x2(r.x), b = unpack_bf16x2(r.y), c = unpack_bf16x2(r.z), d = unpack_bf16x2(r.w);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}
__device__ __forceinline__ void pkv_unpack(const uint4& r, float (&f)[4], float) {
  f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y); f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ uint4 pkv_pack(const float (&f)[8], bf16) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 pkv_pack(const float (&f)[4], float) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// Row n's keys and values go to the slot of (sequence, position); keys and queries are
// rotated on the way: a pair (x, y) of elements becomes (x c - y s, x s + y c) with c, s from
// the table row of the position (rot/2 cosines, then rot/2 sines), computed in fp32 and
// rounded once to T. PAIRS: the pairs are elements (2i, 2i + 1), otherwise (i, i + rot/2);
// elements from rot on are copied. A row with a negative position is padding and touches
// nothing.
// A task is two 16-byte vectors that hold both elements of their pairs (for rotated halves
// vectors rot/2 apart, otherwise neighbours), so every element is read and written once and
// q_out may be q. Bound by HBM: the row is read and written once. A thread reads its vectors
// before it looks up where they go (position, then page, then the table row): the two latencies
// overlap. The grid fills every SM once (a grid of many short blocks spent a fifth of the time
// on starting them), so 32 registers a thread are allowed (rotated halves in bf16 spill 20 bytes
// for it). 16,384 rows of 12 + 12 + 12 heads of 64 in bf16, 151 MB moved: 28.0 us, 5.4 TB/s (a
// plain copy of as many bytes: 24.6 us).
template <class T, bool PAIRS>
__global__ void __launch_bounds__(PKV_THREADS, PKV_BLOCKS) paged_append_kernel(const PagedAppendArgs a) {
  constexpr int VN = 16 / sizeof(T);
  pdl_launch_dependents();
  pdl_wait();
  const int hp = a.c.hd / (2 * VN);   // tasks per head
  const int nrot = a.rot / (2 * VN);  // of which rotated
  const int step = gridDim.x * PKV_THREADS;
  for (int i = blockIdx.x * PKV_THREADS + threadIdx.x; i < a.tasks; i += step) {
    const int r = paged_div_by(i, a.tasks_per_row, a.per_row), t = i - r * a.tasks_per_row;
    const int64_t n = r;
    int hh = paged_div_by(t, hp, a.per_head);
    const int j = t - hh * hp;
    // values are cut into the same pieces as keys
    const bool halves = !PAIRS && j < nrot;
    const int at = halves ? j * VN : j * 2 * VN, gap = halves ? a.rot / 2 : VN;
    const T* src;
    T* dst;
    int64_t head = 0;
    bool turn = j < nrot, cached = true;
    if (hh < a.nh) {
      src = static_cast<const T*>(a.q) + n * a.ldq + hh * a.c.hd;
      dst = static_cast<T*>(a.q_out) + n * a.ldqo + hh * a.c.hd;
      cached = false;
    } else if ((hh -= a.nh) < a.c.nkv) {
      src = static_cast<const T*>(a.k) + n * a.ldk + hh * a.c.hd;
      dst = static_cast<T*>(a.c.k);
      head = hh * a.c.head_stride;
    } else {
      hh -= a.c.nkv;
      src = static_cast<const T*>(a.v) + n * a.ldv + hh * a.c.hd;
      dst = static_cast<T*>(a.c.v);
      head = hh * a.c.head_stride;
      turn = false;
    }
    uint4 va = *reinterpret_cast<const uint4*>(src + at);
    uint4 vb = *reinterpret_cast<const uint4*>(src + at + gap);
    const int pos = a.positions[n];
    if (pos < 0) continue;
    const int seq = a.seqs ? a.seqs[n] : (int)n;
    int page = -1;
    if ((unsigned)seq < (unsigned)a.c.n_seqs && (pos >> a.c.log2_page) < a.c.max_pages &&
        (a.rot == 0 || pos < a.n_positions))
      page = paged_page(a.c, seq, pos);
    if (page < 0) {
      raise_paged_status(a.c.status, PAGED_OUTSIDE);
      continue;
    }
    if (cached) dst += page * a.c.page_stride + (pos & ((1 << a.c.log2_page) - 1)) * a.c.row_stride + head;
    if (turn) {
      // VN cosines and VN sines, for the pairs j * VN ...
      const float* cs = a.cos_sin + (int64_t)pos * a.rot + j * VN;
      float c[VN], s[VN];
#pragma unroll
      for (int e = 0; e < VN; e += 4) {
        const float4 cc = __ldg(reinterpret_cast<const float4*>(cs + e));
        const float4 ss = __ldg(reinterpret_cast<const float4*>(cs + a.rot / 2 + e));
        c[e] = cc.x; c[e + 1] = cc.y; c[e + 2] = cc.z; c[e + 3] = cc.w;
        s[e] = ss.x; s[e + 1] = ss.y; s[e + 2] = ss.z; s[e + 3] = ss.w;
      }
      float x[VN], y[VN];
      pkv_unpack(va, x, T());
      pkv_unpack(vb, y, T());
      if (PAIRS) {
#pragma unroll
        for (int e = 0; e < VN / 2; ++e) {
          const float x0 = x[2 * e], x1 = x[2 * e + 1], y0 = y[2 * e], y1 = y[2 * e + 1];
          x[2 * e] = x0 * c[e] - x1 * s[e];
          x[2 * e + 1] = x0 * s[e] + x1 * c[e];
          y[2 * e] = y0 * c[VN / 2 + e] - y1 * s[VN / 2 + e];
          y[2 * e + 1] = y0 * s[VN / 2 + e] + y1 * c[VN / 2 + e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < VN; ++e) {
          const float x0 = x[e], y0 = y[e];
          x[e] = x0 * c[e] - y0 * s[e];
          y[e] = x0 * s[e] + y0 * c[e];
        }
      }
      va = pkv_pack(x, T());
      vb = pkv_pack(y, T());
    }
    *reinterpret_cast<uint4*>(dst + at) = va;
    *reinterpret_cast<uint4*>(dst + at + gap) = vb;
  }
}

// ---------------------------------------------------------------------------
// attention of one new token per sequence
// ---------------------------------------------------------------------------
struct PagedAttnArgs {
  PagedView c;
  const void* q;
  void* out;
  float* lse;  // nullable, [n_seqs][nh]
  int64_t ldq, ldo;
  int nh;
  const int* lens;
  int window, sinks;
  // scale * log2 e, and scale divided by it (about ln 2) as a sum of two: maxima are held in log2
  // units, and these give them back without the error of a rounded constant
  float scale_log2, ln_hi, ln_lo;
};

// The weights 2^(s - m) of an item are multiplied by 2^-pat_above: they are at most 2^8 (the
// maximum m may lag by 8) and there are 2^4 in each of the item's tiles, so their sum stays below 1
// and a weighted sum of values within the values' own range (without it values of 1e36 overflowed).
// (The same as an offset of m saves the product, but rounds the exponents of the weights that count:
// fp32 outputs of 2,000 keys were off by 1.5e-7 for 0.9e-7, at the same speed.)
__device__ __forceinline__ int pat_above(int tiles) { return 12 + (32 - __clz(tiles)); }
__device__ __forceinline__ float pat_exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// The natural logarithm of l 2^(m + above), m in the units of scale_log2 (l = 0: no visible key).
__device__ __forceinline__ float pat_lse(const PagedAttnArgs& a, float m, float l, int above) {
  if (l == 0.f) return -INFINITY;
  const int e = (int)(__float_as_uint(l) >> 23) - 126;  // l > 0 is far above the subnormal numbers, or NaN
  return fmaf(m, a.ln_hi, fmaf(m, a.ln_lo, fmaf((float)(above + e), 0.69314718056f, logf(l * pat_exp2i(-e)))));
}

// Work split. A call has one item per (sequence, key head, tile of up to QR query heads of
// that key head's group), or per (sequence, HP key heads with their groups) where heads are
// small; an item is a run of 16-key tiles over its visible keys. The tiles of
// all items are laid end to end and every warp of the grid (a worker) takes an equal,
// contiguous share of them, so ragged lengths balance without the host knowing them. A worker
// that takes an item whole writes its output. Otherwise it leaves pieces in shared memory: at
// most one that begins inside an item (its head piece) and one that begins with an item and does
// not reach its end (its tail piece). When a block's workers are done, the block joins the pieces
// of each split item: to its output, or, for an item spread over several blocks, to a partial
// result in the workspace (at most two per block: of the item that comes in from the block
// before, slot 0, and of the one that goes on in the next, slot 1). The block that arrives last
// at such an item joins its partial results, in their order, so results do not depend on the
// order of arrival. (A second kernel for the join cost 3 us more per call.)
// A worker streams its tiles through a ring of its own in shared memory, STAGES tiles ahead and
// on into the next item (the queries of an item arrive with its first tile); it needs no barrier
// but its own mbarriers and the warp's. With pages of 16 tokens or more (BOX) a tile is one
// rectangle of a page and arrives by tensor copies that one lane issues; smaller pages, and
// strides that a tensor map does not take, go through 16-byte copies by all lanes.
// What bounds it. Long caches: reading them from HBM; 128 sequences of 512 to 8,192 tokens with 8
// key heads of 128 (1.46 GB) take 225 us, 6.5 TB/s, as fast as a plain copy moves bytes. Before
// that it was the instructions of a warp: two or three warps per scheduler, each a chain of
// dependent steps, of which 16-byte copies by all lanes were half (300 us). Shorter ones: the
// chain of lengths, place, page, copy, first tile (3.5 us) and, when items cross blocks, arrival
// and join (3 to 4 us): 16 sequences of 1,024 tokens, 12 heads of 64 (50 MB) take 16.5 us, of
// which 7 us stream; one of 100 tokens 5.5 us.
// Pages that keep each head's tokens together read faster than pages of whole tokens, whose rows
// of 128 bytes are far apart (12 and 25 heads of 64: 94 % against 86 and 76 % of the copy rate).
constexpr int PAT_MAX_BLOCKS = 256;
constexpr int PAT_SMEM = 226 * 1024;  // of a block

template <class T, int HD, int QR_, int HP_ = 1>
struct PatShape {
  static constexpr int QR = QR_;              // query rows of a key head, at most
  static constexpr int HP = HP_;              // key heads of an item
  static constexpr int ROW = HD * sizeof(T);  // bytes
  static constexpr int CPR = ROW / 16;        // 16-byte chunks per row
  // keys (and values) of a tile: for each key head, boxes of 16 rows of up to 128 bytes
  static constexpr int BOX_ROW = ROW < 128 ? ROW : 128;
  static constexpr int BOXES = (ROW + BOX_ROW - 1) / BOX_ROW;
  static constexpr int BOX = PAT_TILE * BOX_ROW;
  static constexpr int SUB = BOXES * BOX;  // one key head
  static constexpr int TILE = HP * SUB;
  static_assert(HP == 1 || BOXES == 1, "several heads in one copy");
  static constexpr int STAGES = 2;  // 3: 224 -> 244 us on the 1.46 GB above, with as many warps
  // fp32: a copy of the item's queries and the tile's weights, per warp
  static constexpr int SIDE = sizeof(T) == 4 ? QR * ROW + QR * PAT_TILE * 4 : 0;
  // a piece: outputs, then (maximum, sum), of each row; a warp: its ring of keys and values
  // (after the last tile: the tail piece), of queries, the head piece, the side buffers, the
  // mbarriers and the validity masks of the stages
  __host__ __device__ static constexpr int piece(int rows) { return rows * HD * 4 + (rows * 8 + 15) / 16 * 16; }
  static constexpr int RING = STAGES * 2 * TILE;
  __host__ __device__ static constexpr int head(int rows) { return RING + STAGES * rows * ROW; }
  __host__ __device__ static constexpr int warp_bytes(int rows) {
    return (head(rows) + piece(rows) + SIDE + STAGES * 12 + 1023) / 1024 * 1024;
  }
  // workers of a block: as many as fit beside the n_seqs + 1 counts (the first 1024 bytes align
  // the rest), in equal numbers for the SM's four schedulers where there are two or three each
  // (8 for 10 that fit: 92.5 -> 88.5 us for one sequence of 131,071 tokens)
  static constexpr int warps(int rows, int n_seqs) {
    const int fit = (PAT_SMEM - 1024 - (n_seqs + 1) * 4) / warp_bytes(rows);
    return fit >= 12 ? 12 : fit >= 8 ? 8 : fit;
  }
  // an item of at most so many tiles (128 KB of keys and values) is not split between blocks.
  // Splitting never, or always, against this (1 to 128 sequences of 64 to 8,192 tokens, heads of
  // 32, 64 and 128): one sequence of 256 tokens, 12 heads of 64, 8.3 us split and 6.5 whole, of 512
  // 8.1 and 7.8, of 1,024 8.5 and 10.6. Of 158 such cases the rule is within 3 % of the better side
  // in 129, behind it by up to 13 % (0.2 to 0.8 us) where sequences of up to 128 tokens need no
  // join either way, and by up to 19 % (2.4 us) where 16 sequences of 1,024 to 2,048 tokens, whole,
  // would leave just a few SMs idle (8 heads of 128, 16 of 32).
  static constexpr int WHOLE = 131072 / (2 * TILE);
  static constexpr int smem(int rows, int n_seqs) {
    return 1024 + warps(rows, n_seqs) * warp_bytes(rows) + (n_seqs + 1) * 4;
  }
  // the fewest rows that come to this shape
  static constexpr int MIN_ROWS = HP > 1 ? HP : sizeof(T) == 2 ? (QR == 16 ? 9 : 1) : QR == 8 ? 5 : QR == 4 ? 2 : 1;
  static constexpr int MAX_WARPS = warps(MIN_ROWS, 1);

  // 16-byte chunk `c` of row `r` in a tile: the order in which a tensor copy with 128-byte (64-byte
  // for 64-byte rows) swizzling leaves it; consecutive rows of a chunk are in different banks
  __device__ static __forceinline__ int chunk(int r, int c) {
    if (BOX_ROW == 128) return (c >> 3) * BOX + r * 128 + (((c ^ r) & 7) << 4);
    return r * BOX_ROW + ((c ^ ((r >> 1) & 3)) << 4);
  }
};

struct PagedAttnPlan {
  int warps;    // of a block
  int workers, items, qtiles, group, rows;  // rows: HP min(QR, group), the rows of a partial result
  uint32_t per_item, per_worker, per_block; // inverses of items, workers and blocks, for paged_div_by
  unsigned long long tag;                   // of this call, above the bits of PAT_COUNT
  unsigned long long* arrived;              // [blocks]: see pat_claim
  float2* ml;                               // [blocks][2][rows]: maximum (log2 units) and sum
  float* part;                              // [blocks][2][rows][HD]
};

// The blocks that share an item count their arrivals in the word of its first block; the last to
// arrive joins the item. A word belongs to a call while it carries the call's tag: every block
// that will arrive at a word claims it first (early, and read earlier still, so that nothing waits
// for it), whatever it holds; of several claims one succeeds, and no block can have taken the
// last arrival before the others have claimed. The last one clears the word,
// so that a captured call may run again with the same tag. No block waits for another.
// (Measured and dropped: counting by compare-and-swap, a microsecond for each block that arrives
// at the same time; a flag per block with a fence between setting and looking, 1.2 us more.)
constexpr unsigned long long PAT_COUNT = 0xffffull;
__device__ __forceinline__ unsigned long long pat_look(const unsigned long long* word) {
  return *reinterpret_cast<const volatile unsigned long long*>(word);
}
__device__ __forceinline__ void pat_claim(unsigned long long* word, unsigned long long seen, unsigned long long tag) {
  if ((seen & ~PAT_COUNT) != tag) atomicCAS(word, seen, tag);
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// before[b] = tiles per item of sequences 0..b-1, for b <= n_seqs (whole block); returns the
// largest number of tiles of an item. Up to 32 sequences: every warp writes all of the same
// counts, and waits for nobody.
__device__ __forceinline__ int pat_prefix(const PagedAttnArgs& a, int* before) {
  if (a.c.n_seqs <= 32) {
    const int lane = threadIdx.x & 31;
    int bad = 0, n = 0;
    if (lane < a.c.n_seqs) {
      n = paged_length(a.lens[lane], a.c.max_pages << a.c.log2_page, &bad);
      n = paged_visible(n, a.window, a.sinks).tiles;
    }
    if (bad && blockIdx.x == 0 && threadIdx.x < 32) raise_paged_status(a.c.status, PAGED_OUTSIDE);
    const int most = __reduce_max_sync(0xffffffffu, n);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += v;
    }
    if (lane < a.c.n_seqs) before[lane + 1] = n;
    if (lane == 0) before[0] = 0;
    __syncwarp();
    return most;
  }
  __shared__ int wsum[32], wmax[32];
  const int threads = blockDim.x, B = a.c.n_seqs, per = (B + threads - 1) / threads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cap = a.c.max_pages << a.c.log2_page;
  const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
  int sum = 0, most = 0, bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = paged_visible(paged_length(a.lens[b], cap, &bad), a.window, a.sinks).tiles;
    before[b + 1] = n;
    sum += n;
    most = max(most, n);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (bad && blockIdx.x == 0) raise_paged_status(a.c.status, PAGED_OUTSIDE);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) {
    wsum[warp] = inc;
    wmax[warp] = most;
  }
  __syncthreads();
  for (int w = 0; w < threads / 32; ++w) most = max(most, wmax[w]);
  int base = inc - sum;
  for (int w = 0; w < warp; ++w) base += wsum[w];
  for (int b = b0; b < b1; ++b) {
    base += before[b + 1];
    before[b + 1] = base;
  }
  if (threadIdx.x == 0) before[0] = 0;
  __syncthreads();
  return most;
}

// The place of tile u of the whole order. Every step of the search looks at 32 counts.
__device__ __forceinline__ PagedCursor pat_locate(const int* before, int n_seqs, const PagedAttnPlan& pl, int64_t u) {
  const int lane = threadIdx.x & 31;
  const int r = u >> 31 ? (int)(u / pl.items) : paged_div_by((int)u, pl.items, pl.per_item);
  int lo = 0, span = n_seqs;  // the sequence is one of lo ... lo + span - 1
  while (span > 1) {
    const int step = (span + 31) >> 5, at = lane * step;
    const int k = __popc(__ballot_sync(0xffffffffu, at < span && before[lo + at] <= r)) - 1;
    lo += k * step;
    span = min(step, span - k * step);
  }
  return paged_place(before, lo, pl.items, u);
}

// The first tile of an item at or after tile u, 0 <= u <= total.
__device__ __forceinline__ int64_t pat_item_start(const int* before, int n_seqs, const PagedAttnPlan& pl, int64_t u,
                                                  int64_t total) {
  if (u >= total) return total;
  const PagedCursor c = pat_locate(before, n_seqs, pl, u);
  return c.tile == 0 ? u : u + (c.tiles - c.tile);
}

// The arithmetic of one worker on an item's tiles. Statistics are kept in log2 units (scores
// times scale * log2 e), sums and outputs in fp32.
template <class T, int HD, int QR>
struct PatWarp;

// bf16: m16n8k16 tensor-core products (a key head has at most 16 query rows: the 128-row products
// of the accumulator-memory kind would be at least 7/8 empty, and S and P would travel through
// that memory). S = Q K^T: the query heads are the 16-row operand, a tile's keys two 8-column
// operands. P V: the weights a lane holds after S are exactly the
// first operand's fragment. The weights are not rounded to one bf16: with up to 8 query heads
// (QR 8) rows 8..15 of the operand, otherwise empty, hold the remainders p - bf16(p), and the
// two halves of the result are added at the end; with up to 16 heads the remainders take a
// second product and sums of their own. P is so carried to 2^-16 of its value, with up to 8 heads
// at no cost (the products are far from the tensor cores' rate: the kernel is bound by reading the
// cache; 12 and 16 heads run at 71 and 58 % of the copy rate, bound by a warp's instructions). A
// remainder may be 0 or negative, and its product with an infinite value NaN or of the other sign;
// where the first half is infinite or NaN, it is the result.
// The running maximum moves only when a tile exceeds it by more than 8 (weights and sums against
// an older maximum are at most 2^8 larger, and as exact), so most tiles do not rescale the output.
template <int HD, int QR>
struct PatWarp<bf16, HD, QR> {
  using S = PatShape<bf16, HD, QR>;
  static constexpr int KS = HD / 16, NT = HD / 8;
  static constexpr int RV = QR / 8;  // query rows a lane holds statistics of
  uint32_t qf[KS][2 * RV];
  float acc[NT][4];   // QR 8: [2], [3] for the remainders
  float rest[NT][4];  // QR 16: the remainders'
  float m[RV], l[RV], down;

  __device__ __forceinline__ void init(char*) {}
  __device__ __forceinline__ void begin(const char* q, int rows, int tiles, int lane) {
    down = pat_exp2i(-pat_above(tiles));
    const uint32_t qs = smem_u32(q);
    // rows 0..7 (and 8..15) of Q as first-operand fragments; rows that do not exist repeat row 0
    // and are not written
    const int mat = lane >> 3, row = lane & 7;
#pragma unroll
    for (int k = 0; k < KS; k += (RV == 1 ? 2 : 1)) {
      uint32_t r[4];
      if constexpr (RV == 1) {  // two k steps: chunks 2k .. 2k + 3 of rows 0..7
        ldsm_x4(qs + (row < rows ? row : 0) * S::ROW + 16 * (2 * k + mat), r);
        qf[k][0] = r[0];
        qf[k][1] = r[1];
        qf[k + 1][0] = r[2];
        qf[k + 1][1] = r[3];
      } else {  // rows 0..7, 8..15 at chunk 2k, then at chunk 2k + 1
        const int at = row + 8 * (mat & 1);
        ldsm_x4(qs + (at < rows ? at : 0) * S::ROW + 16 * (2 * k + (mat >> 1)), r);
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[k][i] = r[i];
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[j][i] = 0.f;
        if (RV == 2) rest[j][i] = 0.f;
      }
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(const char* kt, const char* vt, uint32_t mask, float scale_log2, int lane) {
    const uint32_t ks = smem_u32(kt), vs = smem_u32(vt);
    const int mat = lane >> 3, row = lane & 7, q = lane & 3;
    // even and odd k steps in sums of their own: chains half as long
    float s[2][4], s2[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[0][i] = s[1][i] = s2[0][i] = s2[1][i] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t b[4];  // keys 0..7 at chunks 2k, 2k + 1; keys 8..15 at the same
      ldsm_x4(ks + S::chunk(row + 8 * (mat >> 1), 2 * k + (mat & 1)), b);
      const uint32_t a1 = RV == 2 ? qf[k][1] : 0u, a3 = RV == 2 ? qf[k][2 * RV - 1] : 0u;
      const uint32_t a2 = RV == 2 ? qf[k][2 * RV - 2] : qf[k][1];
      dec_mma(k & 1 ? s2[0] : s[0], qf[k][0], a1, a2, a3, b[0], b[1]);
      dec_mma(k & 1 ? s2[1] : s[1], qf[k][0], a1, a2, a3, b[2], b[3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[0][i] += s2[0][i];
      s[1][i] += s2[1][i];
    }
    // lane: query row lane / 4 (+ 8), keys 2q, 2q + 1 and 8 + 2q, 9 + 2q
    float p[RV][4];
    bool move = false;
    float mx[RV];
#pragma unroll
    for (int r = 0; r < RV; ++r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[r][i] = s[i >> 1][2 * r + (i & 1)] * scale_log2;
      if (mask != 0xffffu) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(mask >> ((i >> 1) * 8 + 2 * q + (i & 1)) & 1)) p[r][i] = -INFINITY;
      }
      float t = fmaxf(fmaxf(p[r][0], p[r][1]), fmaxf(p[r][2], p[r][3]));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
      mx[r] = t;
      move |= t > m[r] + 8.f;
    }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int r = 0; r < RV; ++r) {
        const float mn = fmaxf(m[r], mx[r]);
        const float f = mn == -INFINITY ? 1.f : exp2f(m[r] - mn);
        m[r] = mn;
        l[r] *= f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[j][2 * r] *= f;
          acc[j][2 * r + 1] *= f;
          if (RV == 1) {
            acc[j][2] *= f;
            acc[j][3] *= f;
          } else {
            rest[j][2 * r] *= f;
            rest[j][2 * r + 1] *= f;
          }
        }
      }
    }
    uint32_t hi[RV][2], lo[RV][2];
#pragma unroll
    for (int r = 0; r < RV; ++r) {
      const float ref = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[r][i] = ex2_fast(p[r][i] - ref) * down;
      l[r] += (p[r][0] + p[r][1]) + (p[r][2] + p[r][3]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        hi[r][i] = pack_bf16x2(p[r][2 * i], p[r][2 * i + 1]);
        const float2 h = unpack_bf16x2(hi[r][i]);
        lo[r][i] = pack_bf16x2(p[r][2 * i] - h.x, p[r][2 * i + 1] - h.y);
      }
    }
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      uint32_t b[4];  // keys 0..7, 8..15 at chunk j, then at chunk j + 1
      ldsm_x4_t(vs + S::chunk(row + 8 * (mat & 1), j + (mat >> 1)), b);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (RV == 1) {
          dec_mma(acc[j + e], hi[0][0], lo[0][0], hi[0][1], lo[0][1], b[2 * e], b[2 * e + 1]);
        } else {
          dec_mma(acc[j + e], hi[0][0], hi[RV - 1][0], hi[0][1], hi[RV - 1][1], b[2 * e], b[2 * e + 1]);
          dec_mma(rest[j + e], lo[0][0], lo[RV - 1][0], lo[0][1], lo[RV - 1][1], b[2 * e], b[2 * e + 1]);
        }
      }
    }
  }

  // out.stat(row, m, l, first lane of the row) gives the factor of the row's outputs, which
  // then go to out.pair(row, element, two values)
  template <class O>
  __device__ __forceinline__ void finish(int lane, const O& out) {
#pragma unroll
    for (int r = 0; r < RV; ++r) {
      const int row = (lane >> 2) + 8 * r;
      float sum = l[r];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (row >= out.rows) continue;
      const float f = out.stat(row, m[r], sum, (lane & 3) == 0);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float x = acc[j][2 * r], y = acc[j][2 * r + 1];
        const float xr = RV == 1 ? acc[j][2] : rest[j][2 * r], yr = RV == 1 ? acc[j][3] : rest[j][2 * r + 1];
        if (isfinite(x)) x += xr;
        if (isfinite(y)) y += yr;
        out.pair(row, j * 8 + (lane & 3) * 2, x * f, y * f);
      }
    }
  }
};

// fp32: fp32 products and sums. Scores: a lane has a key and half of the elements; weights go
// to the P V loop through shared memory, where a lane holds HD/32 output elements (neighbours,
// or 32 apart for HD 96). One query head per key head is bound by HBM (12 heads of 64: 91 % of
// the copy rate); with 4 and 8 the shared-memory reads of queries and weights bound it (63 % and
// 45 %; packed pairs of fp32 products were slower for the moves they need).
template <int HD, int QR>
struct PatWarp<float, HD, QR> {
  using S = PatShape<float, HD, QR>;
  static constexpr int CPR = HD / 4, E = HD / 32;
  float acc[QR][E];
  float m[QR], l[QR], down;
  float4* qb;  // [QR][CPR]
  float* wb;   // [QR][PAT_TILE]

  __device__ __forceinline__ void init(char* side) {
    qb = reinterpret_cast<float4*>(side);
    wb = reinterpret_cast<float*>(side + QR * HD * 4);
  }
  __device__ __forceinline__ void begin(const char* qs, int rows, int tiles, int lane) {
    down = pat_exp2i(-pat_above(tiles));
    // the stage is refilled before the item ends
    const float4* from = reinterpret_cast<const float4*>(qs);
    for (int i = lane; i < QR * CPR; i += 32)
      qb[i] = i < rows * CPR ? from[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < QR; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(const char* ks, const char* vs, uint32_t mask, float scale_log2, int lane) {
    const int key = lane & 15, half = lane >> 4;
    float s[QR];
#pragma unroll
    for (int r = 0; r < QR; ++r) s[r] = 0.f;
#pragma unroll 4
    for (int i = 0; i < CPR / 2; ++i) {
      const int c = half * (CPR / 2) + i;
      const float4 k = *reinterpret_cast<const float4*>(ks + S::chunk(key, c));
#pragma unroll
      for (int r = 0; r < QR; ++r) {
        const float4 q = qb[r * CPR + c];
        s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
      }
    }
    const bool seen = mask >> key & 1;
#pragma unroll
    for (int r = 0; r < QR; ++r) {
      s[r] += __shfl_xor_sync(0xffffffffu, s[r], 16);
      s[r] = seen ? s[r] * scale_log2 : -INFINITY;
      // as above, the maximum moves only when a score exceeds it by more than 8; most tiles need
      // one vote per row and no reduction
      if (__any_sync(0xffffffffu, s[r] > m[r] + 8.f)) {
        float t = fmaxf(m[r], s[r]);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
        const float f = exp2f(m[r] - t);
        m[r] = t;
        l[r] *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] *= f;
      }
      const float p = exp2f(s[r] - (m[r] == -INFINITY ? 0.f : m[r])) * down;
      l[r] += p;
      if (half == 0) wb[r * PAT_TILE + key] = p;
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < PAT_TILE; k += 4) {
      float v[4][E];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (E == 4) {
          const float4 x = *reinterpret_cast<const float4*>(vs + S::chunk(k + i, lane));
          v[i][0] = x.x; v[i][1 % E] = x.y; v[i][2 % E] = x.z; v[i][3 % E] = x.w;
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int d = E == 2 ? 2 * lane + e : lane + 32 * e;
            v[i][e] = *reinterpret_cast<const float*>(vs + S::chunk(k + i, d >> 2) + 4 * (d & 3));
          }
        }
      }
#pragma unroll
      for (int r = 0; r < QR; ++r) {
        const float4 p = *reinterpret_cast<const float4*>(wb + r * PAT_TILE + k);
#pragma unroll
        for (int e = 0; e < E; ++e)
          acc[r][e] = fmaf(p.x, v[0][e], fmaf(p.y, v[1][e], fmaf(p.z, v[2][e], fmaf(p.w, v[3][e], acc[r][e]))));
      }
    }
    __syncwarp();  // the weights are read before the next tile writes its own
  }

  template <class O>
  __device__ __forceinline__ void finish(int lane, const O& out) {
#pragma unroll
    for (int r = 0; r < QR; ++r) {
      float sum = l[r];
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (r >= out.rows) continue;
      const float f = out.stat(r, m[r], sum, lane == 0);
#pragma unroll
      for (int e = 0; e < E; ++e) out.one(r, E == 4 ? 4 * lane + e : E == 2 ? 2 * lane + e : lane + 32 * e, acc[r][e] * f);
    }
  }
};

// Where a worker's results for one item go: the output (whole items) or a piece.
template <class T>
struct PatOut {
  const PagedAttnArgs& a;
  int rows;     // query rows of the item
  T* out;       // row 0 of the item's output, or nullptr for a piece
  float* lse;   // its row 0 (nullable)
  float* part;  // row 0 of the piece
  float2* ml;
  int hd;
  int above;
  __device__ __forceinline__ float stat(int row, float m, float l, bool first) const {
    if (!out) {
      if (first) ml[row] = make_float2(m, l);
      return 1.f;
    }
    // l is 0 when every page id was bad
    if (first && lse) lse[row] = pat_lse(a, m, l, above);
    return l == 0.f ? 0.f : 1.f / l;
  }
  __device__ __forceinline__ void pair(int row, int d, float x, float y) const {
    if (out)
      *reinterpret_cast<uint32_t*>(out + row * hd + d) = pack_bf16x2(x, y);
    else
      *reinterpret_cast<float2*>(part + row * hd + d) = make_float2(x, y);
  }
  __device__ __forceinline__ void one(int row, int d, float x) const {
    (out ? reinterpret_cast<float*>(out) : part)[row * hd + d] = x;
  }
};

// A join of softmax pieces: o = sum_i o_i 2^(m_i - M), l = sum_i l_i 2^(m_i - M), M = max m_i, of
// four output elements. Pieces are added N at a time: one rescaling for all of them.
struct PatSum {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  template <int N>
  __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&x)[N]) {
    float mn = m;
#pragma unroll
    for (int i = 0; i < N; ++i) mn = fmaxf(mn, ml[i].x);
    const float ref = mn == -INFINITY ? 0.f : mn;  // nothing visible so far: the weights are 0
    const float f = ex2_fast(m - ref);
    m = mn;
    l *= f;
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float g = ex2_fast(ml[i].x - ref);
      l = fmaf(ml[i].y, g, l);
      o.x = fmaf(x[i].x, g, o.x);
      o.y = fmaf(x[i].y, g, o.y);
      o.z = fmaf(x[i].z, g, o.z);
      o.w = fmaf(x[i].w, g, o.w);
    }
  }
  // to `to`, and the logarithm of the sum to lse (nullable)
  template <class T>
  __device__ __forceinline__ void store(const PagedAttnArgs& a, T* to, float* lse, int tiles) const {
    if (lse) *lse = pat_lse(a, m, l, pat_above(tiles));
    const float f = l == 0.f ? 0.f : 1.f / l;
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
    else
      *reinterpret_cast<float4*>(to) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  }
};

// Joins the partial results of an item of `rows` query rows from blocks c0..c1 by `threads`
// threads, t = 0 ... threads - 1: a thread holds four elements of a row over every parts-th
// block, with PAJ_AHEAD of them in flight. All threads of the block go through the barriers of
// `rounds` rounds; `scratch` has 24 bytes per thread.
constexpr int PAJ_AHEAD = 8;
template <class T, int HD>
__device__ __forceinline__ void pat_join(const PagedAttnArgs& a, const PagedAttnPlan& pl, int c0, int c1, int rows, int tiles,
                                         T* out, float* lse, char* scratch, int t, int threads, int rounds) {
  constexpr int VEC = HD / 4;
  float4* s_o = reinterpret_cast<float4*>(scratch);
  float2* s_ml = reinterpret_cast<float2*>(scratch + 16 * blockDim.x);
  const int cols = rows * VEC, n = c1 - c0 + 1;
  // the same for a whole and a half block, so that sums do not depend on who joins
  const int parts = max(1, min((int)blockDim.x / 2 / cols, (n + PAJ_AHEAD - 1) / PAJ_AHEAD));
  for (int k = 0; k < rounds; ++k) {
    const int p = cols <= threads ? t / cols : 0, col = cols <= threads ? t - p * cols : k * threads + t;
    const bool mine = t < threads && p < parts && col < cols;
    const int row = col / VEC, v = col - row * VEC;
    PatSum sum;
    if (mine) {
      for (int c = c0 + p; c <= c1; c += parts * PAJ_AHEAD) {
        float2 ml[PAJ_AHEAD];
        float4 x[PAJ_AHEAD];
#pragma unroll
        for (int j = 0; j < PAJ_AHEAD; ++j) {
          const int cj = c + j * parts;
          const int64_t i = ((int64_t)cj * 2 + (cj == c0 ? 1 : 0)) * pl.rows + row;
          ml[j] = make_float2(-INFINITY, 0.f);
          x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (cj <= c1) {
            ml[j] = __ldcg(pl.ml + i);
            x[j] = __ldcg(reinterpret_cast<const float4*>(pl.part + i * HD) + v);
          }
        }
        sum.add(ml, x);
      }
      s_o[threadIdx.x] = sum.o;
      s_ml[threadIdx.x] = make_float2(sum.m, sum.l);
    }
    __syncthreads();
    if (mine && p == 0) {
      for (int i = 1; i < parts; ++i) {
        const float2 ml[1] = {s_ml[threadIdx.x + i * cols]};
        const float4 x[1] = {s_o[threadIdx.x + i * cols]};
        sum.add(ml, x);
      }
      sum.store(a, out + row * HD + v * 4, lse && v == 0 ? lse + row : nullptr, tiles);
    }
    __syncthreads();
  }
}

template <class T, int HD, int QR, int HP, bool BOX>
__global__ void __launch_bounds__(PatShape<T, HD, QR, HP>::MAX_WARPS * 32, 1)
    paged_attn_kernel(const PagedAttnArgs a, const PagedAttnPlan pl, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  using S = PatShape<T, HD, QR, HP>;
  static_assert(HP == 1 || BOX, "several heads come by tensor copies");
  constexpr int CPR = S::CPR, STAGES = S::STAGES, VN = 16 / sizeof(T);
  constexpr uint64_t LIMIT_NS = 2000000000ull;  // a wait gives up after two seconds
  extern __shared__ char pat_raw[];
  char* pat_smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(pat_raw) + 1023) & ~uintptr_t(1023));
  // items that are split, for the joins: [0] the one that begins before the block's first
  // worker, [1 + warp] the one that begins in a warp and does not end there (seq < 0: none)
  struct Split {
    int seq, h, rows;    // its query heads
    int tiles;
    int b0, b1, p0, p1;  // its blocks, and the warps of this block that have a piece of it
  };
  __shared__ Split s_split[S::MAX_WARPS + 1];
  __shared__ int s_cross[2];  // which of them other blocks share: the one that comes in, that goes on (-1: none)
  __shared__ int s_last[2];   // this block is the last to arrive at it
  __shared__ int s_no_abort;
  __shared__ int64_t s_edge[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  char* ring = pat_smem + warp * S::warp_bytes(pl.rows);
  char* head = ring + S::head(pl.rows);
  char* side = head + S::piece(pl.rows);
  uint64_t* bars = reinterpret_cast<uint64_t*>(side + S::SIDE);
  uint32_t* masks = reinterpret_cast<uint32_t*>(bars + STAGES);
  int* before = reinterpret_cast<int*>(pat_smem + pl.warps * S::warp_bytes(pl.rows));
  if (lane == 0) {
    if (BOX) {
#pragma unroll
      for (int i = 0; i < STAGES; ++i) mbar_init(bars + i, 1);
      fence_barrier_init();
    }
    s_split[warp + 1].seq = -1;
    if (warp == 0) {
      if (BOX) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
      }
      s_split[0].seq = -1;
      s_cross[0] = s_cross[1] = -1;
      s_last[0] = s_last[1] = s_no_abort = 0;
    }
  }
  pdl_launch_dependents();
  __syncthreads();  // the shared words are set
  pdl_wait();       // nothing above touches global memory
  // the arrival words of the items that may go on (0) and come in (1), by the block's first thread
  unsigned long long* word[2] = {pl.arrived + blockIdx.x, nullptr};
  unsigned long long seen_word[2] = {0ull, 0ull};
  if (threadIdx.x == 0) seen_word[0] = pat_look(word[0]);
  const int most = pat_prefix(a, before);
  const int B = a.c.n_seqs;
  // sequences without tokens
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (before[b] == before[b + 1])
      for (int i = threadIdx.x; i < a.nh * HD; i += blockDim.x) {
        static_cast<T*>(a.out)[b * a.ldo + i] = from_f32<T>(0.f);
        if (a.lse && i < a.nh) a.lse[(int64_t)b * a.nh + i] = -INFINITY;
      }
  // the block's tiles [a0, a1), of which each of its warps takes `share`: equal ranges, or, when
  // every item is small, the items that begin in an equal range, so that no item is shared with
  // another block (arriving and joining cost 3 us, a small item more than the others' 1 us)
  const int64_t total = (int64_t)before[B] * pl.items;
  int64_t range, share, a0, a1;
  if (most <= S::WHOLE) {
    range = paged_share(total, gridDim.x, pl.per_block);
    for (int i = warp; i < 2; i += pl.warps) {
      const int64_t edge = pat_item_start(before, B, pl, min(total, (blockIdx.x + i) * range), total);
      if (lane == 0) s_edge[i] = edge;
    }
    __syncthreads();
    a0 = s_edge[0];
    a1 = s_edge[1];
    share = max((int)(a1 - a0 + pl.warps - 1) / pl.warps, 1);
  } else {
    share = paged_share(total, pl.workers, pl.per_worker);
    range = share * pl.warps;
    a0 = min(total, blockIdx.x * range);
    a1 = min(total, a0 + range);
  }
  if (a0 >= a1) return;  // a block without work
  const int64_t u0 = a0 + warp * share, u1 = min(a1, u0 + share);
  if (u0 < u1) {
    const int64_t n = u1 - u0;
    // copies: tile `pc`; the pages of its keys have been read a tile ahead (BOX: the one page, by
    // all lanes; otherwise the page of key `lane`, by the first 16)
    PagedCursor pc = pat_locate(before, B, pl, u0);
    const PagedCursor first = pc;
    if (threadIdx.x == 0 && first.tile > 0) {
      word[1] = pl.arrived + (int)paged_div(u0 - first.tile, range);
      seen_word[1] = pat_look(word[1]);
    }
    const int cap = a.c.max_pages << a.c.log2_page, slots = (1 << a.c.log2_page) - 1;
    int bad = 0, ignore = 0;
    PagedVisible vis = paged_visible(paged_length(a.lens[pc.seq], cap, &ignore), a.window, a.sinks);
    int page = 0, pos = 0;  // of the tile
    auto look_up = [&]() {
      pos = paged_tile_pos(vis, pc.tile);
      const int mine = BOX ? pos : pos + lane;
      if (BOX || (lane < PAT_TILE && mine < vis.len))
        // (the bound: a length that changes during the call must not lead out of the table)
        page = a.c.table[pc.seq * a.c.table_stride + min(mine >> a.c.log2_page, a.c.max_pages - 1)];
    };
    // the item's first key head, the first row of its tile of the group, its query rows
    auto heads = [&](const PagedCursor& at, int& hk, int& q0, int& rows) {
      const int k = pl.qtiles == 1 ? at.item : at.item / pl.qtiles;
      hk = k * HP;
      q0 = (at.item - k * pl.qtiles) * QR;
      rows = HP == 1 ? min(QR, pl.group - q0) : min(HP, a.c.nkv - hk) * pl.group;
    };
    auto copy_tile = [&](int stage, bool with_q) {
      const uint32_t seen = paged_tile_mask(vis, pos);
      int hk, q0, rows;
      heads(pc, hk, q0, rows);
      const T* q = static_cast<const T*>(a.q) + pc.seq * a.ldq + (hk * pl.group + q0) * HD;
      char* qs = ring + S::RING + stage * pl.rows * S::ROW;
      char* ks = ring + stage * 2 * S::TILE;
      if constexpr (BOX) {
        const bool ok = (unsigned)page < (unsigned)a.c.n_pages;
        bad |= !ok;
        if (lane == 0) {
          masks[stage] = ok ? seen : 0u;
          const uint32_t bytes = (ok ? 2 * S::TILE : 0) + (with_q ? rows * S::ROW : 0);
          if (bytes)
            mbar_arrive_expect_tx(bars + stage, bytes);
          else
            mbar_arrive(bars + stage);
          if (ok) {
#pragma unroll
            for (int i = 0; i < S::BOXES; ++i) {
              const int x = i * (S::BOX_ROW / (int)sizeof(T));
              tma_load_4d(ks + i * S::BOX, &kmap, bars + stage, x, pos & slots, hk, page);
              tma_load_4d(ks + S::TILE + i * S::BOX, &vmap, bars + stage, x, pos & slots, hk, page);
            }
          }
          if (with_q) bulk_load_1d(qs, q, rows * S::ROW, bars + stage);
        }
      } else {
        const bool in = lane < PAT_TILE && (seen >> lane & 1);
        const bool ok = in && (unsigned)page < (unsigned)a.c.n_pages;
        bad |= in && !ok;
        const uint32_t mask = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) masks[stage] = mask;
        int64_t off = 0;
        if (ok) off = page * a.c.page_stride + ((pos + lane) & slots) * a.c.row_stride + hk * a.c.head_stride;
        const uint32_t dst = smem_u32(ks);
#pragma unroll
        for (int j = 0; j < PAT_TILE * CPR / 32; ++j) {
          const int c = lane + 32 * j, row = c / CPR, col = c % CPR;
          const bool valid = mask >> row & 1;
          const int64_t o = __shfl_sync(0xffffffffu, (long long)off, row) + (valid ? col * VN : 0);
          const uint32_t to = dst + S::chunk(row, col);
          cp_async_16(to, static_cast<const T*>(a.c.k) + o, valid);
          cp_async_16(to + S::TILE, static_cast<const T*>(a.c.v) + o, valid);
        }
        if (with_q)
          for (int c = lane; c < rows * CPR; c += 32) cp_async_16(smem_u32(qs) + 16 * c, q + c * VN, true);
      }
    };
    auto forward = [&]() {
      if (paged_next(pc, before, pl.items))
        vis = paged_visible(paged_length(a.lens[pc.seq], cap, &ignore), a.window, a.sinks);
      look_up();
    };
    look_up();
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      if (s < n) {
        copy_tile(s, s == 0 || pc.tile == 0);
        if (s + 1 < n) forward();
      }
      if (!BOX) cp_async_commit();
    }

    if (threadIdx.x == 0) {
      pat_claim(word[0], seen_word[0], pl.tag);
      if (word[1]) pat_claim(word[1], seen_word[1], pl.tag);
    }
    PagedCursor c = first;
    PatWarp<T, HD, QR> pw[HP];
#pragma unroll
    for (int i = 0; i < HP; ++i) pw[i].init(side);
    int stage = 0, from = 0;
    uint32_t parity = 0;
    bool dead = false;
    for (int64_t t = 0; t < n; ++t) {
      if constexpr (BOX) {
        const bool ok = dead || mbar_wait_bounded(bars + stage, parity, &s_no_abort, LIMIT_NS);
        if (__any_sync(0xffffffffu, !ok)) {
          // a copy did not arrive: no more copies and waits, the result is void and reported; the
          // copies in flight are waited for once more, so that none outlives the block
          dead = true;
          bad = 2;
          for (int i = 0; i < STAGES && t + i < n; ++i) {
            const int s = stage + i < STAGES ? stage + i : stage + i - STAGES;
            mbar_wait_bounded(bars + s, stage + i < STAGES ? parity : parity ^ 1u, &s_no_abort, LIMIT_NS);
          }
          __syncwarp();
        }
      } else {
        cp_async_wait<STAGES - 1>();
        __syncwarp();
      }
      char* ks = ring + stage * 2 * S::TILE;
      const uint32_t mask = masks[stage];
      if (BOX && mask != 0xffffu) {
        // what a page holds in place of unseen keys may be anything: their weights are 0, and
        // their values must not be infinite or NaN
        for (int i = lane; i < HP * PAT_TILE * CPR; i += 32) {
          const int row = i / CPR % PAT_TILE;
          if (!(mask >> row & 1))
            *reinterpret_cast<uint4*>(ks + S::TILE + i / (PAT_TILE * CPR) * S::SUB + S::chunk(row, i % CPR)) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();  // before the next copy into this stage
        __syncwarp();
      }
      if (t == 0 || c.tile == 0) {
        // the rows that have arrived: what the others' places hold must not count in the warp's votes
        const int rows = HP > 1 || pl.qtiles == 1 ? pl.rows / HP : min(QR, pl.group - c.item % pl.qtiles * QR);
#pragma unroll
        for (int i = 0; i < HP; ++i)
          pw[i].begin(ring + S::RING + (stage * pl.rows + i * pl.group) * S::ROW, rows, c.tiles, lane);
        from = c.tile;
      }
#pragma unroll
      for (int i = 0; i < HP; ++i) pw[i].tile(ks + i * S::SUB, ks + S::TILE + i * S::SUB, mask, a.scale_log2, lane);
      __syncwarp();
      if (t + STAGES < n && !dead) {
        copy_tile(stage, pc.tile == 0);
        if (t + STAGES + 1 < n) forward();
      }
      if (!BOX) cp_async_commit();
      const bool end = c.tile == c.tiles - 1;
      if (end || t == n - 1) {
        int hk, q0, rows;
        heads(c, hk, q0, rows);
        const int h = hk * pl.group + q0;
        const bool whole = end && from == 0;
        // the tail piece goes to the ring, which is done with
        char* piece = from == 0 ? ring : head;
#pragma unroll
        for (int i = 0; i < HP; ++i) {
          const int r0 = i * pl.group;  // its first row
          PatOut<T> out{a};
          out.rows = HP == 1 ? rows : min(pl.group, rows - r0);
          out.out = whole ? static_cast<T*>(a.out) + c.seq * a.ldo + (h + r0) * HD : nullptr;
          out.lse = a.lse ? a.lse + (int64_t)c.seq * a.nh + h + r0 : nullptr;
          out.part = reinterpret_cast<float*>(piece) + r0 * HD;
          out.ml = reinterpret_cast<float2*>(piece + pl.rows * HD * 4) + r0;
          out.hd = HD;
          out.above = pat_above(c.tiles);
          pw[i].finish(lane, out);
        }
        if (!whole && lane == 0 && (from == 0 || warp == 0)) {
          const int64_t start = u0 + t - c.tile, last = start + c.tiles - 1;  // the item's first and last tile
          const int k = from == 0 ? warp + 1 : 0;
          Split sp{c.seq, h, rows, c.tiles, (int)blockIdx.x, (int)blockIdx.x, from == 0 ? warp : 0, pl.warps - 1};
          if (last < a1) sp.p1 = (int)paged_div(last - a0, share);
          if (k == 0) sp.b0 = (int)paged_div(start, range);
          if (last >= a1) sp.b1 = (int)paged_div(last, range);
          s_split[k] = sp;
          if (k == 0 || last >= a1) s_cross[k > 0] = k;
        }
      }
      if (t + 1 < n) paged_next(c, before, pl.items);
      if (++stage == STAGES) {
        stage = 0;
        parity ^= 1u;
      }
    }
    if (!BOX) cp_async_wait<0>();
    if (bad) raise_paged_status(a.c.status, bad == 2 ? PAGED_TIMEOUT : PAGED_OUTSIDE);
  }
  __syncthreads();
  // a thread joins four elements of a split item's row over the block's pieces
  constexpr int VEC = HD / 4;
  const int cols = pl.rows * VEC, bytes = S::warp_bytes(pl.rows), tail = S::head(pl.rows);
  const uint32_t there = __ballot_sync(0xffffffffu, lane <= pl.warps && s_split[min(lane, pl.warps)].seq >= 0);
  for (int i = threadIdx.x; i < __popc(there) * cols; i += blockDim.x) {
    const int nth = i / cols, col = i - nth * cols, row = col / VEC, v = col - row * VEC;
    uint32_t left = there;  // without its first nth
    for (int j = 0; j < nth; ++j) left &= left - 1;
    const int k = __ffs(left) - 1;
    const Split sp = s_split[k];
    if (row >= sp.rows) continue;
    PatSum sum;
    for (int p = sp.p0; p <= sp.p1; p += 4) {
      float2 ml[4];
      float4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ml[j] = make_float2(-INFINITY, 0.f);
        x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p + j <= sp.p1) {  // all pieces but the one that begins the item are head pieces
          const char* piece = pat_smem + (p + j) * bytes + (k > 0 && p + j == sp.p0 ? 0 : tail);
          ml[j] = reinterpret_cast<const float2*>(piece + pl.rows * HD * 4)[row];
          x[j] = reinterpret_cast<const float4*>(piece)[col];
        }
      }
      sum.add(ml, x);
    }
    if (k > 0 && sp.b1 == (int)blockIdx.x) {
      sum.store(a, static_cast<T*>(a.out) + sp.seq * a.ldo + sp.h * HD + col * 4,
                a.lse && v == 0 ? a.lse + (int64_t)sp.seq * a.nh + sp.h + row : nullptr, sp.tiles);
    } else {
      const int64_t slot = ((int64_t)blockIdx.x * 2 + (k > 0 ? 1 : 0)) * pl.rows;
      reinterpret_cast<float4*>(pl.part + slot * HD)[col] = sum.o;
      if (v == 0) pl.ml[slot + row] = make_float2(sum.m, sum.l);
    }
  }
  if (s_cross[0] < 0 && s_cross[1] < 0) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();  // the block's partial results, before its arrivals
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (s_cross[i] < 0) continue;
      const Split sp = s_split[s_cross[i]];
      unsigned long long* word = pl.arrived + sp.b0;
      const unsigned long long old = atomicAdd(word, 1ull);
      if ((int)(old & PAT_COUNT) != sp.b1 - sp.b0) continue;
      s_last[i] = 1;
      *word = 0ull;
    }
    __threadfence();  // those of the blocks that arrived before
  }
  __syncthreads();
  if (!s_last[0] && !s_last[1]) return;
  // two items: half of the threads each
  const bool both = s_last[0] && s_last[1];
  const int threads = both ? blockDim.x / 2 : blockDim.x;
  const int i = both ? (int)threadIdx.x >= threads : !s_last[0];
  const Split sp = s_split[s_cross[i]];
  pat_join<T, HD>(a, pl, sp.b0, sp.b1, sp.rows, sp.tiles, static_cast<T*>(a.out) + sp.seq * a.ldo + sp.h * HD,
                  a.lse ? a.lse + (int64_t)sp.seq * a.nh + sp.h : nullptr, pat_smem, threadIdx.x - (both ? i * threads : 0),
                  threads, (cols + threads - 1) / threads);
}

}  // namespace g2
