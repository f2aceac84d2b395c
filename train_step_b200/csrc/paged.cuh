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

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
constexpr int PKV_THREADS = 256;
constexpr int PKV_MAX_ROWS = 32;  // rows of one block

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
  int rows_per_block, tasks_per_row;
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
// q_out may be q. Bound by HBM: the row is read and written once.
template <class T, bool PAIRS>
__global__ void __launch_bounds__(PKV_THREADS) paged_append_kernel(const PagedAppendArgs a) {
  constexpr int VN = 16 / sizeof(T);
  __shared__ int64_t s_off[PKV_MAX_ROWS];  // element offset of the slot, -1: skip the row
  __shared__ int s_pos[PKV_MAX_ROWS];
  const int row0 = blockIdx.x * a.rows_per_block;
  const int nrows = min(a.rows_per_block, a.rows - row0);
  if ((int)threadIdx.x < nrows) {
    const int n = row0 + threadIdx.x;
    const int pos = a.positions[n];
    int64_t off = -1;
    if (pos >= 0) {
      const int seq = a.seqs ? a.seqs[n] : n;
      int page = -1;
      if ((unsigned)seq < (unsigned)a.c.n_seqs && (pos >> a.c.log2_page) < a.c.max_pages &&
          (a.rot == 0 || pos < a.n_positions))
        page = paged_page(a.c, seq, pos);
      if (page >= 0)
        off = page * a.c.page_stride + (pos & ((1 << a.c.log2_page) - 1)) * a.c.row_stride;
      else
        raise_device_error(a.c.status, DEV_PAGE_RANGE);
    }
    s_off[threadIdx.x] = off;
    s_pos[threadIdx.x] = pos;
  }
  __syncthreads();
  const int hp = a.c.hd / (2 * VN);      // tasks per head
  const int nrot = a.rot / (2 * VN);     // of which rotated
  const int total = nrows * a.tasks_per_row;
  for (int i = blockIdx.y * PKV_THREADS + threadIdx.x; i < total; i += gridDim.y * PKV_THREADS) {
    const int r = i / a.tasks_per_row, t = i - r * a.tasks_per_row;
    const int64_t off = s_off[r];
    if (off < 0) continue;
    const int hh = t / hp, j = t - hh * hp;
    const int64_t n = row0 + r;
    const T* src;
    T* dst;
    bool turn = j < nrot;
    if (hh < a.nh) {
      src = static_cast<const T*>(a.q) + n * a.ldq + hh * a.c.hd;
      dst = static_cast<T*>(a.q_out) + n * a.ldqo + hh * a.c.hd;
    } else if (hh < a.nh + a.c.nkv) {
      const int h = hh - a.nh;
      src = static_cast<const T*>(a.k) + n * a.ldk + h * a.c.hd;
      dst = static_cast<T*>(a.c.k) + off + h * a.c.head_stride;
    } else {
      const int h = hh - a.nh - a.c.nkv;
      src = static_cast<const T*>(a.v) + n * a.ldv + h * a.c.hd;
      dst = static_cast<T*>(a.c.v) + off + h * a.c.head_stride;
      turn = false;
    }
    int ia = j * 2 * VN, ib = ia + VN;
    if (turn && !PAIRS) {
      ia = j * VN;
      ib = a.rot / 2 + ia;
    } else if (!PAIRS && j < nrot) {
      ia = j * VN;  // a value head: the same pieces, copied
      ib = a.rot / 2 + ia;
    }
    uint4 va = *reinterpret_cast<const uint4*>(src + ia);
    uint4 vb = *reinterpret_cast<const uint4*>(src + ib);
    if (turn) {
      // VN cosines and VN sines, for the pairs j * VN ...
      const float* cs = a.cos_sin + (int64_t)s_pos[r] * a.rot + j * VN;
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
    *reinterpret_cast<uint4*>(dst + ia) = va;
    *reinterpret_cast<uint4*>(dst + ib) = vb;
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
  float scale;
  int window, sinks;
};

// Work split. A call has one item per (sequence, key head, tile of up to QR query heads of
// that key head's group); an item is a run of 16-key tiles over its visible keys. The tiles of
// all items are laid end to end and every warp of the grid (a worker) takes an equal share of
// them, so ragged lengths balance without the host knowing them. A worker that takes an item
// whole writes its output; pieces of an item go to the workspace and are joined by
// paged_join_kernel. Each worker has at most one piece that begins inside an item and reaches
// its end (slot 0) and one that does not reach the end (slot 1).
// A worker streams its tiles through a ring of its own in shared memory with 16-byte
// asynchronous copies, STAGES - 1 tiles ahead and on into the next item (the queries of an
// item arrive with its first tile); it needs no barrier but the warp's.
constexpr int PAT_MAX_WORKERS = 2048;
constexpr int PAT_LEAST = 4;  // tiles of a share
constexpr int PAT_SMEM = 184 * 1024;  // of the rings of a block

template <class T, int HD, int QR_>
struct PatShape {
  static constexpr int QR = QR_;               // query rows of an item
  static constexpr int ROW = HD * sizeof(T);   // bytes
  static constexpr int CPR = ROW / 16;         // 16-byte chunks per row
  static constexpr int QOFF = 2 * PAT_TILE * ROW;
  static constexpr int STAGE = QOFF + QR * ROW;  // keys, values, queries
  static constexpr int STAGES = STAGE > 16384 ? 2 : STAGE > 12288 ? 3 : 4;
  static constexpr int FIT = PAT_SMEM / (STAGES * STAGE);
  static constexpr int WARPS = FIT > 12 ? 12 : FIT;
  // fp32: a copy of the item's queries and the tile's weights, per warp
  static constexpr int SIDE = sizeof(T) == 4 ? QR * ROW + QR * PAT_TILE * 4 : 0;
  // per warp: ring, side buffers, the validity masks of the stages
  static constexpr int WARP_BYTES = STAGES * STAGE + SIDE + 16 * ((STAGES + 3) / 4);
  static constexpr size_t smem(int n_seqs) { return (size_t)WARPS * WARP_BYTES + ((size_t)n_seqs + 1) * 4; }
};

struct PagedAttnPlan {
  int workers, items, qtiles, group, rows;  // rows: min(QR, group), the rows of a partial result
  int* rec;                                 // [workers][2]: split item that begins in a worker, its last worker
  float2* ml;                               // [workers][2][rows]: maximum (log2 units) and sum
  float* part;                              // [workers][2][rows][HD]
};

// chunk `c` of row `r` in a tile: consecutive rows at one chunk fall into different banks
template <int CPR>
__device__ __forceinline__ int pat_chunk(int r, int c) {
  return r * CPR + (CPR % 8 == 0 ? c ^ (r & 7) : c ^ ((r >> 1) & 3));
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

// before[b] = tiles per item of sequences 0..b-1, for b <= n_seqs (whole block).
template <int THREADS>
__device__ __forceinline__ void pat_prefix(const PagedAttnArgs& a, int* before) {
  __shared__ int wsum[THREADS / 32];
  const int B = a.c.n_seqs, per = (B + THREADS - 1) / THREADS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cap = a.c.max_pages << a.c.log2_page;
  const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
  int sum = 0, bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = paged_tiles(paged_visible(paged_length(a.lens[b], cap, &bad), a.window, a.sinks).count);
    before[b + 1] = n;
    sum += n;
  }
  if (bad && blockIdx.x == 0) raise_device_error(a.c.status, DEV_PAGE_RANGE);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int base = inc - sum;
  for (int w = 0; w < warp; ++w) base += wsum[w];
  for (int b = b0; b < b1; ++b) {
    base += before[b + 1];
    before[b + 1] = base;
  }
  if (threadIdx.x == 0) before[0] = 0;
  __syncthreads();
}

// The arithmetic of one worker on an item's tiles. Statistics are kept in log2 units (scores
// times scale * log2 e), sums and outputs in fp32.
template <class T, int HD, int QR>
struct PatWarp;

// bf16: m16n8k16 tensor-core products. S = Q K^T: the query heads are the 16-row operand, a
// tile's keys two 8-column operands. P V: the weights a lane holds after S are exactly the
// first operand's fragment. The weights are not rounded to one bf16: with up to 8 query heads
// (QR 8) rows 8..15 of the operand, otherwise empty, hold the remainders p - bf16(p), and the
// two halves of the result are added at the end; with up to 16 heads the remainders take a
// second product. P is so carried to 2^-16 of its value at no or little cost (the products
// are far from the tensor cores' rate: the kernel is bound by reading the cache).
// The running maximum moves only when a tile exceeds it by more than 8 (weights stay below
// 2^8, exact enough in fp32), so most tiles do not rescale the output.
template <int HD, int QR>
struct PatWarp<bf16, HD, QR> {
  static constexpr int CPR = HD / 8, KS = HD / 16, NT = HD / 8;
  static constexpr int RV = QR / 8;  // query rows a lane holds statistics of
  uint32_t qf[KS][2 * RV];
  float acc[NT][4];
  float m[RV], l[RV];

  __device__ __forceinline__ PatWarp(char*) {}
  __device__ __forceinline__ void begin(const char* q, int lane) {
    const uint32_t qs = smem_u32(q);
    // rows 0..7 (and 8..15) of Q as first-operand fragments
#pragma unroll
    for (int k = 0; k < KS; k += (RV == 1 ? 2 : 1)) {
      uint32_t r[4];
      const int mat = lane >> 3, row = lane & 7;
      if constexpr (RV == 1) {  // two k steps: chunks 2k .. 2k + 3 of rows 0..7
        ldsm_x4(qs + 16 * pat_chunk<CPR>(row, 2 * k + mat), r);
        qf[k][0] = r[0];
        qf[k][1] = r[1];
        qf[k + 1][0] = r[2];
        qf[k + 1][1] = r[3];
      } else {  // rows 0..7, 8..15 at chunk 2k, then at chunk 2k + 1
        ldsm_x4(qs + 16 * pat_chunk<CPR>(row + 8 * (mat & 1), 2 * k + (mat >> 1)), r);
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[k][i] = r[i];
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(const char* kt, const char* vt, uint32_t mask, float scale_log2, int lane) {
    const uint32_t ks = smem_u32(kt), vs = smem_u32(vt);
    const int mat = lane >> 3, row = lane & 7, q = lane & 3;
    float s[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[0][i] = s[1][i] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t b[4];  // keys 0..7 at chunks 2k, 2k + 1; keys 8..15 at the same
      ldsm_x4(ks + 16 * pat_chunk<CPR>(row + 8 * (mat >> 1), 2 * k + (mat & 1)), b);
      const uint32_t a1 = RV == 2 ? qf[k][1] : 0u, a3 = RV == 2 ? qf[k][2 * RV - 1] : 0u;
      const uint32_t a2 = RV == 2 ? qf[k][2 * RV - 2] : qf[k][1];
      dec_mma(s[0], qf[k][0], a1, a2, a3, b[0], b[1]);
      dec_mma(s[1], qf[k][0], a1, a2, a3, b[2], b[3]);
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
          }
        }
      }
    }
    uint32_t hi[RV][2], lo[RV][2];
#pragma unroll
    for (int r = 0; r < RV; ++r) {
      const float ref = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[r][i] = ex2_fast(p[r][i] - ref);
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
      ldsm_x4_t(vs + 16 * pat_chunk<CPR>(row + 8 * (mat & 1), j + (mat >> 1)), b);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (RV == 1) {
          dec_mma(acc[j + e], hi[0][0], lo[0][0], hi[0][1], lo[0][1], b[2 * e], b[2 * e + 1]);
        } else {
          dec_mma(acc[j + e], hi[0][0], hi[RV - 1][0], hi[0][1], hi[RV - 1][1], b[2 * e], b[2 * e + 1]);
          dec_mma(acc[j + e], lo[0][0], lo[RV - 1][0], lo[0][1], lo[RV - 1][1], b[2 * e], b[2 * e + 1]);
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
        if (RV == 1) {
          x += acc[j][2];
          y += acc[j][3];
        }
        out.pair(row, j * 8 + (lane & 3) * 2, x * f, y * f);
      }
    }
  }
};

// fp32: fp32 products and sums. Scores: a lane has a key and half of the elements; weights go
// to the P V loop through shared memory, where a lane holds HD/32 output elements (neighbours,
// or 32 apart for HD 96).
template <int HD, int QR>
struct PatWarp<float, HD, QR> {
  static constexpr int CPR = HD / 4, E = HD / 32;
  float acc[QR][E];
  float m[QR], l[QR];
  float4* qb;  // [QR][CPR]
  float* wb;   // [QR][PAT_TILE]

  __device__ __forceinline__ PatWarp(char* side) {
    qb = reinterpret_cast<float4*>(side);
    wb = reinterpret_cast<float*>(side + QR * HD * 4);
  }
  __device__ __forceinline__ void begin(const char* qs, int lane) {
    // the stage is refilled before the item ends
    const float4* from = reinterpret_cast<const float4*>(qs);
    for (int i = lane; i < QR * CPR; i += 32) qb[i] = from[pat_chunk<CPR>(i / CPR, i % CPR)];
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
    const float4* kt = reinterpret_cast<const float4*>(ks);
    const int key = lane & 15, half = lane >> 4;
    float s[QR];
#pragma unroll
    for (int r = 0; r < QR; ++r) s[r] = 0.f;
#pragma unroll 4
    for (int i = 0; i < CPR / 2; ++i) {
      const int c = half * (CPR / 2) + i;
      const float4 k = kt[pat_chunk<CPR>(key, c)];
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
      float t = s[r];
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
      if (t > m[r]) {  // the same for all lanes
        const float f = exp2f(m[r] - t);
        m[r] = t;
        l[r] *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] *= f;
      }
      const float p = exp2f(s[r] - (m[r] == -INFINITY ? 0.f : m[r]));
      l[r] += p;
      if (half == 0) wb[r * PAT_TILE + key] = p;
    }
    __syncwarp();
    const float* vt = reinterpret_cast<const float*>(vs);
#pragma unroll
    for (int k = 0; k < PAT_TILE; k += 4) {
      float v[4][E];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (E == 4) {
          const float4 x = reinterpret_cast<const float4*>(vt)[pat_chunk<CPR>(k + i, lane)];
          v[i][0] = x.x; v[i][1 % E] = x.y; v[i][2 % E] = x.z; v[i][3 % E] = x.w;
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int d = E == 2 ? 2 * lane + e : lane + 32 * e;
            v[i][e] = vt[4 * pat_chunk<CPR>(k + i, d >> 2) + (d & 3)];
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

// Where a worker's results for one item go: the output (whole items) or a partial result.
template <class T>
struct PatOut {
  int rows;     // query rows of the item
  T* out;       // row 0 of the item's output, or nullptr for a partial result
  float* lse;   // its row 0 (nullable)
  float* part;  // row 0 of the partial result
  float2* ml;
  int hd;
  __device__ __forceinline__ float stat(int row, float m, float l, bool first) const {
    if (!out) {
      if (first) ml[row] = make_float2(m, l);
      return 1.f;
    }
    // l is 0 when every page id was bad
    if (first && lse) lse[row] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
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

template <class T, int HD, int QR>
__global__ void __launch_bounds__(PatShape<T, HD, QR>::WARPS * 32, 1)
    paged_attn_kernel(const PagedAttnArgs a, const PagedAttnPlan pl) {
  using S = PatShape<T, HD, QR>;
  constexpr int CPR = S::CPR, STAGES = S::STAGES, VN = 16 / sizeof(T);
  extern __shared__ __align__(128) char pat_smem[];
  int* before = reinterpret_cast<int*>(pat_smem + S::WARPS * S::WARP_BYTES);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  char* ring = pat_smem + warp * S::WARP_BYTES;
  uint32_t* masks = reinterpret_cast<uint32_t*>(ring + STAGES * S::STAGE + S::SIDE);
  pdl_launch_dependents();
  pat_prefix<S::WARPS * 32>(a, before);
  const int B = a.c.n_seqs;
  // sequences without tokens
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (before[b] == before[b + 1])
      for (int i = threadIdx.x; i < a.nh * HD; i += S::WARPS * 32) {
        static_cast<T*>(a.out)[b * a.ldo + i] = from_f32<T>(0.f);
        if (a.lse && i < a.nh) a.lse[(int64_t)b * a.nh + i] = -INFINITY;
      }
  const int w = warp * gridDim.x + blockIdx.x;
  const int64_t total = (int64_t)before[B] * pl.items;
  const int64_t share = paged_share(total, pl.workers, PAT_LEAST);
  const int64_t u0 = w * share, u1 = min(total, u0 + share);
  if (u0 >= u1) {
    if (lane == 0) pl.rec[2 * w + 1] = -1;
    return;
  }
  const int64_t n = u1 - u0;

  // copies: tile `pc`, whose keys' pages the first 16 lanes have read a tile ahead
  PagedCursor pc = paged_locate(before, B, pl.items, u0);
  const PagedCursor first = pc;
  const int cap = a.c.max_pages << a.c.log2_page, slots = (1 << a.c.log2_page) - 1;
  int bad = 0, ignore = 0;
  PagedVisible vis = paged_visible(paged_length(a.lens[pc.seq], cap, &ignore), a.window, a.sinks);
  int page = 0;
  auto look_up = [&]() {
    const int i = pc.tile * PAT_TILE + lane;
    if (lane < PAT_TILE && i < vis.count)
      page = a.c.table[pc.seq * a.c.table_stride + (paged_position(vis, i) >> a.c.log2_page)];
  };
  auto copy_tile = [&](int stage, bool with_q) {
    const uint32_t dst = smem_u32(ring + stage * S::STAGE);
    const int i = pc.tile * PAT_TILE + lane;
    const bool in = lane < PAT_TILE && i < vis.count;
    const bool ok = in && (unsigned)page < (unsigned)a.c.n_pages;
    bad |= in && !ok;
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) masks[stage] = mask;
    const int hk = pc.item / pl.qtiles;
    int64_t off = 0;
    if (ok) off = page * a.c.page_stride + (paged_position(vis, i) & slots) * a.c.row_stride + hk * a.c.head_stride;
#pragma unroll
    for (int j = 0; j < PAT_TILE * CPR / 32; ++j) {
      const int c = lane + 32 * j, row = c / CPR, col = c % CPR;
      const bool valid = mask >> row & 1;
      const int64_t o = __shfl_sync(0xffffffffu, (long long)off, row) + (valid ? col * VN : 0);
      const uint32_t to = dst + 16 * pat_chunk<CPR>(row, col);
      cp_async_16(to, static_cast<const T*>(a.c.k) + o, valid);
      cp_async_16(to + PAT_TILE * S::ROW, static_cast<const T*>(a.c.v) + o, valid);
    }
    if (with_q) {
      const int q0 = (pc.item - hk * pl.qtiles) * QR;  // first row of the tile in the group
      const T* q = static_cast<const T*>(a.q) + pc.seq * a.ldq + (hk * pl.group + q0) * HD;
      for (int c = lane; c < QR * CPR; c += 32) {
        const int row = c / CPR, col = c % CPR;
        const bool valid = q0 + row < pl.group;
        cp_async_16(dst + S::QOFF + 16 * pat_chunk<CPR>(row, col), valid ? q + row * HD + col * VN : a.q, valid);
      }
    }
  };
  auto forward = [&]() {
    if (paged_next(pc, before, pl.items))
      vis = paged_visible(paged_length(a.lens[pc.seq], cap, &ignore), a.window, a.sinks);
    look_up();
  };
  look_up();
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    if (s < n) {
      copy_tile(s, s == 0 || pc.tile == 0);
      if (s + 1 < n) forward();
    }
    cp_async_commit();
  }

  PagedCursor c = first;
  const float scale_log2 = a.scale * 1.4426950408889634f;
  PatWarp<T, HD, QR> pw(ring + STAGES * S::STAGE);
  int stage = 0, from = 0, split = -1;
  for (int64_t t = 0; t < n; ++t) {
    cp_async_wait<STAGES - 2>();
    __syncwarp();
    if (t + STAGES - 1 < n) {
      copy_tile(stage == 0 ? STAGES - 1 : stage - 1, pc.tile == 0);
      if (t + STAGES < n) forward();
    }
    cp_async_commit();
    const char* buf = ring + stage * S::STAGE;
    if (t == 0 || c.tile == 0) {
      pw.begin(buf + S::QOFF, lane);
      from = c.tile;
    }
    pw.tile(buf, buf + PAT_TILE * S::ROW, masks[stage], scale_log2, lane);
    const bool end = c.tile == c.tiles - 1;
    if (end || t == n - 1) {
      const int hk = c.item / pl.qtiles, q0 = (c.item - hk * pl.qtiles) * QR, h = hk * pl.group + q0;
      const bool whole = end && from == 0;
      const int64_t slot = ((int64_t)w * 2 + (end ? 0 : 1)) * pl.rows;
      PatOut<T> out;
      out.rows = min(QR, pl.group - q0);
      out.out = whole ? static_cast<T*>(a.out) + c.seq * a.ldo + h * HD : nullptr;
      out.lse = a.lse ? a.lse + (int64_t)c.seq * a.nh + h : nullptr;
      out.part = pl.part + slot * HD;
      out.ml = pl.ml + slot;
      out.hd = HD;
      pw.finish(lane, out);
      if (!end && from == 0) split = c.seq * pl.items + c.item;
    }
    if (t + 1 < n) paged_next(c, before, pl.items);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  if (bad) raise_device_error(a.c.status, DEV_PAGE_RANGE);
  if (lane == 0) {
    // the item that this worker begins and does not end: its last tile's worker
    int last = -1;
    if (split >= 0) {
      const int64_t end = u1 + (c.tiles - 1 - c.tile);  // c is still at tile u1 - 1
      last = (int)((end - 1) / share);
      pl.rec[2 * w] = split;
    }
    pl.rec[2 * w + 1] = last;
  }
}

// Joins the partial results of the items that begin in workers 8 blockIdx.x ... + 7 and go on in
// later ones: o = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M), M = max m_i. A block does the
// rows blockIdx.y, + gridDim.y, ...; a thread holds four output elements over every PARTS-th
// partial result, with the loads of PAJ_AHEAD of them in flight.
constexpr int PAJ_THREADS = 256, PAJ_WORKERS = 8, PAJ_AHEAD = 4;
template <class T, int HD>
__global__ void __launch_bounds__(PAJ_THREADS) paged_join_kernel(const PagedAttnArgs a, const PagedAttnPlan pl, int qr) {
  constexpr int VEC = HD / 4, PARTS = PAJ_THREADS / VEC;
  __shared__ float4 s_o[PARTS][VEC];
  __shared__ float2 s_ml[PARTS];
  __shared__ int2 s_rec[PAJ_WORKERS];
  pdl_wait();
  const int base = blockIdx.x * PAJ_WORKERS;
  if (threadIdx.x < PAJ_WORKERS)
    s_rec[threadIdx.x] =
        base + (int)threadIdx.x < pl.workers ? *reinterpret_cast<const int2*>(pl.rec + 2 * (base + threadIdx.x)) : make_int2(0, -1);
  __syncthreads();
  const int v = threadIdx.x % VEC, p = threadIdx.x / VEC;
  for (int k = 0; k < PAJ_WORKERS; ++k) {
    const int w0 = base + k, w1 = s_rec[k].y;
    if (w1 < 0) continue;
    const int id = s_rec[k].x, b = id / pl.items, item = id - b * pl.items;
    const int hk = item / pl.qtiles, q0 = (item - hk * pl.qtiles) * qr, rows = min(qr, pl.group - q0);
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
      if (p < PARTS) {
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = w0 + p; w <= w1; w += PARTS * PAJ_AHEAD) {
          float2 ml[PAJ_AHEAD];
          float4 x[PAJ_AHEAD];
#pragma unroll
          for (int j = 0; j < PAJ_AHEAD; ++j) {
            const int wj = w + j * PARTS;
            const int64_t i = ((int64_t)wj * 2 + (wj == w1 ? 0 : 1)) * pl.rows + r;
            ml[j] = make_float2(-INFINITY, 0.f);
            if (wj <= w1) {
              ml[j] = pl.ml[i];
              x[j] = *reinterpret_cast<const float4*>(pl.part + i * HD + v * 4);
            }
          }
#pragma unroll
          for (int j = 0; j < PAJ_AHEAD; ++j) {
            const float mn = fmaxf(m, ml[j].x);
            if (ml[j].x == -INFINITY) continue;  // past the end, or nothing visible in the piece
            const float f = exp2f(m - mn), g = exp2f(ml[j].x - mn);
            m = mn;
            l = l * f + ml[j].y * g;
            o.x = o.x * f + x[j].x * g;
            o.y = o.y * f + x[j].y * g;
            o.z = o.z * f + x[j].z * g;
            o.w = o.w * f + x[j].w * g;
          }
        }
        s_o[p][v] = o;
        if (v == 0) s_ml[p] = make_float2(m, l);
      }
      __syncthreads();
      if (p == 0) {
        float M = -INFINITY;
        for (int i = 0; i < PARTS; ++i) M = fmaxf(M, s_ml[i].x);
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < PARTS; ++i) {
          const float2 ml = s_ml[i];
          if (ml.x == -INFINITY) continue;
          const float g = exp2f(ml.x - M);
          const float4 x = s_o[i][v];
          l += ml.y * g;
          o.x += x.x * g;
          o.y += x.y * g;
          o.z += x.z * g;
          o.w += x.w * g;
        }
        const float f = l == 0.f ? 0.f : 1.f / l;
        const int h = hk * pl.group + q0 + r;
        T* out = static_cast<T*>(a.out) + b * a.ldo + h * HD + v * 4;
        out[0] = from_f32<T>(o.x * f);
        out[1] = from_f32<T>(o.y * f);
        out[2] = from_f32<T>(o.z * f);
        out[3] = from_f32<T>(o.w * f);
        if (a.lse && v == 0) a.lse[(int64_t)b * a.nh + h] = l == 0.f ? -INFINITY : M * 0.6931471805599453f + logf(l);
      }
      __syncthreads();
    }
  }
}

}  // namespace g2
