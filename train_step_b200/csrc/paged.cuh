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

constexpr int PAT_THREADS = 128;

// One block per (query head, sequence): each warp takes every fourth visible key, a lane
// holds hd/32 elements of the query, the key and the output; running maximum m and sum l of
// the softmax per warp, joined through shared memory at the end.
template <class T, int HD>
__global__ void __launch_bounds__(PAT_THREADS) paged_attn_kernel(const PagedAttnArgs a) {
  constexpr int E = HD / 32, NW = PAT_THREADS / 32;
  __shared__ float s_m[NW], s_l[NW], s_o[NW][HD];
  const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = h / (a.nh / a.c.nkv);
  int bad = 0;
  const int len = paged_length(a.lens[b], a.c.max_pages << a.c.log2_page, &bad);
  const PagedVisible vis = paged_visible(len, a.window, a.sinks);
  float q[E], o[E];
  const T* qp = static_cast<const T*>(a.q) + (int64_t)b * a.ldq + h * HD;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = to_f32<T>(qp[lane + 32 * e]) * a.scale * 1.4426950408889634f;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int i = warp; i < vis.count; i += NW) {
    const int pos = paged_position(vis, i);
    const int page = paged_page(a.c, b, pos);
    if (page < 0) {
      bad = 1;
      continue;
    }
    const int64_t off =
        page * a.c.page_stride + (pos & ((1 << a.c.log2_page) - 1)) * a.c.row_stride + hk * a.c.head_stride;
    const T* kp = static_cast<const T*>(a.c.k) + off;
    const T* vp = static_cast<const T*>(a.c.v) + off;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], to_f32<T>(kp[lane + 32 * e]), s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s);
    if (mn == -INFINITY) continue;
    const float r = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * r + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * r + p * to_f32<T>(vp[lane + 32 * e]);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
    if (bad) raise_device_error(a.c.status, DEV_PAGE_RANGE);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane + 32 * e] = o[e];
  __syncthreads();
  float M = s_m[0];
  for (int w = 1; w < NW; ++w) M = fmaxf(M, s_m[w]);
  float L = 0.f;
  for (int w = 0; w < NW; ++w)
    if (s_m[w] != -INFINITY) L += s_l[w] * exp2f(s_m[w] - M);
  for (int d = threadIdx.x; d < HD; d += PAT_THREADS) {
    float acc = 0.f;
    for (int w = 0; w < NW; ++w)
      if (s_m[w] != -INFINITY) acc += s_o[w][d] * exp2f(s_m[w] - M);
    static_cast<T*>(a.out)[(int64_t)b * a.ldo + h * HD + d] = from_f32<T>(L > 0.f ? acc / L : 0.f);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(int64_t)b * a.nh + h] = L > 0.f ? M * 0.6931471805599453f + logf(L) : -INFINITY;
}

}  // namespace g2
