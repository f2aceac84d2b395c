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

}  // namespace g2
