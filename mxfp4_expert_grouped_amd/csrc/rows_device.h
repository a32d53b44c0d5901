// Which rows are whose: what the kernels of the 16-bit products share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxmoe {
namespace rows {

// Rows of a matrix from its two offsets: clamped into [0, rows] and never
// running backwards, so that no value of the offsets reaches outside a buffer.
__device__ __forceinline__ void clamp_rows(int rows, int& lo, int& hi) {
  lo = min(max(lo, 0), rows);
  hi = max(lo, min(max(hi, 0), rows));
}
__device__ __forceinline__ void mat_rows(const int* offsets, int e, int rows, int& lo, int& hi) {
  lo = 0;
  hi = rows;
  if (!offsets) return;
  lo = offsets[e];
  hi = offsets[e + 1];
  clamp_rows(rows, lo, hi);
}

// The rows from the first to the last that any matrix has (lo == hi: none
// has), found by a workgroup of THREADS; part: two words of LDS per wave.
template <int THREADS>
__device__ __forceinline__ void covered_rows(const int* offsets, int mats, int rows, int& lo, int& hi, int* part) {
  lo = rows;
  hi = 0;
  for (int e = threadIdx.x; e < mats; e += THREADS) {
    int l, h;
    mat_rows(offsets, e, rows, l, h);
    if (l < h) {
      lo = min(lo, l);
      hi = max(hi, h);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor(lo, o, 64));
    hi = max(hi, __shfl_xor(hi, o, 64));
  }
  if ((threadIdx.x & 63) == 0) {
    part[2 * (threadIdx.x >> 6)] = lo;
    part[2 * (threadIdx.x >> 6) + 1] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    lo = min(lo, part[2 * w]);
    hi = max(hi, part[2 * w + 1]);
  }
  hi = max(lo, hi);
}

// whether every row of a matrix is on 16 bytes
__device__ __forceinline__ bool rows_on_16(const void* p, int64_t ld_bytes) {
  return (reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld_bytes)) % 16 == 0;
}

}  // namespace rows
}  // namespace mxmoe
