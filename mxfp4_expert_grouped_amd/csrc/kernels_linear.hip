// Product of two MXFP4 matrices, y[r] = A[r] W[e(r)]^T with fp32 accumulation:
// moe_linear_mx4.  e(r) is the matrix whose rows [offsets[e], offsets[e+1])
// hold r (rows sorted by expert), or the one matrix there is.
//
// The products run on the scaled MFMA with both operands FP4 (format 4).  The
// weights are its first operand, so that a lane's results are four
// consecutive columns of one row of y.  Layout of one 16x16x128 step:
// lane (r = lane%16, g = lane/16) holds elements 32g .. 32g+31 of row r, which
// is 16 bytes of canonical codes and exactly one scale byte; the result of
// lane l, register i is (weight row 4(l/16)+i, activation row l%16).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "internal.h"
#include "row_types.h"

namespace mxmoe {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v8i fp4_operand(uint4 v) {
  v8i r = {};
  r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
  return r;
}

__device__ __forceinline__ v4f mfma_fp4(uint4 a, uint4 b, v4f c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a), fp4_operand(b), c, 4, 4, 0,
                                                          static_cast<int>(sa), 0, static_cast<int>(sb));
}

constexpr int kMaxMats = 1024;

// Rows of matrix e as the kernels see them: clamped into [0, rows] and never
// running backwards within a matrix, so that no value of the offsets reaches
// outside A and y.
__device__ __forceinline__ void mat_rows(const LinearArgs& a, int e, int& lo, int& hi) {
  const int rows = static_cast<int>(a.rows);
  if (!a.offsets) {
    lo = 0;
    hi = rows;
    return;
  }
  lo = min(max(a.offsets[e], 0), rows);
  hi = max(lo, min(max(a.offsets[e + 1], 0), rows));
}

// prefix[e] = row tiles (of TM rows) of the matrices before e, for e <= mats;
// one pass of the whole workgroup.  Returns the number of tiles.
template <int THREADS, int TM>
__device__ __forceinline__ int tile_prefix(const LinearArgs& a, int* prefix, int* part) {
  constexpr int PER = kMaxMats / THREADS;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    int lo = 0, hi = 0;
    if (e < a.mats) mat_rows(a, e, lo, hi);
    n[i] = (hi - lo + TM - 1) / TM;
    sum += n[i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(inc, o, 64);
    if (lane >= o) inc += u;
  }
  if (lane == 63) part[wave] = inc;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    before += w < wave ? part[w] : 0;
    total += part[w];
  }
  int at = before + inc - sum;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    if (e <= a.mats && e < kMaxMats) prefix[e] = at;
    at += n[i];
  }
  if (tid == 0) prefix[a.mats] = total;
  __syncthreads();
  return total;
}

// The matrix of tile t: the last e with prefix[e] <= t (a matrix without rows
// shares its prefix with the next).  A wave looks at 64 entries at a time.
__device__ __forceinline__ int tile_matrix(const int* prefix, int mats, int t) {
  const int lane = threadIdx.x & 63;
  int e = 0;
  for (int b = 0; b < mats; b += 64) {
    const bool le = b + lane < mats && prefix[b + lane] <= t;
    const uint64_t m = __ballot(le);
    e += __popcll(m);
    if (m != ~uint64_t(0)) break;
  }
  return __builtin_amdgcn_readfirstlane(e - 1);
}

// four consecutive columns of one row of y
template <typename T>
__device__ __forceinline__ void store_cols(T* y, int64_t ld, int row, int col, int n, bool wide, v4f v) {
  T* p = y + int64_t(row) * ld + col;
  if (wide && col + 3 < n) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + i < n) p[i] = from_f32<T>(v[i]);
}

// ---------------------------------------------------------------------------
// A few rows per matrix: weight streaming.  A unit is 16 rows x 16 columns; a
// persistent grid takes them round-robin, the columns of a tile fastest, so
// that neighbouring workgroups stream neighbouring weight rows.  The four
// waves of a workgroup share a unit's K: wave w takes the 512-wide groups w,
// w + 4, ... (256 bytes of each of 16 weight rows, straight from memory to
// registers in operand order), and the four partial sums meet in LDS in wave
// order.  Bound by the weights' bytes.
//
// SCALES: how the scale bytes come.  0: 16 bytes for a row's four steps
// (k % 512 == 0); 1: a dword per step (k % 128 == 0); 2: single bytes, with
// the last step's missing blocks left out (any multiple of 32).
// ---------------------------------------------------------------------------
constexpr int kStreamThreads = 256, kStreamWaves = kStreamThreads / 64;

template <typename T, int SCALES>
__global__ void __launch_bounds__(kStreamThreads, 4) k_linear_stream(LinearArgs a, bool wide) {
  __shared__ int prefix[kMaxMats + 1];
  __shared__ int part[kStreamWaves];
  __shared__ float4 sums[kStreamWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int tiles = tile_prefix<kStreamThreads, 16>(a, prefix, part);
  const int cblocks = (a.n + 15) / 16;
  const int64_t units = int64_t(tiles) * cblocks;
  const int nb = a.k / 32;                     // blocks of 32 along k
  const int groups = (nb + 15) / 16;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int t = static_cast<int>(u / cblocks), cb = static_cast<int>(u - int64_t(t) * cblocks);
    const int e = tile_matrix(prefix, a.mats, t);
    int lo, hi;
    mat_rows(a, e, lo, hi);
    lo += (t - prefix[e]) * 16;
    const int row = lo + r16, col = cb * 16 + r16;
    const bool row_ok = row < hi, col_ok = col < a.n;
    const uint8_t* ap = a.a_c + int64_t(row) * (a.k / 2);
    const uint8_t* as = a.a_s + int64_t(row) * nb;
    const int64_t wrow = int64_t(e) * a.n + col;
    const uint8_t* wp = a.w_c + wrow * (a.k / 2);
    const uint8_t* ws = a.w_s + wrow * nb;
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int q = wave; q < groups; q += kStreamWaves) {
      uint4 wv[4], av[4];
      uint32_t wsc[4], asc[4];
      if constexpr (SCALES == 0) {
        uint4 x = make_uint4(0, 0, 0, 0), z = x;
        if (col_ok) x = *reinterpret_cast<const uint4*>(ws + 16 * q);
        if (row_ok) z = *reinterpret_cast<const uint4*>(as + 16 * q);
        wsc[0] = x.x; wsc[1] = x.y; wsc[2] = x.z; wsc[3] = x.w;
        asc[0] = z.x; asc[1] = z.y; asc[2] = z.z; asc[3] = z.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int kb = 16 * q + 4 * i + g;     // this lane's block
        const bool in = kb < nb;
        wv[i] = av[i] = make_uint4(0, 0, 0, 0);
        if (in && col_ok) wv[i] = *reinterpret_cast<const uint4*>(wp + 16 * int64_t(kb));
        if (in && row_ok) av[i] = *reinterpret_cast<const uint4*>(ap + 16 * int64_t(kb));
        if constexpr (SCALES == 1) {
          wsc[i] = in && col_ok ? *reinterpret_cast<const uint32_t*>(ws + kb - g) : 0;
          asc[i] = in && row_ok ? *reinterpret_cast<const uint32_t*>(as + kb - g) : 0;
        } else if constexpr (SCALES == 2) {
          wsc[i] = in && col_ok ? ws[kb] : 0;
          asc[i] = in && row_ok ? as[kb] : 0;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int sh = SCALES == 2 ? 0 : 8 * g;
        acc = mfma_fp4(wv[i], av[i], acc, wsc[i] >> sh, asc[i] >> sh);
      }
    }
    sums[wave][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (wave == 0) {
      v4f s = acc;
#pragma unroll
      for (int w = 1; w < kStreamWaves; ++w) {
        const float4 p = sums[w][lane];
        s[0] += p.x; s[1] += p.y; s[2] += p.z; s[3] += p.w;
      }
      if (lo + r16 < hi) store_cols(static_cast<T*>(a.y), a.ld_y, lo + r16, cb * 16 + 4 * g, a.n, wide, s);
    }
    __syncthreads();
  }
}

// four columns of a row can be stored at once
bool wide_stores(const LinearArgs& a, int64_t sz) { return rows_aligned(a.y, a.ld_y * sz, 4 * sz); }

template <typename T>
hipError_t linear_t(const LinearArgs& a, hipStream_t st) {
  const int64_t tiles = a.offsets ? std::min<int64_t>(a.rows, (a.rows + 15) / 16 + a.mats) : (a.rows + 15) / 16;
  const int64_t units = tiles * ((a.n + 15) / 16);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(units, 8 * a.num_cus));
  const bool wide = wide_stores(a, sizeof(T));
  if (a.k % 512 == 0) k_linear_stream<T, 0><<<grid, kStreamThreads, 0, st>>>(a, wide);
  else if (a.k % 128 == 0) k_linear_stream<T, 1><<<grid, kStreamThreads, 0, st>>>(a, wide);
  else k_linear_stream<T, 2><<<grid, kStreamThreads, 0, st>>>(a, wide);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_mx4(const LinearArgs& a, RowType dt, hipStream_t st) {
  switch (dt) {
    case RowType::kBf16: return linear_t<bf16_t>(a, st);
    case RowType::kFp16: return linear_t<_Float16>(a, st);
    default: return linear_t<float>(a, st);
  }
}

}  // namespace mxmoe
