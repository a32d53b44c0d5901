// MXFP4 (E2M1 elements, one E8M0 scale per 32 along the columns) from and to
// bf16, fp16 and fp32: moe_quantize_mx4 and moe_dequantize_mx4.
//
// Quantising a block of 32 values: e = clamp(floor(log2 amax) - 2, -127, 127),
// codes = E2M1 round-to-nearest-even of v / 2^e, saturated to +-6.  With ef
// the exponent field of amax as fp32, e + 127 = max(ef - 2, 0): floor(log2)
// is ef - 127 for normal numbers, and everything below 2^-125 (subnormals and
// zero among them) is at the clamp.  v * 2^-e is exact for every value that
// does not round to zero anyway (2^-e is a normal number: its exponent field
// is 254 - (e + 127), 2 .. 254), so there is one rounding, the conversion's.
// A block that holds an infinity or a NaN has ef = 255: its scale is the NaN
// of E8M0 (255) and its codes are zero.
//
// Both are bound by memory: a thread moves 8 elements (16 bytes of a 16-bit
// type, 4 bytes of codes), and four neighbouring lanes share a block and find
// its largest magnitude with two quad permutes.  Large sources are read with
// the non-temporal hint.  16384 x 7168 fp32: 97 us with the hint and one piece
// per thread (5.5 TB/s), 128 us without it and with four; back 100 us.  8191 x
// 7168 bf16: 28 us (32 without), back 23 us (6.4 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "internal.h"
#include "row_types.h"

namespace mxmoe {

constexpr int kMx4Threads = 256;

// the larger of the magnitudes (as bits) held by a quad of lanes
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, true)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xF, 0xF, true)));
}

// E2M1 codes of eight values already divided by the block scale.
// V_CVT_SCALEF32_PK_FP4_F32 rounds to nearest even and keeps the sign of
// zero; its input is clamped to the largest magnitude.
__device__ __forceinline__ uint32_t e2m1_cvt8(const float* q) {
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __builtin_amdgcn_fmed3f(q[i], -6.0f, 6.0f);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[0], c[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[2], c[3], 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[4], c[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[6], c[7], 1.0f, 3);
}

// Piece p of the matrix: row p / (cols/8), columns 8 (p % (cols/8)) ..; the
// caller keeps the number of pieces below 2^31.  ALIGNED: rows start on 16
// bytes, so a piece is one or two 16-byte loads.
template <typename T, bool ALIGNED, bool NT>
__global__ void __launch_bounds__(kMx4Threads) k_quantize_mx4(const T* __restrict__ src, int pieces, int per_row,
                                                              int64_t ld, uint8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  const int p = blockIdx.x * kMx4Threads + threadIdx.x;
  // pieces come in fours (cols is a multiple of 32): a quad is all in or all out
  if (p >= pieces) return;
  const int row = p / per_row;
  float v[8];
  load8<T, ALIGNED, NT>(src + row * ld + 8 * int64_t(p - row * per_row), v);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  const uint32_t ef = quad_max(amax) >> 23;
  const bool finite = ef < 255;
  const uint32_t sb = finite ? (ef > 2 ? ef - 2 : 0) : 255;
  const float mul = __uint_as_float((254 - (finite ? sb : 0)) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= mul;
  reinterpret_cast<uint32_t*>(codes)[p] = finite ? e2m1_cvt8(v) : 0;
  if ((p & 3) == 0) scales[p >> 2] = static_cast<uint8_t>(sb);
}

// 2^(sb - 127) for every scale byte: 2^-127 is below the normal range, 255 is NaN
__device__ __forceinline__ float e8m0_value(uint32_t sb) {
  return __uint_as_float(sb == 0 ? 0x00400000u : sb == 255 ? 0x7fc00000u : sb << 23);
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kMx4Threads) k_dequantize_mx4(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int pieces,
                                                                int per_row, T* __restrict__ dst, int64_t ld) {
  const int p = blockIdx.x * kMx4Threads + threadIdx.x;
  if (p >= pieces) return;
  const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[p];
  const float s = e8m0_value(scales[p >> 2]);
  typedef float v2f __attribute__((ext_vector_type(2)));
  const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  const float v[8] = {a.x * s, a.y * s, b.x * s, b.y * s, c.x * s, c.y * s, d.x * s, d.y * s};
  const int row = p / per_row;
  store8<T, ALIGNED>(dst + row * ld + 8 * int64_t(p - row * per_row), v);
}

namespace {

// The matrix in slices of whole rows with fewer than 2^31 pieces each.
template <typename F>
hipError_t by_rows(int64_t rows, int64_t cols, F launch) {
  const int64_t per_row = cols / 8;
  const int64_t step = std::max<int64_t>(1, ((int64_t(1) << 31) - kMx4Threads) / per_row);
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t pieces = std::min(step, rows - r) * per_row;
    launch(r, static_cast<int>(pieces), static_cast<int>(per_row),
           static_cast<unsigned>((pieces + kMx4Threads - 1) / kMx4Threads));
  }
  return hipGetLastError();
}

template <typename T>
hipError_t quantize_t(const void* src, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales,
                      hipStream_t st) {
  const T* s = static_cast<const T*>(src);
  const bool al = rows_aligned(src, ld * sizeof(T), 16);
  return by_rows(rows, cols, [&](int64_t r, int pieces, int per_row, unsigned grid) {
    auto* k = !al ? k_quantize_mx4<T, false, false>
              : rows * cols * int64_t(sizeof(T)) >= kStreamedBytes ? k_quantize_mx4<T, true, true> : k_quantize_mx4<T, true, false>;
    k<<<grid, kMx4Threads, 0, st>>>(s + r * ld, pieces, per_row, ld, codes + r * (cols / 2), scales + r * (cols / 32));
  });
}

template <typename T>
hipError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* dst, int64_t ld,
                        hipStream_t st) {
  T* d = static_cast<T*>(dst);
  const bool al = rows_aligned(dst, ld * sizeof(T), 16);
  return by_rows(rows, cols, [&](int64_t r, int pieces, int per_row, unsigned grid) {
    auto* k = al ? k_dequantize_mx4<T, true> : k_dequantize_mx4<T, false>;
    k<<<grid, kMx4Threads, 0, st>>>(codes + r * (cols / 2), scales + r * (cols / 32), pieces, per_row, d + r * ld, ld);
  });
}

}  // namespace

hipError_t launch_quantize_mx4(const void* src, RowType dt, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                               uint8_t* scales, hipStream_t st) {
  switch (dt) {
    case RowType::kBf16: return quantize_t<bf16_t>(src, rows, cols, ld, codes, scales, st);
    case RowType::kFp16: return quantize_t<_Float16>(src, rows, cols, ld, codes, scales, st);
    default: return quantize_t<float>(src, rows, cols, ld, codes, scales, st);
  }
}

hipError_t launch_dequantize_mx4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* dst,
                                 RowType dt, int64_t ld, hipStream_t st) {
  switch (dt) {
    case RowType::kBf16: return dequantize_t<bf16_t>(codes, scales, rows, cols, dst, ld, st);
    case RowType::kFp16: return dequantize_t<_Float16>(codes, scales, rows, cols, dst, ld, st);
    default: return dequantize_t<float>(codes, scales, rows, cols, dst, ld, st);
  }
}

}  // namespace mxmoe
