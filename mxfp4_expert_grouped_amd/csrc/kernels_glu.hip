// Activations kept in 8 bits, and the gated activation between an expert's
// projections: moe_quantize_mx8, moe_dequantize_mx8, moe_swiglu and
// moe_swiglu_backward.
//
// MXFP8 of a block of 32 columns (fewer at a row's end): e = clamp(floor(log2
// amax) - 8, -127, 127), codes = E4M3 round-to-nearest-even of v / 2^e,
// saturated to +-448.  With ef the exponent field of amax as fp32, e + 127 =
// max(ef - 8, 0): floor(log2) is ef - 127 for normal numbers, and everything
// below 2^-119 is at the clamp.  v * 2^-e is exact for every value that does
// not round to zero anyway, so there is one rounding, the conversion's.  A
// block that holds an infinity or a NaN gets the NaN scale (255) and zero
// codes.
//
// a = silu(g) u with silu(g) = g s, s = 1 / (1 + exp(-g)); from the gradient
// da: dg = da u s (1 + g (1 - s)), du = da g s.  fp32 throughout, rounded once.
//
// All are bound by memory: a thread moves 8 columns (of gate and up), and four
// neighbouring lanes share a block and find its largest magnitude with two
// quad permutes.  131072 rows of d_ff 2048, bf16, kept in 8 bits: 365 us forward
// and 365 us backward (calls in a row, 5.9 TB/s each); from a kernel trace, in
// fp16 and 32768 rows kept as they are 68 us and 117 us (5.9 and 5.7 TB/s), and
// 8191 rows of 1365 columns in fp32, whose rows and codes lie on no 16 bytes, 33 us
// and 37 us (4.8 and 4.2 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "mx_device.h"
#include "row_types.h"

namespace mxmoe {

namespace {

constexpr int kGluThreads = 256;

// the larger of the magnitudes (as bits) held by a quad of lanes
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, true)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xF, 0xF, true)));
}

// Eight columns of which n (maybe none) are there; the others are zero.
// VEC: whole pieces are on 16 bytes.
template <typename T, bool VEC, bool NT>
__device__ __forceinline__ void load_part(const T* p, int n, float* v) {
  if (n >= 8) {
    load8<T, VEC, NT>(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32<T>(p[i]) : 0.0f;
}
template <typename T, bool VEC, bool NT>
__device__ __forceinline__ void store_part(T* p, int n, const float* v) {
  if (n >= 8) {
    store8<T, VEC, NT>(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) p[i] = from_f32<T>(v[i]);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// MXFP8 codes of this lane's eight values and the scale byte of its quad's block
__device__ __forceinline__ u32x2 mx8_codes(const float* v, uint32_t& sb) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  const uint32_t ef = quad_max(amax) >> 23;
  const bool finite = ef < 255;
  sb = finite ? (ef > 8 ? ef - 8 : 0) : 255;
  const float mul = __uint_as_float((254 - (finite ? sb : 0)) << 23);
  u32x2 c;
  c[0] = e4m3_cvt4(v[0] * mul, v[1] * mul, v[2] * mul, v[3] * mul);
  c[1] = e4m3_cvt4(v[4] * mul, v[5] * mul, v[6] * mul, v[7] * mul);
  return finite ? c : u32x2{0, 0};
}

// the values that eight codes with scale byte sb stand for
__device__ __forceinline__ void mx8_values(u32x2 c, uint32_t sb, float* v) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  // 2^-127 is below the normal range, 255 is NaN
  const float s = __uint_as_float(sb == 0 ? 0x00400000u : sb == 255 ? 0x7fc00000u : sb << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8(c[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c[h], true);
    v[4 * h] = a.x * s; v[4 * h + 1] = a.y * s; v[4 * h + 2] = b.x * s; v[4 * h + 3] = b.y * s;
  }
}

template <bool VEC, bool NT>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, u32x2 c) {
  if (n >= 8) {
    if constexpr (VEC && NT) __builtin_nontemporal_store(c, reinterpret_cast<u32x2*>(p));
    else if constexpr (VEC) *reinterpret_cast<u32x2*>(p) = c;
    else *reinterpret_cast<u32x2_any*>(p) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) p[i] = static_cast<uint8_t>(c[i / 4] >> (8 * (i % 4)));
}
template <bool VEC, bool NT>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int n) {
  if (n >= 8) {
    if constexpr (VEC && NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    else if constexpr (VEC) return *reinterpret_cast<const u32x2*>(p);
    else return *reinterpret_cast<const u32x2_any*>(p);
  }
  u32x2 c = {0, 0};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) c[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
  return c;
}

// Piece p of a matrix of `pieces` (fewer than 2^31): row p / per_row, columns
// 8 (p % per_row) .., of which some at a row's end are not there.
struct Pieces {
  int pieces, per_row;
};

template <typename T, bool VEC, bool NT>
__global__ void __launch_bounds__(kGluThreads) k_quantize_mx8(const T* __restrict__ src, Pieces s, int cols, int64_t ld,
                                                              uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int p = blockIdx.x * kGluThreads + threadIdx.x;
  // (pieces of a row come in fours: a quad is all in or all out)
  if (p >= s.pieces) return;
  const int row = p / s.per_row, c = 8 * (p - row * s.per_row), n = cols - c;
  float v[8];
  load_part<T, VEC, NT>(src + row * ld + c, n, v);
  uint32_t sb;
  const u32x2 q = mx8_codes(v, sb);
  store_codes<VEC, false>(codes + int64_t(row) * cols + c, n, q);
  if ((p & 3) == 0) scales[p >> 2] = static_cast<uint8_t>(sb);
}

// `pad` columns are written, zeros from cols on
template <typename T, bool VEC>
__global__ void __launch_bounds__(kGluThreads) k_dequantize_mx8(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                                Pieces s, int cols, int pad, T* __restrict__ dst, int64_t ld) {
  const int p = blockIdx.x * kGluThreads + threadIdx.x;
  if (p >= s.pieces) return;
  const int row = p / s.per_row, c = 8 * (p - row * s.per_row);
  if (c >= pad) return;
  float v[8];
  mx8_values(load_codes<VEC, false>(codes + int64_t(row) * cols + c, cols - c), scales[p >> 2], v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? v[i] : 0.0f;  // (a NaN scale stays in its columns)
  store_part<T, VEC, false>(dst + row * ld + c, pad - c, v);
}

// s = 1 / (1 + exp(-g)): for fp32 results with the accurate exponential and
// division, for 16-bit ones with the hardware's exponential and reciprocal: off
// by less than 2^-17 of it, far below half a step of the results, for g >= -87.3
// in fp16 and g >= -88.7 in bf16, and zero for smaller g.  (From -88.7 on exp(-g)
// passes fp32's range.  From -87.3 on s is a subnormal number, which the
// reciprocal does not give.  fp16's g s u and da g s are zero there anyway, but
// bf16's can be any number: its reciprocal is taken of 2^-8 of the argument, and
// the multiplication that scales it back gives subnormal numbers.  It costs the
// activation 0.4 % at 131072 rows of d_ff 2048, and 3 % at 4096 rows, which stay
// in the caches; its gradient less.)
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 4) return 1.0f / (1.0f + expf(-g));
  const float e = __builtin_amdgcn_exp2f(g * -1.44269504088896f);
  if constexpr (std::is_same_v<T, bf16_t>) return __builtin_amdgcn_rcpf(fmaf(e, 0x1p-8f, 0x1p-8f)) * 0x1p-8f;
  else return __builtin_amdgcn_rcpf(1.0f + e);
}

struct GluArgs {
  Pieces s;
  int f;                    // columns of gate and of up
  const void* h; int64_t ld_h;
  void* a; int64_t ld_a;
  uint8_t *codes, *scales;  // [rows][2f], [rows][2 ceil(f/32)]: gate's, then up's
  const void* da; int64_t ld_da;
  void* dh; int64_t ld_dh;
};

template <typename T, bool VEC, bool NT, bool KEEP>
__global__ void __launch_bounds__(kGluThreads) k_swiglu(GluArgs a) {
  const int p = blockIdx.x * kGluThreads + threadIdx.x;
  if (p >= a.s.pieces) return;
  const int row = p / a.s.per_row, q = p - row * a.s.per_row, c = 8 * q, n = a.f - c;
  const T* h = static_cast<const T*>(a.h) + row * a.ld_h + c;
  float g[8], u[8], r[8];
  load_part<T, VEC, NT>(h, n, g);
  load_part<T, VEC, NT>(h + a.f, n, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = g[i] * sigmoid<T>(g[i]) * u[i];
  store_part<T, VEC, false>(static_cast<T*>(a.a) + row * a.ld_a + c, n, r);
  if constexpr (KEEP) {
    uint32_t sg, su;
    const u32x2 cg = mx8_codes(g, sg), cu = mx8_codes(u, su);
    uint8_t* codes = a.codes + int64_t(row) * 2 * a.f + c;
    store_codes<VEC, NT>(codes, n, cg);
    store_codes<VEC, NT>(codes + a.f, n, cu);
    if ((q & 3) == 0) {
      const int nb = a.s.per_row / 4;
      uint8_t* scales = a.scales + int64_t(row) * 2 * nb + q / 4;
      scales[0] = static_cast<uint8_t>(sg);
      scales[nb] = static_cast<uint8_t>(su);
    }
  }
}

// KEPT: gate and up come as codes
template <typename T, bool VEC, bool NT, bool KEPT>
__global__ void __launch_bounds__(kGluThreads) k_swiglu_backward(GluArgs a) {
  const int p = blockIdx.x * kGluThreads + threadIdx.x;
  if (p >= a.s.pieces) return;
  const int row = p / a.s.per_row, q = p - row * a.s.per_row, c = 8 * q, n = a.f - c;
  if (n <= 0) return;
  float g[8], u[8], d[8], r[8];
  if constexpr (KEPT) {
    const uint8_t* codes = a.codes + int64_t(row) * 2 * a.f + c;
    const int nb = a.s.per_row / 4;
    const uint8_t* scales = a.scales + int64_t(row) * 2 * nb + q / 4;
    mx8_values(load_codes<VEC, NT>(codes, n), scales[0], g);
    mx8_values(load_codes<VEC, NT>(codes + a.f, n), scales[nb], u);
  } else {
    const T* h = static_cast<const T*>(a.h) + row * a.ld_h + c;
    load_part<T, VEC, NT>(h, n, g);
    load_part<T, VEC, NT>(h + a.f, n, u);
  }
  load_part<T, VEC, NT>(static_cast<const T*>(a.da) + row * a.ld_da + c, n, d);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = sigmoid<T>(g[i]), gs = g[i] * s;
    r[i] = gs * u[i];
    const float dg = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
    u[i] = d[i] * gs;
    g[i] = dg;
  }
  T* dh = static_cast<T*>(a.dh) + row * a.ld_dh + c;
  store_part<T, VEC, false>(dh, n, g);
  store_part<T, VEC, false>(dh + a.f, n, u);
  if (a.a) store_part<T, VEC, false>(static_cast<T*>(a.a) + row * a.ld_a + c, n, r);
}

// The matrix in slices of whole rows with fewer than 2^31 pieces each.
template <typename F>
hipError_t by_rows(int64_t rows, int64_t per_row, F launch) {
  const int64_t step = std::max<int64_t>(1, ((int64_t(1) << 31) - kGluThreads) / per_row);
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t pieces = std::min(step, rows - r) * per_row;
    launch(r, Pieces{static_cast<int>(pieces), static_cast<int>(per_row)},
           static_cast<unsigned>((pieces + kGluThreads - 1) / kGluThreads));
  }
  return hipGetLastError();
}

template <typename T>
hipError_t quantize_t(const void* src, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const T* s = static_cast<const T*>(src);
  const int64_t nb = (cols + 31) / 32;
  const bool vec = rows_aligned(src, ld * sizeof(T), 16) && rows_aligned(codes, cols, 8);
  const bool nt = vec && rows * cols * int64_t(sizeof(T)) >= kStreamedBytes;
  return by_rows(rows, 4 * nb, [&](int64_t r, Pieces p, unsigned grid) {
    auto* k = nt ? k_quantize_mx8<T, true, true> : vec ? k_quantize_mx8<T, true, false> : k_quantize_mx8<T, false, false>;
    k<<<grid, kGluThreads, 0, st>>>(s + r * ld, p, static_cast<int>(cols), ld, codes + r * cols, scales + r * nb);
  });
}

template <typename T>
hipError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* dst, int64_t ld, int64_t pad,
                        hipStream_t st) {
  T* d = static_cast<T*>(dst);
  const int64_t nb = (cols + 31) / 32;
  const bool vec = rows_aligned(dst, ld * sizeof(T), 16) && rows_aligned(codes, cols, 8);
  return by_rows(rows, 4 * nb, [&](int64_t r, Pieces p, unsigned grid) {
    auto* k = vec ? k_dequantize_mx8<T, true> : k_dequantize_mx8<T, false>;
    k<<<grid, kGluThreads, 0, st>>>(codes + r * cols, scales + r * nb, p, static_cast<int>(cols), static_cast<int>(pad), d + r * ld, ld);
  });
}

template <typename T>
hipError_t swiglu_t(const SwigluArgs& s, hipStream_t st) {
  constexpr int SZ = sizeof(T);
  const bool back = s.dh != nullptr, kept = s.codes != nullptr;
  const int64_t nb = (s.f + 31) / 32, per_row = kept ? 4 * nb : (s.f + 7) / 8;
  auto on16 = [&](const void* p, int64_t ld) { return !p || rows_aligned(p, ld * SZ, 16); };
  const bool vec = s.f * SZ % 16 == 0 && on16(s.h, s.ld_h) && on16(s.a, s.ld_a) && on16(s.da, s.ld_da) && on16(s.dh, s.ld_dh) &&
                   (!kept || rows_aligned(s.codes, s.f, 8));
  const bool nt = vec && s.rows * s.f * SZ >= kStreamedBytes;
  return by_rows(s.rows, per_row, [&](int64_t r, Pieces p, unsigned grid) {
    auto row = [&](const void* q, int64_t ld) { return q ? static_cast<const T*>(q) + r * ld : nullptr; };
    GluArgs a{};
    a.s = p;
    a.f = static_cast<int>(s.f);
    a.h = row(s.h, s.ld_h); a.ld_h = s.ld_h;
    a.a = const_cast<T*>(row(s.a, s.ld_a)); a.ld_a = s.ld_a;
    a.da = row(s.da, s.ld_da); a.ld_da = s.ld_da;
    a.dh = const_cast<T*>(row(s.dh, s.ld_dh)); a.ld_dh = s.ld_dh;
    if (kept) {
      a.codes = s.codes + r * 2 * s.f;
      a.scales = s.scales + r * 2 * nb;
    }
    auto go = [&](auto* k) { k<<<grid, kGluThreads, 0, st>>>(a); };
    if (back) {
      if (kept) go(nt ? k_swiglu_backward<T, true, true, true> : vec ? k_swiglu_backward<T, true, false, true> : k_swiglu_backward<T, false, false, true>);
      else go(nt ? k_swiglu_backward<T, true, true, false> : vec ? k_swiglu_backward<T, true, false, false> : k_swiglu_backward<T, false, false, false>);
    } else {
      if (kept) go(nt ? k_swiglu<T, true, true, true> : vec ? k_swiglu<T, true, false, true> : k_swiglu<T, false, false, true>);
      else go(nt ? k_swiglu<T, true, true, false> : vec ? k_swiglu<T, true, false, false> : k_swiglu<T, false, false, false>);
    }
  });
}

}  // namespace

hipError_t launch_quantize_mx8(const void* src, RowType dt, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales,
                               hipStream_t st) {
  switch (dt) {
    case RowType::kBf16: return quantize_t<bf16_t>(src, rows, cols, ld, codes, scales, st);
    case RowType::kFp16: return quantize_t<_Float16>(src, rows, cols, ld, codes, scales, st);
    default: return quantize_t<float>(src, rows, cols, ld, codes, scales, st);
  }
}

hipError_t launch_dequantize_mx8(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* dst, RowType dt,
                                 int64_t ld, int64_t pad, hipStream_t st) {
  switch (dt) {
    case RowType::kBf16: return dequantize_t<bf16_t>(codes, scales, rows, cols, dst, ld, pad, st);
    case RowType::kFp16: return dequantize_t<_Float16>(codes, scales, rows, cols, dst, ld, pad, st);
    default: return dequantize_t<float>(codes, scales, rows, cols, dst, ld, pad, st);
  }
}

hipError_t launch_swiglu(const SwigluArgs& s, RowType dt, hipStream_t st) {
  switch (dt) {
    case RowType::kBf16: return swiglu_t<bf16_t>(s, st);
    case RowType::kFp16: return swiglu_t<_Float16>(s, st);
    default: return swiglu_t<float>(s, st);
  }
}

}  // namespace mxmoe
