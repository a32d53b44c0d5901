// The element types of rows (bf16, fp16, fp32), eight elements at a time.
// Arithmetic is fp32 throughout; a store rounds once, to nearest even.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxmoe {

typedef __bf16 bf16_t;

// The conversions are the compiler's: V_CVT_PK_BF16_F32 and V_CVT_F16_F32
// round to nearest even and keep NaN, infinities and subnormal numbers.
template <typename T>
__device__ __forceinline__ float to_f32(T v) { return static_cast<float>(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float f) { return static_cast<T>(f); }

// two elements of a 16-bit type as one dword, the first in the low half
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef T v2 __attribute__((ext_vector_type(2)));
  const v2 v = {static_cast<T>(a), static_cast<T>(b)};
  return __builtin_bit_cast(uint32_t, v);
}
template <typename T>
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b);
template <>
__device__ __forceinline__ void unpack2<bf16_t>(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
template <>
__device__ __forceinline__ void unpack2<_Float16>(uint32_t w, float& a, float& b) {
  a = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w)));
  b = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w >> 16)));
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes at p, which is on 16 bytes (ALIGNED) or anywhere (the target reads
// and writes unaligned memory); with the non-temporal hint or without.
template <bool ALIGNED, bool NT, typename V>
__device__ __forceinline__ V load16(const void* p) {
  typedef V U __attribute__((aligned(1)));
  if constexpr (!ALIGNED) return *static_cast<const U*>(p);
  else if constexpr (NT) return __builtin_nontemporal_load(static_cast<const V*>(p));
  else return *static_cast<const V*>(p);
}
template <bool ALIGNED, bool NT, typename V>
__device__ __forceinline__ void store16(void* p, V v) {
  typedef V U __attribute__((aligned(1)));
  if constexpr (!ALIGNED) *static_cast<U*>(p) = v;
  else if constexpr (NT) __builtin_nontemporal_store(v, static_cast<V*>(p));
  else *static_cast<V*>(p) = v;
}

// 16 bytes of elements
template <typename T>
constexpr int kVec = 16 / sizeof(T);
template <typename T, bool ALIGNED, bool NT = false>
__device__ __forceinline__ void load_vec(const T* p, float* v) {
  if constexpr (sizeof(T) == 4) {
    const f32x4 a = load16<ALIGNED, NT, f32x4>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i];
  } else {
    const u32x4 a = load16<ALIGNED, NT, u32x4>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2<T>(a[i], v[2 * i], v[2 * i + 1]);
  }
}
template <typename T, bool ALIGNED, bool NT = false>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) store16<ALIGNED, NT>(p, f32x4{v[0], v[1], v[2], v[3]});
  else
    store16<ALIGNED, NT>(p, u32x4{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])});
}

// eight consecutive elements
template <typename T, bool ALIGNED, bool NT = false>
__device__ __forceinline__ void load8(const T* p, float* v) {
#pragma unroll
  for (int i = 0; i < 8; i += kVec<T>) load_vec<T, ALIGNED, NT>(p + i, v + i);
}
template <typename T, bool ALIGNED, bool NT = false>
__device__ __forceinline__ void store8(T* p, const float* v) {
#pragma unroll
  for (int i = 0; i < 8; i += kVec<T>) store_vec<T, ALIGNED, NT>(p + i, v + i);
}

// Bytes from which on an operand that is read once is read with the
// non-temporal hint: more of it than a part of the 256 MB Infinity Cache would
// not be found there again.
constexpr int64_t kStreamedBytes = int64_t(64) << 20;

// whether every row of a matrix starts on `a` bytes
inline bool rows_aligned(const void* p, int64_t ld_bytes, int64_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0 && ld_bytes % a == 0;
}

}  // namespace mxmoe
