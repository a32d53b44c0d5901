// What stands around the 16-bit products of rows: rows laid out on 16 bytes,
// and fp32 sums of parts joined.  Both are bound by memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "row_types.h"
#include "rows_device.h"

namespace mxmoe {
namespace rows {

namespace {

constexpr int kAuxThreads = 256;
// grid of at most 2^31 threads; the kernels stride over the rest
inline unsigned aux_grid(int64_t n) { return static_cast<unsigned>(std::min<int64_t>((n + kAuxThreads - 1) / kAuxThreads, 1 << 23)); }

struct PadPieces {
  const uint16_t* src;
  uint16_t* dst;
  int64_t first, ld_src;  // first piece of this matrix
  int cols, per_row;
};
struct PadArgs {
  PadPieces m[kMaxPads];
  int64_t pieces;
};

// A thread moves one piece of 16 bytes of dst.
__global__ void __launch_bounds__(kAuxThreads) k_pad_rows(PadArgs a) {
  for (int64_t p = int64_t(blockIdx.x) * kAuxThreads + threadIdx.x; p < a.pieces; p += int64_t(gridDim.x) * kAuxThreads) {
    // (matrices without pieces begin behind all)
    PadPieces m = a.m[0];
#pragma unroll
    for (int i = 1; i < kMaxPads; ++i)
      if (p >= a.m[i].first) m = a.m[i];
    const int64_t q = p - m.first;
    const int64_t row = a.pieces < (int64_t(1) << 31) ? static_cast<uint32_t>(q) / static_cast<uint32_t>(m.per_row) : q / m.per_row;
    const int col = 8 * static_cast<int>(q - row * m.per_row);
    const uint16_t* s = m.src + row * m.ld_src + col;
    u32x4 v;
    if (col + 8 <= m.cols) {
      v = load16<false, false, u32x4>(s);
    } else {
      v = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (col + i < m.cols) v[i / 2] |= static_cast<uint32_t>(s[i]) << (16 * (i % 2));
    }
    reinterpret_cast<u32x4*>(m.dst)[q] = v;
  }
}

// A thread sums four columns over the slices, in their order.
template <typename T>
__global__ void __launch_bounds__(kAuxThreads) k_join(const float* __restrict__ part, int slices, int64_t slice, int64_t quads,
                                                      int per_row, int cols, const int* __restrict__ offsets, int mats, int64_t rows,
                                                      T* __restrict__ out, int64_t ld_out) {
  __shared__ int part_rows[2 * kAuxThreads / 64];
  int lo = 0, hi = 0;
  if (offsets) covered_rows<kAuxThreads>(offsets, mats, static_cast<int>(rows), lo, hi, part_rows);  // (others have no sums)
  for (int64_t p = int64_t(blockIdx.x) * kAuxThreads + threadIdx.x; p < quads; p += int64_t(gridDim.x) * kAuxThreads) {
    const int64_t row = quads < (int64_t(1) << 31) ? static_cast<uint32_t>(p) / static_cast<uint32_t>(per_row) : p / per_row;
    const int col = 4 * static_cast<int>(p - row * per_row);
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (!offsets || (row >= lo && row < hi)) {
      // (slices are a power of two: eight loads on their way at a time, or all)
      auto add = [&](auto n, int i) {
        f32x4 v[decltype(n)::value];
#pragma unroll
        for (int x = 0; x < decltype(n)::value; ++x) v[x] = *reinterpret_cast<const f32x4*>(part + (i + x) * slice + 4 * p);
#pragma unroll
        for (int x = 0; x < decltype(n)::value; ++x) {
          s[0] += v[x][0]; s[1] += v[x][1]; s[2] += v[x][2]; s[3] += v[x][3];
        }
      };
      if (slices == 1) add(std::integral_constant<int, 1>{}, 0);
      else if (slices == 2) add(std::integral_constant<int, 2>{}, 0);
      else if (slices == 4) add(std::integral_constant<int, 4>{}, 0);
      else
        for (int i = 0; i < slices; i += 8) add(std::integral_constant<int, 8>{}, i);
    }
    T* o = out + row * ld_out + col;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < cols) o[i] = from_f32<T>(s[i]);
  }
}

}  // namespace

hipError_t launch_pad_rows(const PadMatrix* m, int count, hipStream_t st) {
  PadArgs a{};
  for (int i = 0; i < kMaxPads; ++i) {
    if (i < count && m[i].rows * (m[i].ld_dst / 8) > 0) {
      a.m[i] = {static_cast<const uint16_t*>(m[i].src), static_cast<uint16_t*>(m[i].dst), a.pieces, m[i].ld_src,
                static_cast<int>(m[i].cols), static_cast<int>(m[i].ld_dst / 8)};
      a.pieces += m[i].rows * (m[i].ld_dst / 8);
    } else {
      a.m[i].first = INT64_MAX;
      a.m[i].per_row = 1;
    }
  }
  if (a.pieces == 0) return hipSuccess;
  k_pad_rows<<<aux_grid(a.pieces), kAuxThreads, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_join(const float* part, int slices, int64_t rows, int64_t cols, int64_t ld, const int* offsets, int mats,
                       void* out, RowType out_t, int64_t ld_out, hipStream_t st) {
  const int64_t quads = rows * (ld / 4);
  auto go = [&](auto* o) {
    k_join<<<aux_grid(quads), kAuxThreads, 0, st>>>(part, slices, rows * ld, quads, static_cast<int>(ld / 4), static_cast<int>(cols),
                                                    offsets, mats, rows, o, ld_out);
    return hipGetLastError();
  };
  switch (out_t) {
    case RowType::kBf16: return go(static_cast<bf16_t*>(out));
    case RowType::kFp16: return go(static_cast<_Float16*>(out));
    default: return go(static_cast<float*>(out));
  }
}

}  // namespace rows
}  // namespace mxmoe
