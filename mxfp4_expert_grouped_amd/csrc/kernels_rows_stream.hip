// y[r] = x[r] W_e(r)^T in 16 bits for few products: straight from memory to
// registers in operand order.  A unit is 16 rows x 16 columns; a persistent
// grid takes them round-robin, the columns of a row tile fastest, so that
// neighbouring workgroups read neighbouring weight rows.  The NW waves of a
// workgroup share a unit's sums: wave w takes the groups of 128 products (256
// bytes of each row) w, w + NW, ..., and the partial sums meet in LDS in wave
// order.  Bound by the bytes of the weights.  With at most one unit per CU NW
// is 8 and a wave has the next group's loads on their way while it multiplies
// this one; with more units NW is 4 and several workgroups per CU hide each
// other's loads.  1 row x 4096 columns, sums of 7168, bf16, calls in a row: 11.1
// us on up to four sets of operands in turn, which the Infinity Cache holds (5.3
// TB/s), and 13.2 us on eight (4.4 TB/s).
//
// The weights are the first operand of the 16x16x32 MFMA: lane (r = lane%16,
// g = lane/16) holds elements 8g .. 8g+7 of row r, and the result of lane l,
// register i is (column 4(l/16)+i, row l%16), four consecutive columns of y.
#include "rows_tile.h"

namespace mxmoe {
namespace rows {

namespace {

template <typename T>
__device__ __forceinline__ v4f mfma16(v8s b, v8s a, v4f c) {
  if constexpr (std::is_same_v<T, bf16_t>) {
    typedef __bf16 v __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v, b), __builtin_bit_cast(v, a), c, 0, 0, 0);
  } else {
    typedef _Float16 v __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v, b), __builtin_bit_cast(v, a), c, 0, 0, 0);
  }
}

// ALIGNED: rows of x and W are whole numbers of 16 bytes, on 16 bytes.
// Otherwise they are read in the same pieces at any address, and the last
// piece of a row by elements.
template <typename T, int NW, bool ALIGNED>
__global__ void __launch_bounds__(64 * NW, NW == 4 ? 4 : 2) k_rows_stream(RowsArgs a, bool wide) {
  __shared__ int prefix[kMaxRowMats];
  __shared__ int part[2 * NW];
  __shared__ v4f sums[NW][64];
  const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x >> 6));
  const int r16 = lane & 15, g = lane >> 4;
  const int tiles = tile_prefix<64 * NW, 16>(a, prefix, part);
  const int cblocks = (a.n + 15) / 16;
  const int64_t units = int64_t(tiles) * cblocks;
  const int groups = (a.l + 127) / 128;
  struct Operand {
    v8s v[4];
  };
  // group q of one row (ok: the row is there)
  auto load = [&](Operand& o, const T* p, bool ok, int q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 128 * q + 32 * i + 8 * g;
      o.v[i] = v8s{};
      if constexpr (ALIGNED) {
        if (ok && at < a.l) o.v[i] = load16<true, false, v8s>(p + at);
      } else if (ok && at + 8 <= a.l) {
        o.v[i] = load16<false, false, v8s>(p + at);
      } else if (ok && at < a.l) {
#pragma unroll
        for (int x = 0; x < 7; ++x)
          if (at + x < a.l) o.v[i][x] = reinterpret_cast<const short*>(p)[at + x];
      }
    }
  };
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    // (a 64-bit division takes a tenth of a short call)
    const int t = static_cast<int>(units < (int64_t(1) << 31) ? static_cast<uint32_t>(u) / static_cast<uint32_t>(cblocks) : u / cblocks);
    const int cb = static_cast<int>(u - int64_t(t) * cblocks);
    const int e = tile_matrix(prefix, a.mats, t);
    int lo, hi;
    mat_rows(a.offsets, e, static_cast<int>(a.rows), lo, hi);
    lo += (t - prefix[e]) * 16;
    const int row = lo + r16, col = cb * 16 + r16;
    const bool row_ok = row < hi, col_ok = col < a.n;
    const T* xp = static_cast<const T*>(a.a) + row * a.ld_a;
    const T* wp = static_cast<const T*>(a.b) + e * a.mat_b + col * a.ld_b;
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto products = [&](const Operand& x, const Operand& w) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = mfma16<T>(w.v[i], x.v[i], acc);
    };
    if constexpr (NW == 8) {
      Operand x[2], w[2];
      int q = wave;
      if (q < groups) {
        load(w[0], wp, col_ok, q);
        load(x[0], xp, row_ok, q);
      }
      while (q < groups) {
        if (q + NW < groups) {
          load(w[1], wp, col_ok, q + NW);
          load(x[1], xp, row_ok, q + NW);
        }
        products(x[0], w[0]);
        x[0] = x[1];
        w[0] = w[1];
        q += NW;
      }
    } else {
      Operand x, w;
      for (int q = wave; q < groups; q += NW) {
        load(w, wp, col_ok, q);
        load(x, xp, row_ok, q);
        products(x, w);
      }
    }
    sums[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
      v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const v4f p = sums[w][lane];
        s[0] += p[0]; s[1] += p[1]; s[2] += p[2]; s[3] += p[3];
      }
      const int c0 = cb * 16 + 4 * g;
      T* y = static_cast<T*>(a.c) + row * a.ld_c + c0;
      if (row_ok) {
        if (wide && c0 + 3 < a.n) {
          *reinterpret_cast<uint2*>(y) = make_uint2(pack2<T>(s[0], s[1]), pack2<T>(s[2], s[3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c0 + i < a.n) y[i] = from_f32<T>(s[i]);
        }
      }
    }
    __syncthreads();
  }
  if (a.offsets) zero_uncovered<64 * NW, T>(a, part);
}

template <typename T>
hipError_t stream_t(const RowsArgs& a, const RowsChoice& c, hipStream_t st) {
  const bool aligned = a.l % 8 == 0 && rows_aligned(a.a, a.ld_a * 2, 16) && rows_aligned(a.b, a.ld_b * 2, 16);
  // four columns of a row can be stored at once
  const bool wide = rows_aligned(a.c, a.ld_c * 2, 8);
  auto go = [&](auto k, int nw) {
    const unsigned grid = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(c.tiles, (nw == 4 ? 8 : 2) * a.num_cus)));
    k<<<grid, 64 * nw, 0, st>>>(a, wide);
    return hipGetLastError();
  };
  if (c.tiles <= a.num_cus) return aligned ? go(k_rows_stream<T, 8, true>, 8) : go(k_rows_stream<T, 8, false>, 8);
  return aligned ? go(k_rows_stream<T, 4, true>, 4) : go(k_rows_stream<T, 4, false>, 4);
}

}  // namespace

hipError_t launch_stream(const RowsArgs& a, const RowsChoice& c, RowType in, hipStream_t st) {
  return in == RowType::kBf16 ? stream_t<bf16_t>(a, c, st) : stream_t<_Float16>(a, c, st);
}

}  // namespace rows
}  // namespace mxmoe
