// Tokens sorted by expert and back, with both gradients: moe_sort_tokens,
// moe_dispatch_rows, moe_combine_rows and moe_combine_rows_backward.
//
// A pair p = t*k + j is token t's j-th choice.  The order is the stable
// counting sort of the pairs by expert: row r of the sorted rows belongs to
// pair row_src[r], pair p went to row token_row[p], and a choice outside
// [0, E) has no row (token_row -1).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "internal.h"
#include "row_types.h"

namespace mxmoe {

// ---------------------------------------------------------------------------
// Sorting.  A workgroup of 16 waves ranks a chunk of pairs: wave w takes the
// w-th sixteenth of it, 64 pairs at a time.  Lanes with equal keys find each
// other by one ballot per key bit; the number of equal lanes below is a pair's
// rank among the 64, and the first lane of each key adds their number to the
// wave's own count of that key in LDS.  No atomics: equal keys keep the order
// of their pairs, and a token that names an expert twice has two rows.
// Up to kSortSmall pairs one workgroup does everything in one launch; above
// it, the chunks are counted, the counts summed along the chunks by one
// workgroup (a thread per expert), and the chunks ranked again and written.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kMaxExperts = 1024;

template <typename I>
__device__ __forceinline__ int sort_key(const I* ids, int p, int E) {
  const I v = ids[p];
  return v >= 0 && v < E ? static_cast<int>(v) : -1;
}

// lanes of the wave with this lane's key (valid lanes only)
__device__ __forceinline__ uint64_t equal_lanes(int key, int bits) {
  uint64_t m = __ballot(key >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint64_t s = __ballot(one);
    m &= one ? s : ~s;
  }
  return m;
}

__device__ __forceinline__ int lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0));
}

// Exclusive sum over the threads of a workgroup of kSortThreads; `total` gets
// the sum of all.  part: kSortWaves ints of LDS, free again on return.
__device__ __forceinline__ int block_exclusive(int v, int* part, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(inc, o, 64);
    if (lane >= o) inc += u;
  }
  if (lane == 63) part[wave] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    const int s = part[w];
    before += w < wave ? s : 0;
    all += s;
  }
  __syncthreads();
  total = all;
  return before + inc - v;
}

// One wave's pass over its pairs [lo, hi): f(pair, key, rank among equals in
// this batch, first lane of its key, lanes of its key)
template <typename I, typename F>
__device__ __forceinline__ void each_batch(const I* ids, int lo, int hi, int E, int bits, F f) {
  const int lane = threadIdx.x & 63;
  for (int at = lo; at < hi; at += 64) {
    const int p = at + lane;
    const int key = p < hi ? sort_key(ids, p, E) : -1;
    const uint64_t eq = equal_lanes(key, bits);
    const int rank = lanes_below(eq);
    f(p, key, rank, rank == 0, __popcll(eq));
  }
}

// Whole sort (SMALL) or one chunk's part of it.  base: first row of each
// (expert, chunk), [chunks][E], when not SMALL.
template <typename I, bool SMALL>
__global__ void __launch_bounds__(kSortThreads) k_sort_rank(const I* __restrict__ ids, int P, int E, int bits, int chunk,
                                                            const int* __restrict__ base, int* __restrict__ offsets,
                                                            int* __restrict__ row_src, int* __restrict__ token_row) {
  __shared__ int cnt[kSortWaves * kMaxExperts];
  __shared__ int part[kSortWaves];
  const int tid = threadIdx.x, wave = tid >> 6;
  const int c0 = SMALL ? 0 : blockIdx.x * chunk;
  const int n = min(chunk, P - c0);
  const int per = (((n + kSortWaves - 1) / kSortWaves) + 63) & ~63;
  const int lo = c0 + min(n, wave * per), hi = c0 + min(n, (wave + 1) * per);
  // volatile: a lane reads counts that other lanes of its wave have moved on
  volatile int* mine = cnt + wave * E;
  for (int i = tid; i < kSortWaves * E; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  each_batch(ids, lo, hi, E, bits, [&](int, int key, int, bool first, int same) {
    if (key >= 0 && first) mine[key] = mine[key] + same;
  });
  __syncthreads();
  int rows;   // rows in all
  {
    int sum = 0;
    if (tid < E)
      for (int w = 0; w < kSortWaves; ++w) {
        const int c = cnt[w * E + tid];
        cnt[w * E + tid] = sum;
        sum += c;
      }
    int from;
    if (SMALL) {
      from = block_exclusive(sum, part, rows);
      if (tid < E) offsets[tid] = from;
      if (tid == 0) offsets[E] = rows;
    } else {
      from = tid < E ? base[int64_t(blockIdx.x) * E + tid] : 0;
      rows = offsets[E];
    }
    if (tid < E)
      for (int w = 0; w < kSortWaves; ++w) cnt[w * E + tid] += from;
  }
  __syncthreads();
  each_batch(ids, lo, hi, E, bits, [&](int p, int key, int rank, bool first, int same) {
    const int row = key >= 0 ? mine[key] + rank : -1;
    // every lane has read its key's count before the first one moves it on
    __builtin_amdgcn_wave_barrier();
    if (key >= 0 && first) mine[key] = row + same;
    if (key >= 0) row_src[row] = p;
    if (p < hi) token_row[p] = row;
    __builtin_amdgcn_wave_barrier();
  });
  // entries of this chunk's range behind the last row
  for (int i = max(c0, rows) + tid; i < c0 + n; i += kSortThreads) row_src[i] = -1;
}

// counts[chunk][e] of one chunk (sums of integers: any order gives the same)
template <typename I>
__global__ void __launch_bounds__(kSortThreads) k_sort_count(const I* __restrict__ ids, int P, int E, int chunk,
                                                             int* __restrict__ counts) {
  __shared__ int cnt[kMaxExperts];
  for (int i = threadIdx.x; i < E; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int c0 = blockIdx.x * chunk, c1 = min(P, c0 + chunk);
  for (int p = c0 + threadIdx.x; p < c1; p += kSortThreads) {
    const int key = sort_key(ids, p, E);
    if (key >= 0) atomicAdd(&cnt[key], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += kSortThreads) counts[int64_t(blockIdx.x) * E + i] = cnt[i];
}

// counts -> first row of each (chunk, expert), in place, and the offsets
__global__ void __launch_bounds__(kSortThreads) k_sort_scan(int* __restrict__ counts, int chunks, int E,
                                                            int* __restrict__ offsets) {
  __shared__ int part[kSortWaves];
  const int e = threadIdx.x;
  int sum = 0;
  if (e < E) {
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) sum += counts[int64_t(c) * E + e];
  }
  int rows;
  int at = block_exclusive(sum, part, rows);
  if (e < E) {
    offsets[e] = at;
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) {
      const int n = counts[int64_t(c) * E + e];
      counts[int64_t(c) * E + e] = at;
      at += n;
    }
  }
  if (e == 0) offsets[E] = rows;
}

namespace {

template <typename I>
hipError_t sort_t(const I* ids, int64_t pairs, int E, int* offsets, int* row_src, int* token_row, int* counts,
                  hipStream_t st) {
  const int P = static_cast<int>(pairs);
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  if (pairs <= kSortSmallPairs) {
    k_sort_rank<I, true><<<1, kSortThreads, 0, st>>>(ids, P, E, bits, P, nullptr, offsets, row_src, token_row);
    return hipGetLastError();
  }
  const int chunk = sort_chunk(pairs), chunks = (P + chunk - 1) / chunk;
  k_sort_count<I><<<chunks, kSortThreads, 0, st>>>(ids, P, E, chunk, counts);
  k_sort_scan<<<1, kSortThreads, 0, st>>>(counts, chunks, E, offsets);
  k_sort_rank<I, false><<<chunks, kSortThreads, 0, st>>>(ids, P, E, bits, chunk, counts, offsets, row_src, token_row);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sort_tokens(const void* ids, bool ids64, int64_t pairs, int E, int* offsets, int* row_src,
                              int* token_row, int* counts, hipStream_t st) {
  return ids64 ? sort_t(static_cast<const int64_t*>(ids), pairs, E, offsets, row_src, token_row, counts, st)
               : sort_t(static_cast<const int32_t*>(ids), pairs, E, offsets, row_src, token_row, counts, st);
}

// ---------------------------------------------------------------------------
// Dispatch: every token's row to the rows of its pairs.  A workgroup takes a
// token's row once (or one of `splits` stretches of it) and writes each copy,
// so x is read once from memory.  Element-agnostic: V is the widest word that
// rows and strides are aligned to.  num_rows (may be null): the same
// workgroup zero-fills its share of the rows from *num_rows on.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

template <typename V>
__global__ void __launch_bounds__(kRowThreads) k_dispatch(const char* __restrict__ x, int64_t ld_x, int64_t row_words,
                                                          const int* __restrict__ token_row, int k, int64_t T,
                                                          int64_t R, const int* __restrict__ num_rows,
                                                          char* __restrict__ out, int64_t ld_out, int splits) {
  const int64_t t = blockIdx.x / splits;
  const int s = blockIdx.x - static_cast<int>(t * splits);
  const int64_t per = (row_words + splits - 1) / splits;
  const int64_t c0 = s * per, c1 = min(row_words, c0 + per);
  const int* tr = token_row + t * k;
  const V* src = reinterpret_cast<const V*>(x + t * ld_x);
  for (int64_t c = c0 + threadIdx.x; c < c1; c += kRowThreads) {
    const V v = src[c];
    for (int j = 0; j < k; ++j) {
      const int64_t r = tr[j];
      if (r >= 0 && r < R) reinterpret_cast<V*>(out + r * ld_out)[c] = v;
    }
  }
  if (num_rows) {
    const int64_t n = max(0, *num_rows);
    // rows t, t + T, ... at or past n
    int64_t r = t;
    if (r < n) r += (n - r + T - 1) / T * T;
    for (; r < R; r += T)
      for (int64_t c = c0 + threadIdx.x; c < c1; c += kRowThreads) reinterpret_cast<V*>(out + r * ld_out)[c] = V{};
  }
}

namespace {

// stretches a row is cut into so that few tokens still fill the chip: at
// least one pass of the workgroup each
int row_splits(int64_t T, int64_t passes) {
  int64_t s = std::min<int64_t>(passes, (1024 + T - 1) / T);
  return static_cast<int>(std::max<int64_t>(1, s));
}

template <typename V>
hipError_t dispatch_v(const void* x, int64_t row_bytes, int64_t ld_x, const int* token_row, int64_t T, int k, int64_t R,
                      const int* num_rows, void* out, int64_t ld_out, hipStream_t st) {
  const int64_t words = row_bytes / sizeof(V);
  const int splits = row_splits(T, (words + kRowThreads - 1) / kRowThreads);
  k_dispatch<V><<<static_cast<unsigned>(T * splits), kRowThreads, 0, st>>>(
      static_cast<const char*>(x), ld_x, words, token_row, k, T, R, num_rows, static_cast<char*>(out), ld_out, splits);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch_rows(const void* x, int64_t row_bytes, int64_t ld_x, const int* token_row, int64_t T, int k,
                                int64_t R, const int* num_rows, void* out, int64_t ld_out, hipStream_t st) {
  auto fits = [&](int64_t a) { return row_bytes % a == 0 && rows_aligned(x, ld_x, a) && rows_aligned(out, ld_out, a); };
  auto go = [&](auto v) {
    return dispatch_v<decltype(v)>(x, row_bytes, ld_x, token_row, T, k, R, num_rows, out, ld_out, st);
  };
  if (fits(16)) return go(uint4{});
  if (fits(4)) return go(uint32_t{});
  if (fits(2)) return go(uint16_t{});
  return go(uint8_t{});
}

// ---------------------------------------------------------------------------
// Combine: y[t] = sum over j ascending of w[t,j] rows[token_row[t,j]] in fp32,
// rounded once; dropped pairs are neither read nor added.  A thread holds VEC
// columns (16 bytes) of one token; the loop over the pairs starts kAhead rows'
// loads before it adds the first.
// ---------------------------------------------------------------------------
constexpr int kAhead = 4;

template <typename T, int VEC>
struct Piece {
  float v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ void load_piece(const T* p, float* v) {
  if constexpr (VEC == 1) v[0] = to_f32(*p);
  else if constexpr (VEC == 8) load8<T, true>(p, v);
  else {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_piece(T* p, const float* v) {
  if constexpr (VEC == 1) *p = from_f32<T>(v[0]);
  else if constexpr (VEC == 8) store8<T, true>(p, v);
  else *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kRowThreads) k_combine_rows(const T* __restrict__ rows, int64_t ld, int64_t R,
                                                              const int* __restrict__ token_row,
                                                              const float* __restrict__ w, int k, int64_t pieces,
                                                              T* __restrict__ y, int64_t ld_y, int splits) {
  const int64_t t = blockIdx.x / splits;
  const int s = blockIdx.x - static_cast<int>(t * splits);
  const int64_t per = (pieces + splits - 1) / splits;
  const int64_t c0 = s * per, c1 = min(pieces, c0 + per);
  const int* tr = token_row + t * k;
  const float* wt = w ? w + t * k : nullptr;
  for (int64_t c = c0 + threadIdx.x; c < c1; c += kRowThreads) {
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += kAhead) {
      Piece<T, VEC> v[kAhead];
      bool there[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int64_t r = j0 + a < k ? tr[j0 + a] : -1;
        there[a] = r >= 0 && r < R;
        if (there[a]) load_piece<T, VEC>(rows + r * ld + c * VEC, v[a].v);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (!there[a]) continue;
        const float f = wt ? wt[j0 + a] : 1.0f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = fmaf(f, v[a].v[i], acc[i]);
      }
    }
    store_piece<T, VEC>(y + t * ld_y + c * VEC, acc);
  }
}

// ---------------------------------------------------------------------------
// Gradients of combine: a wave per pair reads its row and the token's dy once,
// drows = w dy (rounded once) and dw = <dy, row> in fp32, lane sums joined by
// a butterfly (a fixed order).  A dropped pair has dw = 0.  num_rows (may be
// null): the wave of pair p also zero-fills the rows p, p + T*k, ... of drows
// from *num_rows on.
// ---------------------------------------------------------------------------
template <typename T, int VEC>
__global__ void __launch_bounds__(kRowThreads) k_combine_bwd(const T* __restrict__ dy, int64_t ld_dy,
                                                             const T* __restrict__ rows, int64_t ld, int64_t R,
                                                             const int* __restrict__ token_row,
                                                             const float* __restrict__ w, int k, int64_t P,
                                                             int64_t pieces, const int* __restrict__ num_rows,
                                                             T* __restrict__ drows, int64_t ld_d, float* __restrict__ dw) {
  const int lane = threadIdx.x & 63;
  const int64_t p = int64_t(blockIdx.x) * (kRowThreads / 64) + (threadIdx.x >> 6);
  if (p >= P) return;
  const int64_t r = token_row[p];
  const bool there = r >= 0 && r < R;
  if (there) {
    const T* d = dy + (p / k) * ld_dy;
    const T* row = rows + r * ld;
    T* out = drows ? drows + r * ld_d : nullptr;
    const float f = w ? w[p] : 1.0f;
    float sum = 0.0f;
#pragma unroll 4
    for (int64_t c = lane; c < pieces; c += 64) {
      float g[VEC];
      load_piece<T, VEC>(d + c * VEC, g);
      if (dw) {
        float v[VEC];
        load_piece<T, VEC>(row + c * VEC, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum = fmaf(g[i], v[i], sum);
      }
      if (out) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[i] *= f;
        store_piece<T, VEC>(out + c * VEC, g);
      }
    }
    if (dw) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
      if (lane == 0) dw[p] = sum;
    }
  } else if (dw && lane == 0) {
    dw[p] = 0.0f;
  }
  if (drows && num_rows) {
    const int64_t n = max(0, *num_rows);
    float zero[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) zero[i] = 0.0f;
    int64_t q = p;
    if (q < n) q += (n - q + P - 1) / P * P;
    for (; q < R; q += P)
      for (int64_t c = lane; c < pieces; c += 64) store_piece<T, VEC>(drows + q * ld_d + c * VEC, zero);
  }
}

namespace {

template <typename T, int VEC>
hipError_t combine_v(const CombineArgs& a, hipStream_t st) {
  const int64_t pieces = a.d / VEC;
  const int splits = row_splits(a.T, (pieces + kRowThreads - 1) / kRowThreads);
  k_combine_rows<T, VEC><<<static_cast<unsigned>(a.T * splits), kRowThreads, 0, st>>>(
      static_cast<const T*>(a.rows), a.ld, a.R, a.token_row, a.w, a.k, pieces, static_cast<T*>(a.y), a.ld_y, splits);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t combine_bwd_v(const CombineArgs& a, hipStream_t st) {
  const int64_t P = a.T * a.k, per = kRowThreads / 64;
  k_combine_bwd<T, VEC><<<static_cast<unsigned>((P + per - 1) / per), kRowThreads, 0, st>>>(
      static_cast<const T*>(a.dy), a.ld_y, static_cast<const T*>(a.rows), a.ld, a.R, a.token_row, a.w, a.k, P, a.d / VEC,
      a.num_rows, static_cast<T*>(a.drows), a.ld_d, a.dw);
  return hipGetLastError();
}

// 16-byte pieces where every row allows them, else single elements
template <typename T>
bool wide_rows(const CombineArgs& a, const void* extra, int64_t ld_extra) {
  auto ok = [&](const void* p, int64_t ld) { return !p || rows_aligned(p, ld * sizeof(T), 16); };
  return a.d % (16 / int64_t(sizeof(T))) == 0 && ok(a.rows, a.ld) && ok(extra, ld_extra) && ok(a.drows, a.ld_d);
}

template <typename T>
hipError_t combine_t(const CombineArgs& a, hipStream_t st) {
  return wide_rows<T>(a, a.y, a.ld_y) ? combine_v<T, 16 / sizeof(T)>(a, st) : combine_v<T, 1>(a, st);
}
template <typename T>
hipError_t combine_bwd_t(const CombineArgs& a, hipStream_t st) {
  return wide_rows<T>(a, a.dy, a.ld_y) ? combine_bwd_v<T, 16 / sizeof(T)>(a, st) : combine_bwd_v<T, 1>(a, st);
}

}  // namespace

hipError_t launch_combine_rows(const CombineArgs& a, RowType dt, hipStream_t st) {
  switch (dt) {
    case RowType::kBf16: return combine_t<bf16_t>(a, st);
    case RowType::kFp16: return combine_t<_Float16>(a, st);
    default: return combine_t<float>(a, st);
  }
}

hipError_t launch_combine_rows_backward(const CombineArgs& a, RowType dt, hipStream_t st) {
  switch (dt) {
    case RowType::kBf16: return combine_bwd_t<bf16_t>(a, st);
    case RowType::kFp16: return combine_bwd_t<_Float16>(a, st);
    default: return combine_bwd_t<float>(a, st);
  }
}

}  // namespace mxmoe
