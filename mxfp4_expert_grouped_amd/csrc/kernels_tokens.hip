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
// Sorting.  A workgroup of 16 waves ranks at most 4096 pairs: a wave takes a
// contiguous stretch of them, 64 pairs at a time, at most four times, and
// keeps their keys in registers.  Lanes with equal keys find each other by one
// ballot per key bit; the number of equal lanes below is a pair's rank among
// the 64, and the first lane of each key adds their number to the wave's own
// count of that key in LDS.  No atomics: equal keys keep the order of their
// pairs, and a token that names an expert twice has two rows.
//
// Bound by the latency of its few steps, so their number is kept low: up to
// kSortSmallPairs everything is one launch of one workgroup (256 tokens, top
// 16 of 896: 11.9 us when every pass loaded the ids again and the waves'
// counts were summed one after the other, 9.8 us now; one token 4.3 us).  Above it a first launch
// counts the keys of every chunk, and each ranking workgroup sums those of the
// chunks before its own and of all (131072 pairs, 64 chunks: two launches of
// together 16 us; with a workgroup of its own that summed, 24 us).  Above
// kSortFusedChunks chunks that reading would grow with their square, and a
// launch between the two sums them.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortBatches = kSortSmallPairs / kSortThreads;  // of 64 pairs, per wave
constexpr int kMaxExperts = 1024;

template <typename I>
__device__ __forceinline__ int sort_key(const I* ids, int p, int E) {
  const I v = ids[p];
  return v >= 0 && v < E ? static_cast<int>(v) : -1;
}

// Lanes of the wave with this lane's key (valid lanes only): per key bit those
// with the same bit, m & ~(ballot ^ the bit in all places).
__device__ __forceinline__ uint64_t equal_lanes(int key, int bits) {
  const uint64_t valid = __ballot(key >= 0);
  uint32_t lo = static_cast<uint32_t>(valid), hi = static_cast<uint32_t>(valid >> 32);
  for (int b = 0; b < bits; ++b) {
    const uint32_t bit = static_cast<uint32_t>(__builtin_amdgcn_sbfe(key, b, 1));
    const uint64_t s = __ballot(bit != 0);
    lo &= ~(static_cast<uint32_t>(s) ^ bit);
    hi &= ~(static_cast<uint32_t>(s >> 32) ^ bit);
  }
  return static_cast<uint64_t>(hi) << 32 | lo;
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

// How the pairs outside a workgroup's chunk come in.  kAlone: there are none.
// kCounts: `table` has every chunk's count of every expert, [chunks][E].
// kBases: `table` has the first row of every (chunk, expert).
enum SortTable { kAlone, kCounts, kBases };

template <typename I, SortTable TABLE>
__global__ void __launch_bounds__(kSortThreads) k_sort_rank(const I* __restrict__ ids, int P, int E, int bits, int chunk,
                                                            const int* __restrict__ table, int* __restrict__ offsets,
                                                            int* __restrict__ row_src, int* __restrict__ token_row) {
  __shared__ int cnt[kSortWaves * kMaxExperts];
  __shared__ int part[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c0 = TABLE == kAlone ? 0 : blockIdx.x * chunk;
  const int n = min(chunk, P - c0);
  // batches per wave, and waves that have any
  const int per = (n + kSortThreads - 1) / kSortThreads;
  const int waves = per ? (n + 64 * per - 1) / (64 * per) : 0;
  int key[kSortBatches];
#pragma unroll
  for (int b = 0; b < kSortBatches; ++b) {
    const int i = (wave * per + b) * 64 + lane;
    key[b] = b < per && i < n ? sort_key(ids, c0 + i, E) : -1;
  }
  int before = 0, total = 0;   // of this thread's expert: rows in earlier chunks, in all (kCounts)
  if (TABLE == kCounts && tid < E) {
    // 32 loads on their way at a time
    const int chunks = gridDim.x;
    for (int c = 0; c < chunks; c += 32) {
      int v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = c + i < chunks ? table[(c + i) * E + tid] : 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        total += v[i];
        before += c + i < static_cast<int>(blockIdx.x) ? v[i] : 0;
      }
    }
  }
  // volatile: a lane reads counts that other lanes of its wave have moved on
  volatile int* mine = cnt + wave * E;
  for (int i = tid; i < waves * E; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  uint64_t equal[kSortBatches];
#pragma unroll
  for (int b = 0; b < kSortBatches; ++b) {
    if (b >= per || wave >= waves) break;
    equal[b] = equal_lanes(key[b], bits);
    if (key[b] >= 0 && lanes_below(equal[b]) == 0) mine[key[b]] = mine[key[b]] + __popcll(equal[b]);
  }
  __syncthreads();
  int rows;   // rows in all
  {
    int c[kSortWaves], sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c[w] = tid < E && w < waves ? cnt[w * E + tid] : 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) sum += c[w];
    int from;
    if (TABLE == kBases) {
      from = tid < E ? table[int64_t(blockIdx.x) * E + tid] : 0;
      rows = offsets[E];
    } else {
      from = block_exclusive(TABLE == kAlone ? sum : total, part, rows);
      if (blockIdx.x == 0) {
        if (tid < E) offsets[tid] = from;
        if (tid == 0) offsets[E] = rows;
      }
      from += before;
    }
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      if (tid < E && w < waves) cnt[w * E + tid] = from;
      from += c[w];
    }
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < kSortBatches; ++b) {
    if (b >= per || wave >= waves) break;
    const int i = (wave * per + b) * 64 + lane;
    const int rank = key[b] >= 0 ? lanes_below(equal[b]) : 0;
    const int row = key[b] >= 0 ? mine[key[b]] + rank : -1;
    // every lane has read its key's count before the first one moves it on
    __builtin_amdgcn_wave_barrier();
    if (key[b] >= 0 && rank == 0) mine[key[b]] = row + __popcll(equal[b]);
    if (key[b] >= 0) row_src[row] = c0 + i;
    if (i < n) token_row[c0 + i] = row;
    __builtin_amdgcn_wave_barrier();
  }
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
#pragma unroll 16
    for (int c = 0; c < chunks; ++c) sum += counts[int64_t(c) * E + e];
  }
  int rows;
  int at = block_exclusive(sum, part, rows);
  if (e < E) {
    offsets[e] = at;
    for (int c = 0; c < chunks; c += 16) {
      int n[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) n[i] = c + i < chunks ? counts[int64_t(c + i) * E + e] : 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (c + i < chunks) counts[int64_t(c + i) * E + e] = at;
        at += n[i];
      }
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
    k_sort_rank<I, kAlone><<<1, kSortThreads, 0, st>>>(ids, P, E, bits, P, nullptr, offsets, row_src, token_row);
    return hipGetLastError();
  }
  const int chunk = sort_chunk(pairs), chunks = (P + chunk - 1) / chunk;
  k_sort_count<I><<<chunks, kSortThreads, 0, st>>>(ids, P, E, chunk, counts);
  if (chunks > kSortFusedChunks) {
    k_sort_scan<<<1, kSortThreads, 0, st>>>(counts, chunks, E, offsets);
    k_sort_rank<I, kBases><<<chunks, kSortThreads, 0, st>>>(ids, P, E, bits, chunk, counts, offsets, row_src, token_row);
  } else {
    k_sort_rank<I, kCounts><<<chunks, kSortThreads, 0, st>>>(ids, P, E, bits, chunk, counts, offsets, row_src, token_row);
  }
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
// so x is read once from memory (8192 tokens, top 16, 7168 bf16: 380 us, 5.3
// TB/s, of which 16/17 are the copies; no hint on them gained).  Bytes whatever
// the elements: 16 at a time, ALIGNED if rows start on 16 bytes, and the last
// few one by one.  num_rows (may be null): the same workgroup zero-fills its
// share of the rows from *num_rows on.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

template <bool ALIGNED>
__global__ void __launch_bounds__(kRowThreads) k_dispatch(const char* __restrict__ x, int64_t ld_x, int64_t row_bytes,
                                                          const int* __restrict__ token_row, int k, int64_t T,
                                                          int64_t R, const int* __restrict__ num_rows,
                                                          char* __restrict__ out, int64_t ld_out, int splits) {
  const int64_t t = blockIdx.x / splits;
  const int s = blockIdx.x - static_cast<int>(t * splits);
  const int64_t words = row_bytes / 16, per = (words + splits - 1) / splits;
  const int64_t c0 = s * per, c1 = min(words, c0 + per);
  // the last stretch's first threads take the bytes behind the last word
  const int64_t tail = 16 * words + threadIdx.x;
  const bool has_tail = s == splits - 1 && tail < row_bytes;
  const int* tr = token_row + t * k;
  const char* src = x + t * ld_x;
  for (int64_t c = c0 + threadIdx.x; c < c1; c += kRowThreads) {
    const u32x4 v = load16<ALIGNED, false, u32x4>(src + 16 * c);
    for (int j = 0; j < k; ++j) {
      const int64_t r = tr[j];
      if (r >= 0 && r < R) store16<ALIGNED, false>(out + r * ld_out + 16 * c, v);
    }
  }
  if (has_tail)
    for (int j = 0; j < k; ++j) {
      const int64_t r = tr[j];
      if (r >= 0 && r < R) out[r * ld_out + tail] = src[tail];
    }
  if (num_rows) {
    const int64_t n = max(0, *num_rows);
    // rows t, t + T, ... at or past n
    int64_t r = t;
    if (r < n) r += (n - r + T - 1) / T * T;
    for (; r < R; r += T) {
      for (int64_t c = c0 + threadIdx.x; c < c1; c += kRowThreads)
        store16<ALIGNED, false>(out + r * ld_out + 16 * c, u32x4{0, 0, 0, 0});
      if (has_tail) out[r * ld_out + tail] = 0;
    }
  }
}

namespace {

// stretches a row is cut into so that few tokens still fill the chip: at
// least one pass of the workgroup each
int row_splits(int64_t T, int64_t passes) {
  int64_t s = std::min<int64_t>(passes, (1024 + T - 1) / T);
  return static_cast<int>(std::max<int64_t>(1, s));
}

}  // namespace

hipError_t launch_dispatch_rows(const void* x, int64_t row_bytes, int64_t ld_x, const int* token_row, int64_t T, int k,
                                int64_t R, const int* num_rows, void* out, int64_t ld_out, hipStream_t st) {
  const int splits = row_splits(T, (row_bytes / 16 + kRowThreads - 1) / kRowThreads);
  auto* go = rows_aligned(x, ld_x, 16) && rows_aligned(out, ld_out, 16) ? k_dispatch<true> : k_dispatch<false>;
  go<<<static_cast<unsigned>(T * splits), kRowThreads, 0, st>>>(static_cast<const char*>(x), ld_x, row_bytes, token_row, k,
                                                                T, R, num_rows, static_cast<char*>(out), ld_out, splits);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Combine: y[t] = sum over j ascending of w[t,j] rows[token_row[t,j]] in fp32,
// rounded once; dropped pairs are neither read nor added.  A thread holds 16
// bytes of columns of one token; the loop over the pairs starts kAhead rows'
// loads before it adds the first.  Bound by reading the rows once: 131072 x
// 7168 bf16 373 us (5.4 TB/s; 400 with kAhead = 8, 547 with 16), 65520 x 7168
// fp32 362 us; NT, the non-temporal hint for rows and result, is for more rows
// than a cache keeps (454 and 421 us without it).
// ---------------------------------------------------------------------------
constexpr int kAhead = 4;

// The kVec elements of a row from column at on; of a row's last piece only
// those before column d are there (FULL: d is a whole number of pieces and
// rows are on 16 bytes).
template <typename T, bool FULL, bool NT = false>
__device__ __forceinline__ void load_piece(const T* row, int64_t at, int64_t d, float* v) {
  if (FULL || at + kVec<T> <= d) return load_vec<T, FULL, NT>(row + at, v);
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) v[i] = at + i < d ? to_f32(row[at + i]) : 0.0f;
}
template <typename T, bool FULL, bool NT = false>
__device__ __forceinline__ void store_piece(T* row, int64_t at, int64_t d, const float* v) {
  if (FULL || at + kVec<T> <= d) return store_vec<T, FULL, NT>(row + at, v);
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i)
    if (at + i < d) row[at + i] = from_f32<T>(v[i]);
}

template <typename T, bool FULL, bool NT>
__global__ void __launch_bounds__(kRowThreads) k_combine_rows(const T* __restrict__ rows, int64_t ld, int64_t R,
                                                              const int* __restrict__ token_row,
                                                              const float* __restrict__ w, int k, int64_t d,
                                                              T* __restrict__ y, int64_t ld_y, int splits) {
  constexpr int VEC = kVec<T>;
  const int64_t t = blockIdx.x / splits;
  const int s = blockIdx.x - static_cast<int>(t * splits);
  const int64_t pieces = (d + VEC - 1) / VEC, per = (pieces + splits - 1) / splits;
  const int64_t c0 = s * per, c1 = min(pieces, c0 + per);
  const int* tr = token_row + t * k;
  const float* wt = w ? w + t * k : nullptr;
  for (int64_t c = c0 + threadIdx.x; c < c1; c += kRowThreads) {
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += kAhead) {
      // row numbers and weights first, then the rows: one wait for each
      int r[kAhead];
      float f[kAhead], v[kAhead][VEC];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const bool in = j0 + a < k;
        r[a] = in ? tr[j0 + a] : -1;
        f[a] = wt && in ? wt[j0 + a] : 1.0f;
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (r[a] >= 0 && r[a] < R) load_piece<T, FULL, NT>(rows + r[a] * ld, c * VEC, d, v[a]);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (r[a] < 0 || r[a] >= R) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = fmaf(f[a], v[a][i], acc[i]);
      }
    }
    store_piece<T, FULL, NT>(y + t * ld_y, c * VEC, d, acc);
  }
}

// ---------------------------------------------------------------------------
// Gradients of combine: a wave per pair reads its row and the token's dy once,
// drows = w dy (rounded once) and dw = <dy, row> in fp32: a lane has a sum for
// each element of its 16-byte piece, joined in pairs, and the lanes' are joined
// by a butterfly (a fixed order; of 7168 fp32 columns a product passes through
// 36 roundings, with one sum per lane it was 118).  Bound by memory: 65520 x 7168 fp32 754 us (5.1
// TB/s; 925 with the non-temporal hint, as a token's waves share its dy).  A
// dropped pair has dw = 0.  num_rows (may be
// null): the wave of pair p also zero-fills the rows p, p + T*k, ... of drows
// from *num_rows on.
// ---------------------------------------------------------------------------
template <typename T, bool FULL>
__global__ void __launch_bounds__(kRowThreads) k_combine_bwd(const T* __restrict__ dy, int64_t ld_dy,
                                                             const T* __restrict__ rows, int64_t ld, int64_t R,
                                                             const int* __restrict__ token_row,
                                                             const float* __restrict__ w, int k, int64_t P,
                                                             int64_t d, const int* __restrict__ num_rows,
                                                             T* __restrict__ drows, int64_t ld_d, float* __restrict__ dw) {
  constexpr int VEC = kVec<T>;
  const int lane = threadIdx.x & 63;
  const int64_t p = int64_t(blockIdx.x) * (kRowThreads / 64) + (threadIdx.x >> 6);
  if (p >= P) return;
  const int64_t pieces = (d + VEC - 1) / VEC;
  const int64_t r = token_row[p];
  if (r >= 0 && r < R) {
    const T* g_row = dy + (p / k) * ld_dy;
    const T* row = rows + r * ld;
    T* out = drows ? drows + r * ld_d : nullptr;
    const float f = w ? w[p] : 1.0f;
    float sum[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
#pragma unroll 4
    for (int64_t c = lane; c < pieces; c += 64) {
      float g[VEC];
      load_piece<T, FULL>(g_row, c * VEC, d, g);
      if (dw) {
        float v[VEC];
        load_piece<T, FULL>(row, c * VEC, d, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] = fmaf(g[i], v[i], sum[i]);
      }
      if (out) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[i] *= f;
        store_piece<T, FULL>(out, c * VEC, d, g);
      }
    }
    if (dw) {
#pragma unroll
      for (int h = VEC / 2; h > 0; h >>= 1)
#pragma unroll
        for (int i = 0; i < h; ++i) sum[i] += sum[i + h];
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum[0] += __shfl_xor(sum[0], o, 64);
      if (lane == 0) dw[p] = sum[0];
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
      for (int64_t c = lane; c < pieces; c += 64) store_piece<T, FULL>(drows + q * ld_d, c * VEC, d, zero);
  }
}

namespace {

// whole 16-byte pieces at 16-byte addresses in every row
template <typename T>
bool full_rows(const CombineArgs& a, const void* extra, int64_t ld_extra) {
  auto ok = [&](const void* p, int64_t ld) { return !p || rows_aligned(p, ld * sizeof(T), 16); };
  return a.d % kVec<T> == 0 && ok(a.rows, a.ld) && ok(extra, ld_extra) && ok(a.drows, a.ld_d);
}

template <typename T>
hipError_t combine_t(const CombineArgs& a, hipStream_t st) {
  const int64_t pieces = (a.d + kVec<T> - 1) / kVec<T>;
  const int splits = row_splits(a.T, (pieces + kRowThreads - 1) / kRowThreads);
  auto* go = !full_rows<T>(a, a.y, a.ld_y) ? k_combine_rows<T, false, false>
             : a.T * a.k * a.d * int64_t(sizeof(T)) >= kStreamedBytes ? k_combine_rows<T, true, true>
                                                                      : k_combine_rows<T, true, false>;
  go<<<static_cast<unsigned>(a.T * splits), kRowThreads, 0, st>>>(static_cast<const T*>(a.rows), a.ld, a.R, a.token_row, a.w,
                                                                  a.k, a.d, static_cast<T*>(a.y), a.ld_y, splits);
  return hipGetLastError();
}

template <typename T>
hipError_t combine_bwd_t(const CombineArgs& a, hipStream_t st) {
  const int64_t P = a.T * a.k, per = kRowThreads / 64;
  auto* go = full_rows<T>(a, a.dy, a.ld_y) ? k_combine_bwd<T, true> : k_combine_bwd<T, false>;
  go<<<static_cast<unsigned>((P + per - 1) / per), kRowThreads, 0, st>>>(
      static_cast<const T*>(a.dy), a.ld_y, static_cast<const T*>(a.rows), a.ld, a.R, a.token_row, a.w, a.k, P, a.d,
      a.num_rows, static_cast<T*>(a.drows), a.ld_d, a.dw);
  return hipGetLastError();
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
