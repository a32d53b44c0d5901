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
#include <type_traits>

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

// ---------------------------------------------------------------------------
// Many rows per matrix: BM x 256 tiles through LDS.  One workgroup of four
// waves per CU walks its tiles; a step is 128 of K.  The step's codes (64
// bytes of each of BM activation and 256 weight rows) come by direct-to-LDS
// copies into a ring of S slots, and the stream of steps runs on across the
// tiles: while a tile ends, the first steps of the next are already on their
// way.  Per step a wave issues
//   16 MI NI / 16 MFMAs 32x32x64 of K half 0, between them the LDS reads of
//   half 1; then, with its own copies of step s + 1 landed and a barrier (all
//   waves' copies have landed, and all have read slot s), those of half 1,
//   between them the reads of half 0 of step s + 1 and the copies of step
//   s + S into slot s.
// The weights are the first MFMA operand: lane (l32, g32) register r of a
// 32x32 result is column 8(r/4) + 4 g32 + r%4 of activation row l32, so four
// registers are four consecutive columns of y.
//
// LDS slot: activation rows, then weight rows, 64 bytes each; the 16-byte
// chunk c of row r sits at chunk c ^ ((r/4) % 4), so that the eight lanes that
// the LDS serves together (eight rows, one chunk) touch all banks once.  A copy
// moves 16 rows: lane l brings chunk (l%4) ^ (l/16) of row l/4, four lanes the
// 64 bytes of a row.
//
// Scales.  AG (k % 512 == 0, scale rows on 16 bytes): one 16-byte piece per
// row holds four steps' scales, copied every fourth step into one of two
// buffers and kept in registers for those steps.  Otherwise a dword per row
// and step, in the slot.  Byte 2h + g32 of a step's dword belongs to K half h
// of lane (l32, g32): shifted by 8 g32 once per step, the MFMA takes byte 2h.
//
// Rows past the tile's or the matrix's end are copied from the last valid row
// and their results not stored.
// ---------------------------------------------------------------------------
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

// Copies of 16 (4) bytes per lane from base + off to LDS byte address
// lds + 16 lane (4 lane).  Written as assembly (with no register output) so
// that the compiler does not wait for them at every later LDS read; the kernel
// counts its own copies.  M0 holds the LDS address.
__device__ __forceinline__ void copy16(uint32_t off, const uint8_t* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}
__device__ __forceinline__ void copy4(uint32_t off, const uint8_t* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}
// two consecutive ints of wave-uniform metadata, waited for in the statement
// (a vector load would make the compiler wait for every copy in flight)
__device__ __forceinline__ void sload2(const int* p, int& a, int& b) {
  typedef int v2i __attribute__((ext_vector_type(2)));
  v2i v;
  asm volatile("s_load_dwordx2 %0, %1, 0x0\n\ts_waitcnt lgkmcnt(0)" : "=s"(v) : "s"(p) : "memory");
  a = v.x;
  b = v.y;
}
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32));
  return reinterpret_cast<const uint8_t*>(uint64_t(hi) << 32 | lo);
}

template <int N>
__device__ __forceinline__ void wait_vm() {  // at most N vector-memory operations left
  static_assert(N < 64, "vmcnt has six bits");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (0xF << 8) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }

__device__ __forceinline__ void tile_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <int N>
using Int = std::integral_constant<int, N>;
template <int B, int E, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (B < E) {
    f(Int<B>{});
    unrolled<B + 1, E>(f);
  }
}

template <int H>
__device__ __forceinline__ v16f mfma32_fp4(uint4 w, uint4 a, v16f c, uint32_t sw, uint32_t sa) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(w), fp4_operand(a), c, 4, 4, 2 * H,
                                                         static_cast<int>(sw), 2 * H, static_cast<int>(sa));
}

constexpr int kTileN = 256, kTileThreads = 256;
constexpr int kMaxTiles = 1 << 30;
constexpr int kPanel = 4;  // row tiles that share a column block's weights in time

template <int BM, bool AG>
struct TileShape {
  static constexpr int WM = BM == 64 ? 1 : 2, WN = 4 / WM;        // waves along rows, columns
  static constexpr int MI = BM / WM / 32, NI = kTileN / WN / 32;  // 32-row, 32-column blocks of a wave
  static constexpr int S = BM == 256 ? 4 : BM == 128 ? 5 : 7;     // ring slots
  static constexpr int A = 0, W = BM * 64, SC = W + kTileN * 64;  // slot: activations, weights, scale dwords
  static constexpr int SLOT = SC + (AG ? 0 : (BM + kTileN) * 4);
  static constexpr int GROUP = S * SLOT;                          // scale pieces of AG, two buffers
  static constexpr int LDS = GROUP + (AG ? 2 * (BM + kTileN) * 16 : 0);
  static constexpr int CA = BM / 64, CW = 4;                      // copies of codes per wave and step
  // copies of a wave for a step that is the I-th of its group
  static constexpr int copies(int i) { return CA + CW + (AG ? (i % 4 == 0 ? 2 : 0) : 2); }
};

// WIDE: n and the rows of y are whole numbers of 16-byte pieces.
template <typename T, int BM, bool AG, bool WIDE>
__global__ void __launch_bounds__(kTileThreads, 1) k_linear_tile(LinearArgs a) {
  using P = TileShape<BM, AG>;
  constexpr int S = P::S, MI = P::MI, NI = P::NI, NM = MI * NI;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[P::LDS];
  __shared__ int prefix[kMaxMats + 1];
  __shared__ int part[kTileThreads / 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int l32 = lane & 31, g32 = lane >> 5;
  const int wm = wave / P::WN, wn = wave % P::WN;
  const int mtiles = __builtin_amdgcn_readfirstlane(tile_prefix<kTileThreads, BM>(a, prefix, part));
  const int ntn = (a.n + kTileN - 1) / kTileN;
  // (rows / BM + mats row tiles of at most 4096 column blocks stay below the
  // limit; only ranges that overlap could have more)
  const int total = min(mtiles, kMaxTiles / ntn) * ntn;
  const int nsteps = a.k / 128;

  // ---- which tiles are this workgroup's: runs of gridDim/8 consecutive
  // tiles go to one XCD (workgroups go to the XCDs round-robin), so that the
  // tiles that share rows or weights share an L2; few tiles are spread
  const int G = gridDim.x, b = blockIdx.x;
  const bool by_xcd = G % 8 == 0 && total > G;
  const int first = by_xcd ? (b & 7) * (G / 8) + (b >> 3) : b;
  if (first >= total) return;

  struct TileAt {
    int e, row0, rows, col0;
  };
  // tile `pos` of the list: matrix by matrix, panels of kPanel row tiles, in
  // a panel column block by column block
  auto tile_at = [&](int pos) -> TileAt {
    const int q = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(ntn)));
    TileAt t;
    t.e = tile_matrix(prefix, a.mats, q);
    const int p0 = __builtin_amdgcn_readfirstlane(prefix[t.e]), p1 = __builtin_amdgcn_readfirstlane(prefix[t.e + 1]);
    const uint32_t local = pos - p0 * ntn, pn = kPanel * ntn;
    const int panel = __builtin_amdgcn_readfirstlane(static_cast<int>(local / pn)), within = local - panel * pn;
    const int gm = min(kPanel, p1 - p0 - panel * kPanel);
    const int nt = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(within) / static_cast<uint32_t>(gm))), mt = panel * kPanel + within - nt * gm;
    int lo = 0, hi = static_cast<int>(a.rows);
    if (a.offsets) {
      sload2(a.offsets + t.e, lo, hi);
      const int rows = static_cast<int>(a.rows);
      lo = min(max(lo, 0), rows);
      hi = max(lo, min(max(hi, 0), rows));
    }
    t.row0 = lo + mt * BM;
    t.rows = min(BM, hi - t.row0);
    t.col0 = nt * kTileN;
    return t;
  };

  // ---- issue side
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)lds));
  int iss_pos = first, iss_step = 0, iss_slot = 0, iss_group = 0;
  const uint8_t *ia = nullptr, *iw = nullptr, *ias = nullptr, *iws = nullptr;  // the tile's first row, column
  uint32_t oa[P::CA], ow[P::CW], osa, osw;
  const int kb = a.k / 2, sb = a.k / 32;
  const int sa_blk = wave % P::CA;  // 64-row block of activation scales that this wave copies
  auto iss_setup = [&](const TileAt& t) {
    ia = uniform(a.a_c + int64_t(t.row0) * kb);
    ias = uniform(a.a_s + int64_t(t.row0) * sb);
    const int64_t wrow = int64_t(t.e) * a.n + t.col0;
    iw = uniform(a.w_c + wrow * kb);
    iws = uniform(a.w_s + wrow * sb);
    const int rlast = t.rows - 1, clast = min(kTileN, a.n - t.col0) - 1;
    const int chunk = 16 * ((lane & 3) ^ (lane >> 4));
#pragma unroll
    for (int q = 0; q < P::CA; ++q) oa[q] = min(16 * (P::CA * wave + q) + (lane >> 2), rlast) * kb + chunk;
#pragma unroll
    for (int q = 0; q < P::CW; ++q) ow[q] = min(16 * (P::CW * wave + q) + (lane >> 2), clast) * kb + chunk;
    osa = min(64 * sa_blk + lane, rlast) * sb;
    osw = min(64 * wave + lane, clast) * sb;
  };
  // (total and G are at most 2^30: no overflow)
  auto next_pos = [&](int pos) { return pos + G; };
  // The copies of the step at the issue side, numbered 0 .. copies-1; I: its
  // place in its group of four steps.
  auto issue = [&](auto ic, auto mc) {
    constexpr int I = decltype(ic)::value, m = decltype(mc)::value;
    const uint32_t slot = lds0 + iss_slot * P::SLOT;
    if constexpr (m < P::CA) copy16(oa[m], ia, slot + P::A + (P::CA * wave + m) * 1024);
    else if constexpr (m < P::CA + P::CW) copy16(ow[m - P::CA], iw, slot + P::W + (P::CW * wave + m - P::CA) * 1024);
    else if constexpr (!AG) {
      if constexpr (m == P::CA + P::CW) copy4(osa, ias, slot + P::SC + sa_blk * 256);
      if constexpr (m == P::CA + P::CW + 1) copy4(osw, iws, slot + P::SC + BM * 4 + wave * 256);
    } else if constexpr (I == 0) {
      const uint32_t buf = lds0 + P::GROUP + iss_group * (BM + kTileN) * 16;
      if constexpr (m == P::CA + P::CW) copy16(osa, ias, buf + sa_blk * 1024);
      if constexpr (m == P::CA + P::CW + 1) copy16(osw, iws, buf + BM * 16 + wave * 1024);
    }
  };
  // to the next step; behind the last tile the last one is copied again, into
  // slots that are not read
  auto advance = [&](auto ic) {
    constexpr int I = decltype(ic)::value;
    iss_slot = iss_slot + 1 == S ? 0 : iss_slot + 1;
    ia += 64;
    iw += 64;
    if (!AG) {
      ias += 4;
      iws += 4;
    } else if (I == 3) {
      ias += 16;
      iws += 16;
      iss_group ^= 1;
    }
    ++iss_step;
    // (with AG a tile ends with a group of four steps)
    if ((!AG || I == 3) && iss_step == nsteps) {
      iss_step = 0;
      if (next_pos(iss_pos) < total) iss_pos = next_pos(iss_pos);
      iss_setup(tile_at(iss_pos));
    }
  };

  // ---- read side: byte offsets in a slot of this lane's fragments of K half
  // 0 (half 1: chunk ^ 2), row blocks 2048 bytes apart
  const int swz = (l32 >> 2) & 3;
  const int fa = P::A + (wm * MI * 32 + l32) * 64, fw = P::W + (wn * NI * 32 + l32) * 64;
  const int ch[2] = {16 * (g32 ^ swz), 16 * ((2 + g32) ^ swz)};
  uint4 av[2][MI], wv[2][NI];
  uint4 agr[MI], wgr[NI];           // AG: four steps' scales
  uint32_t araw[MI], wraw[NI];      // otherwise the next step's
  uint32_t asc[MI], wsc[NI];
  auto read_frag = [&](int slot, auto hc, auto jc) {
    constexpr int H = decltype(hc)::value, j = decltype(jc)::value;
    const uint8_t* p = lds + slot * P::SLOT;
    if constexpr (j < NI) wv[H][j] = *reinterpret_cast<const uint4*>(p + fw + ch[H] + j * 2048);
    else av[H][j - NI] = *reinterpret_cast<const uint4*>(p + fa + ch[H] + (j - NI) * 2048);
  };
  // scales of the step in `slot`, the I-th of its group (group buffer grp)
  auto read_scales = [&](int slot, int grp, auto ic) {
    constexpr int I = decltype(ic)::value;
    if constexpr (AG) {
      if constexpr (I == 0) {
        const uint8_t* p = lds + P::GROUP + grp * (BM + kTileN) * 16;
#pragma unroll
        for (int j = 0; j < NI; ++j) wgr[j] = *reinterpret_cast<const uint4*>(p + (BM + (wn * NI + j) * 32 + l32) * 16);
#pragma unroll
        for (int i = 0; i < MI; ++i) agr[i] = *reinterpret_cast<const uint4*>(p + ((wm * MI + i) * 32 + l32) * 16);
      }
    } else {
      const uint8_t* p = lds + slot * P::SLOT + P::SC;
#pragma unroll
      for (int j = 0; j < NI; ++j) wraw[j] = *reinterpret_cast<const uint32_t*>(p + (BM + (wn * NI + j) * 32 + l32) * 4);
#pragma unroll
      for (int i = 0; i < MI; ++i) araw[i] = *reinterpret_cast<const uint32_t*>(p + ((wm * MI + i) * 32 + l32) * 4);
    }
  };
  auto shift_scales = [&](auto ic) {
    constexpr int I = decltype(ic)::value;
    auto pick = [&](const uint4& g, uint32_t raw) -> uint32_t {
      return (AG ? (I == 0 ? g.x : I == 1 ? g.y : I == 2 ? g.z : g.w) : raw) >> (8 * g32);
    };
#pragma unroll
    for (int j = 0; j < NI; ++j) wsc[j] = pick(wgr[j], wraw[j]);
#pragma unroll
    for (int i = 0; i < MI; ++i) asc[i] = pick(agr[i], araw[i]);
  };

  v16f acc[MI][NI];
  // The products so far stay before this point (without it the compiler moves
  // them past the branches below, to where the sums are next used).
  auto settle = [&] {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) asm volatile("" : "+a"(acc[i][j]));
  };
  int slot = 0, group = 0;
  // One step.  after_stores: the last tile's stores are among the
  // outstanding operations, so the wait takes them all.
  auto step = [&](auto ic, bool after_stores) {
    constexpr int I = decltype(ic)::value;
    const int nslot = slot + 1 == S ? 0 : slot + 1;
    shift_scales(ic);
    unrolled<0, NM>([&](auto kc) {
      constexpr int k = decltype(kc)::value, i = k / NI, j = k % NI;
      acc[i][j] = mfma32_fp4<0>(wv[0][j], av[0][i], acc[i][j], wsc[j], asc[i]);
      // the reads of half 1, spread over the first three quarters
      constexpr int R = MI + NI, lo = k * R / (NM * 3 / 4), hi = (k + 1) * R / (NM * 3 / 4);
      unrolled<(lo < R ? lo : R), (hi < R ? hi : R)>([&](auto jc) { read_frag(slot, Int<1>{}, jc); });
      __builtin_amdgcn_sched_barrier(0);
    });
    settle();
    wait_lds();
    // outstanding: the copies of steps s + 1 .. s + S - 1, of which s + 1's
    // have to be done
    constexpr int left = [] {
      int n = 0;
      for (int q = 2; q < S; ++q) n += P::copies(I + q);
      return n;
    }();
    if (after_stores) wait_vm<0>();
    else wait_vm<left>();
    tile_barrier();
    constexpr int C = P::copies(I + S);
    unrolled<0, NM>([&](auto kc) {
      constexpr int k = decltype(kc)::value, i = k / NI, j = k % NI;
      acc[i][j] = mfma32_fp4<1>(wv[1][j], av[1][i], acc[i][j], wsc[j], asc[i]);
      if constexpr (k == 0) read_scales(nslot, I == 3 ? group ^ 1 : group, Int<(I + 1) % 4>{});
      constexpr int R = MI + NI, H = NM / 2;
      unrolled<(k < H ? k * R / H : R), (k < H ? (k + 1) * R / H : R)>([&](auto jc) { read_frag(nslot, Int<0>{}, jc); });
      // the copies of step s + S, in the later half
      unrolled<(k < H ? 0 : (k - H) * C / (NM - H)), (k < H ? 0 : (k - H + 1) * C / (NM - H))>(
          [&](auto mc) { issue(Int<(I + S) % 4>{}, mc); });
      __builtin_amdgcn_sched_barrier(0);
    });
    settle();
    advance(Int<(I + S) % 4>{});
    slot = nslot;
    if (I == 3) group ^= 1;
  };

  // ---- results: acc[i][j] of this wave.  Buffer stores with the tile's first
  // row as base: a lane whose row or columns are not there takes an offset past
  // the buffer's end and stores nothing, so there are no branches (which would
  // cost copies of the accumulators).
  constexpr uint32_t kNowhere = 0x80000000u;  // the buffer ends here
  auto store_tile = [&](const TileAt& t) {
    constexpr int SZ = sizeof(T), PER = 16 / SZ;
    const uint64_t base = reinterpret_cast<uint64_t>(static_cast<T*>(a.y) + int64_t(t.row0) * a.ld_y + t.col0);
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, kNowhere, 0x00027000);
    const int row = wm * MI * 32 + l32, cols = a.n - t.col0;
    const uint32_t ld = static_cast<uint32_t>(a.ld_y) * SZ;
    // the last MFMA's results take 16 passes (18 wait states); the compiler
    // counts them for its own reads, not for the assembly's below
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    uint32_t at[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) at[i] = row + 32 * i < t.rows ? (row + 32 * i) * ld : kNowhere;
    unrolled<0, NM>([&](auto bc) {
      constexpr int i = decltype(bc)::value / NI, j = decltype(bc)::value % NI;
      typedef uint32_t v4u __attribute__((ext_vector_type(4)));
      const v16f& r = acc[i][j];
      // result x of the block out of its accumulator register, here and not
      // earlier: the compiler would move every block's together, and there is
      // no room for them
      auto c = [&](int x) -> float {
        if constexpr (SZ == 4 && WIDE) return r[x];  // stored from there
        float f;
        asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(f) : "a"(r[x]));
        return f;
      };
      auto put = [&](int cx, v4u v) {
        __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, cx < cols ? at[i] + cx * SZ : kNowhere, 0, 0);
      };
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = (wn * NI + j) * 32 + 8 * q;
        if constexpr (!WIDE) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int cx = col + 4 * g32 + x;
            const uint32_t off = cx < cols ? at[i] + cx * SZ : kNowhere;
            const T v = from_f32<T>(c(4 * q + x));
            if constexpr (SZ == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), rsrc, off, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), rsrc, off, 0, 0);
          }
        } else if constexpr (SZ == 4) {
          const v4f v = {c(4 * q), c(4 * q + 1), c(4 * q + 2), c(4 * q + 3)};
          put(col + 4 * g32, __builtin_bit_cast(v4u, v));
        } else if (q % 2 == 0) {
          // lanes l and l + 32 exchange halves: 16 bytes of a row each
          const uint32_t x0 = pack2<T>(c(4 * q), c(4 * q + 1)), x1 = pack2<T>(c(4 * q + 2), c(4 * q + 3));
          const uint32_t y0 = pack2<T>(c(4 * q + 4), c(4 * q + 5)), y1 = pack2<T>(c(4 * q + 6), c(4 * q + 7));
          const auto s0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
          put(col + 8 * g32, v4u{s0[0], s1[0], s0[1], s1[1]});
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // ---- the stream of steps
  iss_setup(tile_at(iss_pos));
  if constexpr (AG) {
    // a matrix has at least four steps, and S of them start here
    unrolled<0, S>([&](auto sc) {
      constexpr int I = decltype(sc)::value % 4;
      unrolled<0, P::copies(I)>([&](auto mc) { issue(Int<I>{}, mc); });
      advance(Int<I>{});
    });
  } else {
    for (int q = 0; q < S; ++q) {
      unrolled<0, P::copies(0)>([&](auto mc) { issue(Int<0>{}, mc); });
      advance(Int<0>{});
    }
  }
  constexpr int ahead = [] {
    int n = 0;
    for (int q = 1; q < S; ++q) n += P::copies(q);
    return n;
  }();
  wait_vm<ahead>();
  tile_barrier();
  read_scales(0, 0, Int<0>{});
  unrolled<0, MI + NI>([&](auto jc) { read_frag(0, Int<0>{}, jc); });

  bool stored = false;
  for (int pos = first; pos < total; pos = next_pos(pos)) {
    const TileAt t = tile_at(pos);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = v16f{};
    if constexpr (AG) {
      int s = 0;
      do {
        step(Int<0>{}, stored);
        stored = false;
        step(Int<1>{}, false);
        step(Int<2>{}, false);
        step(Int<3>{}, false);
      } while ((s += 4) < nsteps);
    } else {
      int s = 0;
      do {
        step(Int<0>{}, stored);
        stored = false;
      } while (++s < nsteps);
    }
    store_tile(t);
    stored = true;
  }
  // the copies still on their way land in this workgroup's LDS
  wait_vm<0>();
}

// four columns of a row can be stored at once
bool wide_stores(const LinearArgs& a, int64_t sz) { return rows_aligned(a.y, a.ld_y * sz, 4 * sz); }

template <typename T>
hipError_t stream_t(const LinearArgs& a, hipStream_t st) {
  const int64_t tiles = a.offsets ? std::min<int64_t>(a.rows, (a.rows + 15) / 16 + a.mats) : (a.rows + 15) / 16;
  const int64_t units = tiles * ((a.n + 15) / 16);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(units, 8 * a.num_cus));
  const bool wide = wide_stores(a, sizeof(T));
  const int64_t sb = a.k / 32;
  auto on = [&](int64_t al) { return rows_aligned(a.a_s, sb, al) && rows_aligned(a.w_s, sb, al); };
  if (a.k % 512 == 0 && on(16)) k_linear_stream<T, 0><<<grid, kStreamThreads, 0, st>>>(a, wide);
  else if (a.k % 128 == 0 && on(4)) k_linear_stream<T, 1><<<grid, kStreamThreads, 0, st>>>(a, wide);
  else k_linear_stream<T, 2><<<grid, kStreamThreads, 0, st>>>(a, wide);
  return hipGetLastError();
}

template <typename T, int BM>
hipError_t tile_t(const LinearArgs& a, hipStream_t st) {
  const int64_t mtiles = a.offsets ? std::min<int64_t>(a.rows, (a.rows + BM - 1) / BM + a.mats) : (a.rows + BM - 1) / BM;
  const int64_t tiles = mtiles * ((a.n + kTileN - 1) / kTileN);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, a.num_cus));
  const int64_t sb = a.k / 32;
  const bool wide = rows_aligned(a.y, a.ld_y * sizeof(T), 16) && a.n % (16 / sizeof(T)) == 0;
  if (!wide)
    k_linear_tile<T, BM, false, false><<<grid, kTileThreads, 0, st>>>(a);
  else if (a.k % 512 == 0 && rows_aligned(a.a_s, sb, 16) && rows_aligned(a.w_s, sb, 16))
    k_linear_tile<T, BM, true, true><<<grid, kTileThreads, 0, st>>>(a);
  else
    k_linear_tile<T, BM, false, true><<<grid, kTileThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t linear_t(const LinearArgs& a, hipStream_t st) {
  // rows per matrix on average; the offsets are on the device
  const int64_t avg = a.rows / a.mats;
  const int64_t sb = a.k / 32;
  // (the tile kernel's stores reach 2^31 bytes from a tile's first row)
  if (a.ld_y * sizeof(T) * 256 > (int64_t(1) << 31)) return stream_t<T>(a, st);
  if (a.k % 128 || !rows_aligned(a.a_s, sb, 4) || !rows_aligned(a.w_s, sb, 4) || avg <= 16) return stream_t<T>(a, st);
  if (avg <= 96) return tile_t<T, 64>(a, st);
  if (avg <= 192) return tile_t<T, 128>(a, st);
  return tile_t<T, 256>(a, st);
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
