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
#include "linear_choice.h"
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

// prefix[e] = row tiles (of TM rows) of the matrices before e; one pass of the
// whole workgroup (part: a word of LDS per wave).  Returns the number of tiles.
template <int THREADS, int TM>
__device__ __forceinline__ int tile_prefix(const LinearArgs& a, int* prefix, int* part) {
  if (!a.offsets) {
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    return static_cast<int>((a.rows + TM - 1) / TM);
  }
  constexpr int PER = (kMaxMats + THREADS - 1) / THREADS;
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
    if (e < a.mats) prefix[e] = at;
    at += n[i];
  }
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
// Few products: straight from memory to registers in operand order.  A unit is
// 16 MT rows x 16 NB columns; a persistent grid takes them round-robin, the
// columns of a row tile fastest, so that neighbouring workgroups read
// neighbouring weight rows.  The NW waves of a workgroup share a unit's K:
// wave w takes the 512-wide groups w, w + NW, ... (256 bytes of each row), and
// the partial sums meet in LDS in wave order.  With at most one unit per CU
// NW is 8 and a wave has the next group's loads on their way while it
// multiplies this one: the time is that of one or two loads (1 row x 4096
// columns, k = 7168: 6.5 us against 7.4 with four waves).  With more units
// NW is 4 and several workgroups per CU hide each other's loads.
//
// SCALES: how the scale bytes come.  0: 16 bytes for a row's four steps
// (k % 512 == 0); 1: a dword per step (k % 128 == 0); 2: single bytes, with
// the last step's missing blocks left out (any multiple of 32).
// ---------------------------------------------------------------------------
template <typename T, int SCALES, int MT, int NB, int NW>
__global__ void __launch_bounds__(64 * NW, NW == 4 ? 4 : 2) k_linear_stream(LinearArgs a, bool wide) {
  static_assert(MT * NB <= NW, "a wave joins one block of a unit");
  __shared__ int prefix[kMaxMats];
  __shared__ int part[NW];
  __shared__ float4 sums[NW][MT * NB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int r16 = lane & 15, g = lane >> 4;
  const int tiles = tile_prefix<64 * NW, 16 * MT>(a, prefix, part);
  const int cblocks = (a.n + 16 * NB - 1) / (16 * NB);
  const int64_t units = int64_t(tiles) * cblocks;
  const int nb = a.k / 32;                     // blocks of 32 along k
  const int groups = (nb + 15) / 16;
  struct Operand {
    uint4 v[4];
    uint32_t s[4];
  };
  // group q of one row (its codes at c, its scales at s; ok: the row is there)
  auto load = [&](Operand& o, const uint8_t* c, const uint8_t* s, bool ok, int q) {
    if constexpr (SCALES == 0) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (ok) x = *reinterpret_cast<const uint4*>(s + 16 * q);
      o.s[0] = x.x; o.s[1] = x.y; o.s[2] = x.z; o.s[3] = x.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = 16 * q + 4 * i + g;        // this lane's block
      const bool in = ok && b < nb;
      o.v[i] = make_uint4(0, 0, 0, 0);
      if (in) o.v[i] = *reinterpret_cast<const uint4*>(c + 16 * int64_t(b));
      if constexpr (SCALES == 1) o.s[i] = in ? *reinterpret_cast<const uint32_t*>(s + b - g) : 0;
      if constexpr (SCALES == 2) o.s[i] = in ? s[b] : 0;
    }
  };
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    // (a 64-bit division takes a tenth of a short call)
    const int t = static_cast<int>(units < (int64_t(1) << 31) ? static_cast<uint32_t>(u) / static_cast<uint32_t>(cblocks)
                                                              : u / cblocks);
    const int cb = static_cast<int>(u - int64_t(t) * cblocks);
    const int e = tile_matrix(prefix, a.mats, t);
    int lo, hi;
    mat_rows(a, e, lo, hi);
    lo += (t - prefix[e]) * 16 * MT;
    const uint8_t *ap[MT], *as[MT], *wp[NB], *ws[NB];
    bool row_ok[MT], col_ok[NB];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = lo + 16 * i + r16;
      row_ok[i] = row < hi;
      ap[i] = a.a_c + int64_t(row) * (a.k / 2);
      as[i] = a.a_s + int64_t(row) * nb;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int col = (cb * NB + j) * 16 + r16;
      col_ok[j] = col < a.n;
      wp[j] = a.w_c + (int64_t(e) * a.n + col) * (a.k / 2);
      ws[j] = a.w_s + (int64_t(e) * a.n + col) * nb;
    }
    v4f acc[MT][NB];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto loads = [&](Operand* x, Operand* w, int q) {
#pragma unroll
      for (int j = 0; j < NB; ++j) load(w[j], wp[j], ws[j], col_ok[j], q);
#pragma unroll
      for (int i = 0; i < MT; ++i) load(x[i], ap[i], as[i], row_ok[i], q);
    };
    auto products = [&](const Operand* x, const Operand* w) {
      const int sh = SCALES == 2 ? 0 : 8 * g;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j) acc[i][j] = mfma_fp4(w[j].v[k], x[i].v[k], acc[i][j], w[j].s[k] >> sh, x[i].s[k] >> sh);
    };
    if constexpr (MT * NB == 1 && NW == 8) {
      Operand x[2], w[2];
      int q = wave;
      if (q < groups) loads(&x[0], &w[0], q);
      while (q < groups) {
        if (q + NW < groups) loads(&x[1], &w[1], q + NW);
        products(&x[0], &w[0]);
        x[0] = x[1];
        w[0] = w[1];
        q += NW;
      }
    } else {
      Operand x[MT], w[NB];
      for (int q = wave; q < groups; q += NW) {
        loads(x, w, q);
        products(x, w);
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        sums[wave][i * NB + j][lane] = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
    __syncthreads();
    // waves 0 .. MT NB - 1 each join one block of the unit
    if (wave < MT * NB) {
      v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float4 p = sums[w][wave][lane];
        s[0] += p.x; s[1] += p.y; s[2] += p.z; s[3] += p.w;
      }
      const int row = lo + 16 * (wave / NB) + r16;
      if (row < hi) store_cols(static_cast<T*>(a.y), a.ld_y, row, (cb * NB + wave % NB) * 16 + 4 * g, a.n, wide, s);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Many rows per matrix: BM x 256 tiles through LDS.  One workgroup of four
// waves per CU walks its tiles; a step is 256 of K, four quarters of 64.  The
// step's codes (128 bytes of each of BM activation and 256 weight rows) come
// by direct-to-LDS copies into a ring of S slots, and the stream of steps runs
// on across the tiles: while a tile ends, the first steps of the next are
// already on their way.  In a quarter a wave issues its MI x NI MFMAs
// 32x32x64 and between them the LDS reads of the next quarter; before the last
// quarter it waits for its own copies of step s + 1 and at a barrier (all
// waves' copies have landed, and all have read slot s), and from there on the
// copies of step s + S go into slot s, spread over the following quarters so
// that the waves do not queue behind them.
// The weights are the first MFMA operand: lane (l32, g32) register r of a
// 32x32 result is column 8(r/4) + 4 g32 + r%4 of activation row l32, so four
// registers are four consecutive columns of y.
//
// LDS slot: activation rows, then weight rows, 128 bytes each; the 16-byte
// chunk c of row r sits at chunk c ^ (r%8), so that the eight lanes that the
// LDS serves together (eight rows, one chunk) touch all banks once.  A copy
// moves 8 rows: lane l brings chunk (l%8) ^ (l/8) of row l/8, eight lanes the
// 128 bytes (one cache line) of a row.  Pieces of 64 bytes, from steps half as
// wide, cost a quarter of the copies' rate: 95 against 75 us for the copies
// alone of 8192 x 4096 x 7168.
//
// Scales come in pieces of GS steps, 8 GS bytes of each row, into one of two
// buffers, from where every second step 16 bytes per row go to registers: GS
// = 4 (k % 1024 == 0; 64-row tiles, whose rows are many for their products)
// or 2 (k % 512 == 0), scale rows on 16 bytes; GS = 0 otherwise: two dwords
// per row and step, in the slot.  The number of pieces matters more than their
// bytes: in one comparison 4096 rows over 64 matrices of 4096 x 7168 took 213 us
// without any (and wrong results), 243 us with GS = 2.  A dword holds half a step's scales, byte 2q + g32 that
// of its quarter q of lane (l32, g32): shifted by 8 g32 once per step, the
// MFMA takes byte 2q.
//
// Measured (medians of single calls): 8192 x 4096, k = 7168, 112 us (4.3 PF; the
// matrix cores busy 54 % of the cycles, at a clock of 1.9 GHz); 131072 rows over
// 64 matrices of 7168 x 2048 1.15 ms in a row of calls, 1.22 ms among pauses
// (3.3 PF; busy 49 %, 1.35 to 1.65 GHz): a tile's results are stored while no
// MFMA runs; 16 rows for 16 of 64 matrices of 4096 x 7168 41.8 us (6.0 TB/s of
// weights).
//
// With k % 256 == 128 a row's last step is half a step: its copies bring the
// first 64 bytes twice, and it has two quarters.  Rows past the tile's or the
// matrix's end are copied from the last valid row and their results not stored.
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
// the same with the non-temporal hint
__device__ __forceinline__ void copy16_nt(uint32_t off, const uint8_t* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(off), "s"(base), "s"(lds)
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

constexpr int kTileThreads = 256;
constexpr int kPanel = 4;  // row tiles that share a column block's weights in time

template <int SZ, int BM, int GS>
struct TileShape {
  static constexpr int WM = BM == 64 ? 1 : 2, WN = 4 / WM;        // waves along rows, columns
  static constexpr int MI = BM / WM / 32, NI = kTileN / WN / 32;  // 32-row, 32-column blocks of a wave
  static constexpr int S = BM == 256 ? 2 : 3;                     // ring slots
  static constexpr int A = 0, W = BM * 128, SC = W + kTileN * 128;  // slot: activations, weights, scale dwords
  static constexpr int SLOT = SC + (GS ? 0 : (BM + kTileN) * 8);
  static constexpr int GROUP = S * SLOT, PIECE = 8 * GS;          // scale pieces, two buffers
  static constexpr int LDS = GROUP + 2 * (BM + kTileN) * PIECE;
  static constexpr int U = GS ? GS : 1;                           // steps that are unrolled
  static constexpr int CA = BM / 32, CW = 8;                      // copies of codes per wave and step
  // of scales: rows per copy, copies of a wave (waves that have none left
  // over repeat another's, so that all count alike)
  static constexpr int PR = GS ? 1024 / PIECE : 64;
  static constexpr int CSA = GS ? (BM / PR + 3) / 4 : 2, CSW = GS ? kTileN / PR / 4 : 2;
  // copies of a wave for a step, the i-th of its group
  static constexpr int copies(int i) { return CA + CW + (i % U == 0 ? CSA + CSW : 0); }
  static constexpr int copies_from(int i, int n) { return n <= 0 ? 0 : copies(i) + copies_from(i + 1, n - 1); }
  // those issued in the last quarter before their step's slot is S - 1 steps
  // away: half of them with two slots (they have to land soon), else a quarter
  static constexpr int first_part(int i) { return copies(i) / (S == 2 ? 2 : 4); }
  static constexpr int STORES = MI * NI * 4 * SZ / 4;             // a wave's stores of a tile (16 bytes a lane)
};

// WIDE: n and the rows of y are whole numbers of 16-byte pieces.
// ONCE: nearly every matrix has one row tile, so its weights are read once:
// their copies carry the non-temporal hint (16 rows for 16 of 64 matrices of
// 4096 x 7168: 43.7 against 46.7 us; with several row tiles it costs 5 %).
template <typename T, int BM, int GS, bool WIDE, bool ONCE>
__global__ void __launch_bounds__(kTileThreads, 1) k_linear_tile(LinearArgs a) {
  using P = TileShape<sizeof(T), BM, GS>;
  constexpr int S = P::S, U = P::U, MI = P::MI, NI = P::NI, NM = MI * NI;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[P::LDS];
  __shared__ int prefix[kMaxMats];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int l32 = lane & 31, g32 = lane >> 5;
  const int wm = wave / P::WN, wn = wave % P::WN;
  const int mtiles =
      __builtin_amdgcn_readfirstlane(tile_prefix<kTileThreads, BM>(a, prefix, reinterpret_cast<int*>(lds)));
  const int ntn = (a.n + kTileN - 1) / kTileN;
  // (the caller has seen to it that rows / BM + mats row tiles stay below the
  // limit: only ranges that overlap, many times over, can have more)
  const int total = min(mtiles, static_cast<int>(kMaxLinearTiles) / ntn) * ntn;
  const int nsteps = (a.k + 255) / 256;
  const bool odd = !GS && (a.k & 128);  // the last step is half a step

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
    const int p0 = __builtin_amdgcn_readfirstlane(prefix[t.e]);
    const int p1 = t.e + 1 < a.mats ? __builtin_amdgcn_readfirstlane(prefix[t.e + 1]) : mtiles;
    const uint32_t local = pos - p0 * ntn, pn = kPanel * ntn;
    const int panel = __builtin_amdgcn_readfirstlane(static_cast<int>(local / pn)), within = local - panel * pn;
    const int gm = min(kPanel, p1 - p0 - panel * kPanel);
    const int nt = __builtin_amdgcn_readfirstlane(
        static_cast<int>(static_cast<uint32_t>(within) / static_cast<uint32_t>(gm)));
    const int mt = panel * kPanel + within - nt * gm;
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
  uint32_t oa[P::CA], ow[P::CW], osa[GS ? P::CSA : 1], osw[GS ? P::CSW : 1];
  const int kb = a.k / 2, sb = a.k / 32;
  // block of PR activation rows whose scales this wave's copy number n brings
  auto sa_blk = [&](int n) { return (P::CSA * wave + n) % (BM / P::PR); };
  // half a step's copies: chunks 4-7 are not there, the first four come again
  const int chunk = (lane & 7) ^ (lane >> 3);
  const uint32_t half_back = chunk & 4 ? 64 : 0;
  auto iss_setup = [&](const TileAt& t) {
    ia = uniform(a.a_c + int64_t(t.row0) * kb);
    ias = uniform(a.a_s + int64_t(t.row0) * sb);
    const int64_t wrow = int64_t(t.e) * a.n + t.col0;
    iw = uniform(a.w_c + wrow * kb);
    iws = uniform(a.w_s + wrow * sb);
    const int rlast = t.rows - 1, clast = min(kTileN, a.n - t.col0) - 1;
#pragma unroll
    for (int q = 0; q < P::CA; ++q) oa[q] = min(8 * (P::CA * wave + q) + (lane >> 3), rlast) * kb + 16 * chunk;
#pragma unroll
    for (int q = 0; q < P::CW; ++q) ow[q] = min(8 * (P::CW * wave + q) + (lane >> 3), clast) * kb + 16 * chunk;
    constexpr int LR = 64 / P::PR;  // lanes that share a row's piece
#pragma unroll
    for (int n = 0; n < (GS ? P::CSA : 1); ++n)
      osa[n] = min(P::PR * (GS ? sa_blk(n) : wave % (BM / 64)) + lane / LR, rlast) * sb + 16 * (lane % LR);
#pragma unroll
    for (int n = 0; n < (GS ? P::CSW : 1); ++n)
      osw[n] = min(P::PR * (GS ? P::CSW * wave + n : wave) + lane / LR, clast) * sb + 16 * (lane % LR);
  };
  // (total and G are at most 2^30: no overflow)
  auto next_pos = [&](int pos) { return pos + G; };
  // Copy number m of the step at the issue side, the I-th of its group.
  auto issue = [&](auto ic, auto mc) {
    constexpr int I = decltype(ic)::value, m = decltype(mc)::value, n = m - P::CA - P::CW;
    const uint32_t slot = lds0 + iss_slot * P::SLOT;
    const bool half = odd && iss_step == nsteps - 1;
    const uint32_t back = half ? half_back : 0;
    if constexpr (m < P::CA) copy16(oa[m] - back, ia, slot + P::A + (P::CA * wave + m) * 1024);
    else if constexpr (n < 0 && ONCE) copy16_nt(ow[m - P::CA] - back, iw, slot + P::W + (P::CW * wave + m - P::CA) * 1024);
    else if constexpr (n < 0) copy16(ow[m - P::CA] - back, iw, slot + P::W + (P::CW * wave + m - P::CA) * 1024);
    else if constexpr (!GS) {
      // dword n/2 of the step (half a step has one: it comes again)
      const uint32_t d = n >= 2 && !half ? 4 : 0, at = slot + P::SC + (n / 2) * (BM + kTileN) * 4;
      if constexpr (n % 2 == 0) copy4(osa[0] + d, ias, at + wave % (BM / 64) * 256);
      else copy4(osw[0] + d, iws, at + BM * 4 + wave * 256);
    } else if constexpr (I == 0) {
      const uint32_t buf = lds0 + P::GROUP + iss_group * (BM + kTileN) * P::PIECE;
      if constexpr (n < P::CSA) copy16(osa[n], ias, buf + sa_blk(n) * 1024);
      else copy16(osw[n - P::CSA], iws, buf + BM * P::PIECE + (P::CSW * wave + n - P::CSA) * 1024);
    }
  };
  // to the next step; behind the last tile the last one is copied again, into
  // slots that are not read
  auto advance = [&](auto ic) {
    constexpr int I = decltype(ic)::value;
    iss_slot = iss_slot + 1 == S ? 0 : iss_slot + 1;
    ia += 128;
    iw += 128;
    if (I == U - 1) {
      ias += 8 * U;
      iws += 8 * U;
      iss_group ^= 1;
    }
    ++iss_step;
    // (a tile ends with a group of steps)
    if (I == U - 1 && iss_step == nsteps) {
      iss_step = 0;
      if (next_pos(iss_pos) < total) iss_pos = next_pos(iss_pos);
      iss_setup(tile_at(iss_pos));
    }
  };

  // ---- read side: byte offsets in a slot of this lane's fragments, row
  // blocks 4096 bytes apart; quarter h of a step is chunks 2h and 2h + 1
  const int fa = P::A + (wm * MI * 32 + l32) * 128, fw = P::W + (wn * NI * 32 + l32) * 128;
  const int ch[4] = {16 * (g32 ^ (l32 & 7)), 16 * ((2 + g32) ^ (l32 & 7)), 16 * ((4 + g32) ^ (l32 & 7)),
                     16 * ((6 + g32) ^ (l32 & 7))};
  uint4 av[2][MI], wv[2][NI];       // the fragments of this quarter and of the next
  uint4 agr[MI], wgr[NI];           // GS: two steps' scales
  uint2 araw[MI], wraw[NI];         // otherwise the next step's
  uint32_t asc[2][MI], wsc[2][NI];  // this step's, of its first and second half
  auto read_frag = [&](int slot, auto hc, auto jc) {
    constexpr int H = decltype(hc)::value, j = decltype(jc)::value;
    const uint8_t* p = lds + slot * P::SLOT;
    if constexpr (j < NI) wv[H % 2][j] = *reinterpret_cast<const uint4*>(p + fw + ch[H] + j * 4096);
    else av[H % 2][j - NI] = *reinterpret_cast<const uint4*>(p + fa + ch[H] + (j - NI) * 4096);
  };
  // scales of the step in `slot`, the I-th of its group (scale buffer grp)
  auto read_scales = [&](int slot, int grp, auto ic) {
    constexpr int I = decltype(ic)::value;
    if constexpr (GS) {
      if constexpr (I % 2 == 0) {
        const uint8_t* p = lds + P::GROUP + grp * (BM + kTileN) * P::PIECE + 8 * I;
#pragma unroll
        for (int j = 0; j < NI; ++j) wgr[j] = *reinterpret_cast<const uint4*>(p + (BM + (wn * NI + j) * 32 + l32) * P::PIECE);
#pragma unroll
        for (int i = 0; i < MI; ++i) agr[i] = *reinterpret_cast<const uint4*>(p + ((wm * MI + i) * 32 + l32) * P::PIECE);
      }
    } else {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(lds + slot * P::SLOT + P::SC);
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int at = BM + (wn * NI + j) * 32 + l32;
        wraw[j] = make_uint2(p[at], p[at + BM + kTileN]);
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int at = (wm * MI + i) * 32 + l32;
        araw[i] = make_uint2(p[at], p[at + BM + kTileN]);
      }
    }
  };
  auto shift_scales = [&](auto ic) {
    constexpr int I = decltype(ic)::value;
    const int sh = 8 * g32;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      wsc[0][j] = (GS ? (I % 2 == 0 ? wgr[j].x : wgr[j].z) : wraw[j].x) >> sh;
      wsc[1][j] = (GS ? (I % 2 == 0 ? wgr[j].y : wgr[j].w) : wraw[j].y) >> sh;
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      asc[0][i] = (GS ? (I % 2 == 0 ? agr[i].x : agr[i].z) : araw[i].x) >> sh;
      asc[1][i] = (GS ? (I % 2 == 0 ? agr[i].y : agr[i].w) : araw[i].y) >> sh;
    }
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
  // One step, the I-th of its group, of NQ quarters (4, or 2 for half a step).
  // FIRST: the tile's first, its products start from zero.  after_stores: the
  // last tile's stores may still be on their way (operations finish in the
  // order in which they were issued).
  auto step = [&](auto ic, auto nq, auto first_c, bool after_stores) {
    constexpr int I = decltype(ic)::value, NQ = decltype(nq)::value;
    constexpr bool FIRST = decltype(first_c)::value != 0;
    const int nslot = slot + 1 == S ? 0 : slot + 1;
    shift_scales(ic);
    // the copies of step s + S - 1, begun in the last quarter of step s - 1,
    // go on over the quarters before the barrier (with two slots: the first)
    constexpr int IP = (I + S - 1) % U, CP = P::copies(IP), C0 = P::first_part(IP);
    constexpr int QI = S == 2 ? 1 : NQ - 1;  // quarters that issue them
    unrolled<0, NQ>([&](auto qc) {
      constexpr int q = decltype(qc)::value;
      constexpr bool LAST = q == NQ - 1;
      if constexpr (q == QI || (LAST && QI > NQ - 1)) {
        settle();
        advance(Int<IP>{});
      }
      if constexpr (LAST) {
        settle();
        wait_lds();
        // outstanding: the copies of steps s + 1 .. s + S - 1, of which
        // s + 1's have to be done (with more than two slots all of them were
        // issued before the stores)
        constexpr int left = P::copies_from(I + 2, S - 2);
        if (S > 2 && after_stores) wait_vm<(left + P::STORES < 63 ? left + P::STORES : 63)>();
        else wait_vm<left>();
        tile_barrier();
      }
      unrolled<0, NM>([&](auto kc) {
        constexpr int k = decltype(kc)::value, i = k / NI, j = k % NI;
        acc[i][j] = mfma32_fp4<q % 2>(wv[q % 2][j], av[q % 2][i], FIRST && q == 0 ? v16f{} : acc[i][j], wsc[q / 2][j], asc[q / 2][i]);
        if constexpr (LAST && k == 0) read_scales(nslot, I == U - 1 ? group ^ 1 : group, Int<(I + 1) % U>{});
        // the next quarter's reads, in the first three quarters of this one
        constexpr int R = MI + NI, lo = k * R / (NM * 3 / 4), hi = (k + 1) * R / (NM * 3 / 4);
        unrolled<(lo < R ? lo : R), (hi < R ? hi : R)>(
            [&](auto jc) { read_frag(LAST ? nslot : slot, Int<LAST ? 0 : q + 1>{}, jc); });
        if constexpr (q < QI) {
          constexpr int n = NM * QI, x = q * NM + k;
          unrolled<C0 + x * (CP - C0) / n, C0 + (x + 1) * (CP - C0) / n>([&](auto mc) { issue(Int<IP>{}, mc); });
        }
        if constexpr (LAST) {
          constexpr int C = P::first_part(I + S);
          unrolled<k * C / NM, (k + 1) * C / NM>([&](auto mc) { issue(Int<(I + S) % U>{}, mc); });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    settle();
    slot = nslot;
    if (I == U - 1) group ^= 1;
  };

  // ---- results: acc[i][j] of this wave.  WIDE: buffer stores with the tile's
  // first row as base: a lane whose row or columns are not there takes an
  // offset past the buffer's end and stores nothing, so there are no branches
  // (which would cost copies of the accumulators).  Otherwise the same 16-byte
  // pieces at any address, and only a row's last one by elements (8192 x 4095,
  // k = 2048, bf16: 66 us, 121 us with every element on its own; 4096 columns
  // 44 us).
  constexpr uint32_t kNowhere = 0x80000000u;  // the buffer ends here
  auto store_tile = [&](const TileAt& t) {
    constexpr int SZ = sizeof(T), PER = 16 / SZ;
    const uint64_t base = reinterpret_cast<uint64_t>(static_cast<T*>(a.y) + int64_t(t.row0) * a.ld_y + t.col0);
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, kNowhere, 0x00027000);
    const int cols = a.n - t.col0;
    const uint32_t ld = static_cast<uint32_t>(a.ld_y) * SZ;
    // the last MFMA's results take 16 passes (18 wait states); the compiler
    // counts them for its own reads, not for the assembly's below
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    // this lane's rows: with 16-bit results lane l stores rows l%16 and
    // 16 + l%16 of each block of 32, otherwise row l%32
    constexpr bool HALVES = SZ == 2;
    constexpr int NR = HALVES ? 2 : 1;
    uint32_t at[MI][NR];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int h = 0; h < NR; ++h) {
        const int row = (wm * MI + i) * 32 + (HALVES ? 16 * h + (lane & 15) : l32);
        at[i][h] = row < t.rows ? row * ld : kNowhere;
      }
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
      auto put = [&](int h, int cx, v4u v) {
        if constexpr (WIDE) {
          __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, cx < cols ? at[i][h] + cx * SZ : kNowhere, 0, 0);
        } else if (at[i][h] != kNowhere && cx < cols) {
          // rows anywhere in memory, and a row's last piece in part
          char* to = reinterpret_cast<char*>(base) + at[i][h] + cx * SZ;
          if (cx + PER <= cols) {
            store16<false, false>(to, v);
          } else {
#pragma unroll
            for (int x = 0; x < PER - 1; ++x) {
              if (cx + x >= cols) break;
              if constexpr (SZ == 2) reinterpret_cast<uint16_t*>(to)[x] = static_cast<uint16_t>(v[x / 2] >> (16 * (x % 2)));
              else reinterpret_cast<uint32_t*>(to)[x] = v[x];
            }
          }
        }
      };
      const int col = (wn * NI + j) * 32;
      if constexpr (HALVES) {
        // lane (l32, g32) has columns 8q + 4 g32 .. + 3 of row l32, q = 0..3.
        // Lanes l and l + 32 exchange halves, and it has 8 columns (16 bytes),
        // 16p + 8 g32 .., p = 0, 1; then the 16-lane rows of the wave do, and
        // four lanes have the 64 bytes of a row of the block.
        uint32_t v[2][4];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const auto e = __builtin_amdgcn_permlane32_swap(pack2<T>(c(8 * p + 2 * x), c(8 * p + 2 * x + 1)),
                                                            pack2<T>(c(8 * p + 4 + 2 * x), c(8 * p + 5 + 2 * x)), false, false);
            v[p][x] = e[0];
            v[p][2 + x] = e[1];
          }
        v4u o[2];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const auto e = __builtin_amdgcn_permlane16_swap(v[0][x], v[1][x], false, false);
          o[0][x] = e[0];
          o[1][x] = e[1];
        }
        const int cx = col + 16 * ((lane >> 4) & 1) + 8 * g32;
        put(0, cx, o[0]);
        put(1, cx, o[1]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v4f v = {c(4 * q), c(4 * q + 1), c(4 * q + 2), c(4 * q + 3)};
          put(0, col + 8 * q + 4 * g32, __builtin_bit_cast(v4u, v));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // ---- the stream of steps: the first S - 1 and the first part of the next
  // are on their way before the first product
  iss_setup(tile_at(iss_pos));
  unrolled<0, S - 1>([&](auto sc) {
    constexpr int I = decltype(sc)::value % U;
    unrolled<0, P::copies(I)>([&](auto mc) { issue(Int<I>{}, mc); });
    advance(Int<I>{});
  });
  unrolled<0, P::first_part(S - 1)>([&](auto mc) { issue(Int<(S - 1) % U>{}, mc); });
  wait_vm<P::copies_from(1, S - 2) + P::first_part(S - 1)>();
  tile_barrier();
  read_scales(0, 0, Int<0>{});
  unrolled<0, MI + NI>([&](auto jc) { read_frag(0, Int<0>{}, jc); });

  bool stored = false;
  for (int pos = first; pos < total; pos = next_pos(pos)) {
    const TileAt t = tile_at(pos);
    // without WIDE the number of stores is not known here: wait for all
    if (!WIDE && stored) wait_vm<0>();
    stored &= WIDE;
    if constexpr (GS) {
      step(Int<0>{}, Int<4>{}, Int<1>{}, stored);
      step(Int<1>{}, Int<4>{}, Int<0>{}, false);
      if constexpr (U == 4) {
        step(Int<2>{}, Int<4>{}, Int<0>{}, false);
        step(Int<3>{}, Int<4>{}, Int<0>{}, false);
      }
      for (int s = U; s < nsteps; s += U) {
        step(Int<0>{}, Int<4>{}, Int<0>{}, false);
        step(Int<1>{}, Int<4>{}, Int<0>{}, false);
        if constexpr (U == 4) {
          step(Int<2>{}, Int<4>{}, Int<0>{}, false);
          step(Int<3>{}, Int<4>{}, Int<0>{}, false);
        }
      }
    } else {
      // half a step, if there is one, comes last; alone it is the first too
      if (nsteps == 1 && odd) {
        step(Int<0>{}, Int<2>{}, Int<1>{}, stored);
      } else {
        step(Int<0>{}, Int<4>{}, Int<1>{}, stored);
        const int full = odd ? nsteps - 1 : nsteps;
        for (int s = 1; s < full; ++s) step(Int<0>{}, Int<4>{}, Int<0>{}, false);
        if (odd) step(Int<0>{}, Int<2>{}, Int<0>{}, false);
      }
    }
    store_tile(t);
    stored = true;
  }
  // the copies still on their way land in this workgroup's LDS
  wait_vm<0>();
}

LinearShape shape_of(const LinearArgs& a, int size) {
  const int64_t sb = a.k / 32;
  auto on = [&](int64_t al) { return rows_aligned(a.a_s, sb, al) && rows_aligned(a.w_s, sb, al); };
  const bool pieces = rows_aligned(a.y, a.ld_y * size, 16) && a.n % (16 / size) == 0;
  return {a.rows, a.n, a.k, a.mats, a.offsets != nullptr, size, a.ld_y * size, pieces, on(16) ? 16 : on(4) ? 4 : 1, a.num_cus};
}

template <typename T, int SCALES, int MT, int NB, int NW>
hipError_t stream_v(const LinearArgs& a, const LinearShape& s, hipStream_t st) {
  const int64_t units = row_tiles_max(s, 16 * MT) * ((a.n + 16 * NB - 1) / (16 * NB));
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(units, (NW == 4 ? 8 : 2) * a.num_cus));
  // four columns of a row can be stored at once
  const bool wide = rows_aligned(a.y, a.ld_y * sizeof(T), 4 * sizeof(T));
  k_linear_stream<T, SCALES, MT, NB, NW><<<grid, 64 * NW, 0, st>>>(a, wide);
  return hipGetLastError();
}

template <typename T>
hipError_t stream_t(const LinearArgs& a, const LinearShape& s, const LinearChoice& c, hipStream_t st) {
  if (c.scales == 0) return c.waves == 8 ? stream_v<T, 0, 1, 1, 8>(a, s, st) : stream_v<T, 0, 1, 1, 4>(a, s, st);
  if (c.scales == 1) return c.waves == 8 ? stream_v<T, 1, 1, 1, 8>(a, s, st) : stream_v<T, 1, 1, 1, 4>(a, s, st);
  return c.mt == 4 ? stream_v<T, 2, 4, 2, 8>(a, s, st) : stream_v<T, 2, 1, 1, 4>(a, s, st);
}

template <typename T, int BM>
hipError_t tile_t(const LinearArgs& a, const LinearShape& s, const LinearChoice& c, hipStream_t st) {
  const int64_t tiles = row_tiles_max(s, BM) * ((a.n + kTileN - 1) / kTileN);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, a.num_cus));
  auto go = [&](auto k) {
    k<<<grid, kTileThreads, 0, st>>>(a);
    return hipGetLastError();
  };
  if constexpr (BM != 256 || sizeof(T) != 4)
    if (!c.wide) return go(k_linear_tile<T, BM, 0, false, false>);
  if constexpr (BM == 64) {
    if (c.scales == 4) return c.once ? go(k_linear_tile<T, BM, 4, true, true>) : go(k_linear_tile<T, BM, 4, true, false>);
    if (c.once) return c.scales ? go(k_linear_tile<T, BM, 2, true, true>) : go(k_linear_tile<T, BM, 0, true, true>);
  }
  return c.scales ? go(k_linear_tile<T, BM, 2, true, false>) : go(k_linear_tile<T, BM, 0, true, false>);
}

template <typename T>
hipError_t linear_t(const LinearArgs& a, hipStream_t st) {
  const LinearShape s = shape_of(a, sizeof(T));
  const LinearChoice c = choose_linear(s);
  if (c.bm == 0) return stream_t<T>(a, s, c, st);
  return c.bm == 64 ? tile_t<T, 64>(a, s, c, st) : c.bm == 128 ? tile_t<T, 128>(a, s, c, st) : tile_t<T, 256>(a, s, c, st);
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
