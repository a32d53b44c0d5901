// The tile kernel of the 16-bit products of rows sorted by expert, for the
// product itself and for both gradients:
//   kForward  y[r] = x[r] W_e^T         x [rows][k], W_e [n][k]
//   kInput    dx[r] = dy[r] W_e         dy [rows][n]
//   kWeight   dW_e = sum over e's rows of dy[r]^T x[r]
// e(r) is the matrix whose rows [offsets[e], offsets[e+1]) hold r, or the one
// matrix there is.  C [M x N] is computed in tiles of BM x 256; the sums run
// over L (k, n, or the rows of a matrix) in steps of 64, in fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "rows_choice.h"
#include "row_types.h"
#include "rows_device.h"

namespace mxmoe {
namespace rows {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;

template <typename T>
__device__ __forceinline__ v16f mfma32(v8s b, v8s a, v16f c) {
  if constexpr (std::is_same_v<T, bf16_t>) {
    typedef __bf16 v __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v, b), __builtin_bit_cast(v, a), c, 0, 0, 0);
  } else {
    typedef _Float16 v __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v, b), __builtin_bit_cast(v, a), c, 0, 0, 0);
  }
}

// prefix[e] = row tiles (of TM rows) of the matrices before e; one pass of the
// whole workgroup (part: a word of LDS per wave).  Returns the number of tiles.
template <int THREADS, int TM>
__device__ __forceinline__ int tile_prefix(const RowsArgs& a, int* prefix, int* part) {
  if (!a.offsets) {
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    return static_cast<int>((a.rows + TM - 1) / TM);
  }
  constexpr int PER = (kMaxRowMats + THREADS - 1) / THREADS;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    int lo = 0, hi = 0;
    if (e < a.mats) mat_rows(a.offsets, e, static_cast<int>(a.rows), lo, hi);
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

// Zeros in the rows of C that no matrix has, by all workgroups together; part:
// two words of LDS per wave.
template <int THREADS, typename TO>
__device__ __forceinline__ void zero_uncovered(const RowsArgs& a, int* part) {
  int lo, hi;
  covered_rows<THREADS>(a.offsets, a.mats, static_cast<int>(a.rows), lo, hi, part);
  const int none = lo + static_cast<int>(a.rows) - hi;
  TO* c = static_cast<TO*>(a.c);
  constexpr int PER = 16 / sizeof(TO);
  const bool pieces = rows_on_16(c, a.ld_c * sizeof(TO));
  for (int i = blockIdx.x; i < none; i += gridDim.x) {
    TO* row = c + (i < lo ? i : i - lo + hi) * a.ld_c;
    const int whole = pieces ? a.n / PER * PER : 0;
    for (int x = threadIdx.x * PER; x < whole; x += THREADS * PER) *reinterpret_cast<u32x4*>(row + x) = u32x4{0, 0, 0, 0};
    for (int x = whole + threadIdx.x; x < a.n; x += THREADS) row[x] = static_cast<TO>(0.0f);
  }
}

// Copy of 16 bytes per lane from the buffer's byte off to LDS byte lds + 16
// lane; a lane whose offset is past the buffer's end brings zeros.  Written as
// assembly (with no register output) so that the compiler does not wait for it
// at every later LDS read; the kernel counts its own copies.
__device__ __forceinline__ void copy16(uint32_t off, v4i rsrc, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(rsrc), "s"(lds)
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
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32));
  return uint64_t(hi) << 32 | lo;
}

template <int N>
__device__ __forceinline__ void wait_vm() {  // at most N vector-memory operations left
  static_assert(N >= 0 && N < 64, "vmcnt has six bits");
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

constexpr int kThreads = 256;
constexpr int kPanel = 4;                    // row tiles that share a column block's operand in time
constexpr uint32_t kNowhere = 0x80000000u;   // past the end of every buffer below

template <int BM, int SZ>
struct Shape {
  static constexpr int WM = BM == 64 ? 1 : 2, WN = 4 / WM;            // waves along rows, columns
  static constexpr int MI = BM / WM / 32, NI = kRowsTileN / WN / 32;  // 32-row, 32-column blocks of a wave
  static constexpr int S = BM == 256 ? 2 : 3;                         // ring slots
  static constexpr int A = 0, B = BM * 128, SLOT = B + kRowsTileN * 128;
  static constexpr int CA = BM / 32, CB = kRowsTileN / 32, C = CA + CB;  // copies of a wave and step
  // those issued in a step's last quarter, S - 1 steps ahead of their slot's
  // use: half of them with two slots (they have to land soon), else a quarter
  static constexpr int C0 = C / (S == 2 ? 2 : 4);
  static constexpr int STORES = MI * NI * SZ;  // a wave's stores of a tile (16 bytes a lane)
};

// One operand's side of a step.  Plain: 64 elements (128 bytes) of each of
// its W rows, the 16-byte chunk c of row r at chunk c ^ (r/2 % 8): the 16
// lanes that the LDS serves together (16 rows, one chunk) touch all 64 banks
// once.  With c ^ (r % 8) they touch half of them (304 against 584 bytes per
// ns and CU).  Transposed (its rows run along L): 64 rows of W elements, the
// 64-byte piece p of row r at p ^ (r % 4); ds_read_b64_tr_b16 gives lane i of
// 16 column i of four rows, of which lane j has read 8 bytes of row j/4.
template <bool TRANS, int W>
struct Side {
  static constexpr int RB = TRANS ? 2 * W : 128;   // bytes of a row in LDS
  static constexpr int RPC = 1024 / RB, LPR = 64 / RPC;  // rows of a copy, lanes of a row
  // where lane `lane` of the wave's copy `c` (counted over the workgroup) reads: row, chunk of 16 bytes
  static __device__ __forceinline__ void source(int c, int lane, int& row, int& chunk) {
    row = c * RPC + lane / LPR;
    chunk = TRANS ? (lane % LPR) ^ (4 * (row & 3)) : (lane & 7) ^ ((row >> 1) & 7);
  }
  // this lane's byte of column (row) block `blk` of 32, in the first quarter
  static __device__ __forceinline__ int frag(int blk, int lane) {
    if constexpr (TRANS) {
      const int i = lane & 15, s = i >> 2;
      return (8 * (lane >> 5) + s) * RB + ((blk ^ s) * 64) + 32 * ((lane >> 4) & 1) + 8 * (i & 3);
    } else {
      return (blk * 32 + (lane & 31)) * 128;
    }
  }
};

// One workgroup of four waves per CU walks its tiles of BM x 256; a step is 64
// of L, four quarters of 16.  A step's operands, 128 bytes for each of BM rows
// and 256 columns, come by direct-to-LDS copies into a ring of S slots, and the
// stream of steps runs on across the tiles: while a tile ends, the first steps
// of the next are already on their way.  In a quarter a wave issues its MI x NI
// MFMAs 32x32x16 and between them the LDS reads of the next quarter; before the
// last quarter it waits for its own copies of step s + 1 and at a barrier (all
// waves' copies have landed, and all have read slot s), and from there on the
// copies of step s + S go into slot s, spread over the following quarters so
// that the waves do not queue behind them.  What lies past an operand's end
// comes as zeros by the buffers' bounds: ragged ends of a matrix's rows (which
// are the sums' length for the weights' gradient), rows and columns of the last
// tiles, the end of L.  The columns' side is the first MFMA operand, so that
// four registers of a lane are four consecutive columns of C.
//
// TO: element type of C.  WIDE: N and the rows of C are whole numbers of
// 16-byte pieces.
//
// Measured (bf16, 256-row tiles, calls in a row on changing operands): 8192 x
// 4096, sums of 7168, forward 362 us (1.33 PF; short runs on the same operands
// 340 us), 8192^3 0.81, 0.80 and 0.78 ms for the three passes (1.37 to 1.41 PF); a
// library's product reaches 1.62, 1.39 and 1.21 PF for the three layouts of
// 8192^3, under the same power.  What bounds it first are the copies: the matrix
// cores idle 21 to 28 % of the cycles of 8192^3, and each of a step's 16 copies
// costs its wave about 30 cycles in which no MFMA is issued, next to 2048 cycles
// of MFMAs.  Without the copies (and with wrong results) it makes 1.68 PF, with
// half of them 1.53, with all of them from lines in L2 1.44, without the LDS
// reads 1.38.  Behind that stands the card's power, which holds the clock at 1.7
// GHz: these MFMAs alone, from registers, make 1.79 PF on normal numbers and 2.48
// on zeros.
// 32768 rows over 64 matrices of 4096 x 7168, uneven: forward 1.82 ms, dx 1.82
// ms, dW 2.06 ms, of which 0.68 ms are the stores of its 3.8 GB: with two slots
// half of a step's copies are issued behind the stores of the tile before, and
// the barrier that needs these copies waits for the stores too.
template <typename T, typename TO, Pass PASS, int BM, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) k_rows_tile(RowsArgs a) {
  constexpr bool TA = PASS == Pass::kWeight, TB = PASS != Pass::kForward;
  using P = Shape<BM, sizeof(TO)>;
  using SA = Side<TA, BM>;
  using SB = Side<TB, kRowsTileN>;
  constexpr int S = P::S, MI = P::MI, NI = P::NI;
  // A tile of 256 rows with 128 or fewer in it takes half the products: the
  // waves then share its columns alone, 128 x 64 each.  (For the weights'
  // gradient, whose rows are many, it gained nothing.)
  constexpr bool HALVES = BM == 256 && PASS != Pass::kWeight;
  // (of half a tile the last wave reads two blocks of columns past a plain side's eight, and leaves them)
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S * P::SLOT + (HALVES && !TB ? 2 * 32 * 128 : 0)];
  __shared__ int prefix[PASS == Pass::kWeight ? 1 : kMaxRowMats];
  const int lane = threadIdx.x & 63, wave = uniform(static_cast<int>(threadIdx.x >> 6));
  const int l32 = lane & 31, g32 = lane >> 5;
  const int wm = wave / P::WN, wn = wave % P::WN;
  const int ntn = (a.n + kRowsTileN - 1) / kRowsTileN;
  // row tiles in all; the weights' gradient has the same number for each matrix
  const int mt1 = PASS == Pass::kWeight ? (a.m + BM - 1) / BM : 0;
  const int mtiles = PASS == Pass::kWeight ? a.mats * mt1
                                           : uniform(tile_prefix<kThreads, BM>(a, prefix, reinterpret_cast<int*>(lds)));
  // (the caller has seen to it that the tiles stay below the limit: only
  // ranges that overlap, many times over, can have more)
  const int per_slice = min(mtiles, static_cast<int>(kMaxRowTiles / a.slices) / ntn) * ntn;
  const int tiles = per_slice * a.slices;

  // ---- which tiles are this workgroup's: runs of gridDim/8 consecutive
  // tiles go to one XCD (workgroups go to the XCDs round-robin), so that the
  // tiles that share rows or weights share an L2; few tiles are spread
  const int G = gridDim.x, b = blockIdx.x;
  // If the last round of tiles would keep half of the workgroups busy at most,
  // its tiles go to two workgroups each (8192 x 7168, sums of 4096, 3.5 rounds:
  // 368 against 392 us)
  const int rest = tiles % G;
  const bool split = HALVES && 2 * rest <= G;
  const int whole = split ? tiles - rest : tiles, total = split ? tiles + rest : tiles;
  const bool by_xcd = G % 8 == 0 && total > G;
  const int first = by_xcd ? (b & 7) * (G / 8) + (b >> 3) : b;

  struct TileAt {
    int e, slice;
    int row0, rows;   // kWeight: first row of C and how many
    int lo;           // kWeight: first row of the matrix
    int col0;
    int step0, steps, l;  // steps of 64 along L, its length
  };
  // tile `pos` of the list: slice by slice, matrix by matrix, panels of kPanel
  // row tiles, in a panel column block by column block
  auto tile_at = [&](int pos) -> TileAt {
    TileAt t;
    int part = -1;  // of a tile that two workgroups share
    if (pos >= whole) {
      part = (pos - whole) & 1;
      pos = whole + (pos - whole) / 2;
    }
    t.slice = 0;
    if (a.slices > 1) {
      t.slice = uniform(static_cast<int>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(per_slice)));
      pos -= t.slice * per_slice;
    }
    const int q = uniform(static_cast<int>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(ntn)));
    int p0, p1;
    if constexpr (PASS == Pass::kWeight) {
      t.e = uniform(static_cast<int>(static_cast<uint32_t>(q) / static_cast<uint32_t>(mt1)));
      p0 = t.e * mt1;
      p1 = p0 + mt1;
    } else {
      t.e = tile_matrix(prefix, a.mats, q);
      p0 = uniform(prefix[t.e]);
      p1 = t.e + 1 < a.mats ? uniform(prefix[t.e + 1]) : mtiles;
    }
    const uint32_t local = pos - p0 * ntn, pn = kPanel * ntn;
    const int panel = uniform(static_cast<int>(local / pn)), within = local - panel * pn;
    const int gm = min(kPanel, p1 - p0 - panel * kPanel);
    const int nt = uniform(static_cast<int>(static_cast<uint32_t>(within) / static_cast<uint32_t>(gm)));
    const int mt = panel * kPanel + within - nt * gm;
    int lo = 0, hi = static_cast<int>(a.rows);
    if (a.offsets) {
      sload2(a.offsets + t.e, lo, hi);
      clamp_rows(static_cast<int>(a.rows), lo, hi);
    }
    t.col0 = nt * kRowsTileN;
    if constexpr (PASS == Pass::kWeight) {
      t.row0 = mt * BM;
      t.rows = min(BM, a.m - t.row0);
      t.lo = lo;
      t.l = hi - lo;
    } else {
      t.row0 = lo + mt * BM;
      t.rows = min(BM, hi - t.row0);
      t.lo = 0;
      t.l = a.l;
    }
    if (part >= 0) {
      t.row0 += 128 * part;
      t.rows = min(128, t.rows - 128 * part);  // (none left: nothing is stored)
    }
    // (a tile without products has one step, of zeros)
    const int all = (t.l + 63) / 64, each = a.slices > 1 ? (all + a.slices - 1) / a.slices : all;
    t.step0 = t.slice * each;
    t.steps = uniform(max(1, min(each, all - t.step0)));
    return t;
  };

  // ---- issue side
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)lds));
  int iss_pos = first, iss_tile = 0, iss_left = 0, iss_rem = 0, iss_slot = 0;
  // What the other side will ask of a tile, the workgroup's n-th, in the lanes
  // of one register: it is one or two tiles behind, and there are not enough
  // scalar registers for so many tiles.
  enum { kRow0, kRows, kCol0, kMat, kSlice, kSteps };
  int tiles_at = 0;
  auto get = [&](int n, int field) { return __builtin_amdgcn_readlane(tiles_at, (n & 3) * 8 + field); };
  uint64_t ia = 0, ib = 0;          // the step's first byte of each side
  v4i ra, rb;                       // and their buffers
  uint32_t oa[P::CA], ob[P::CB];
  uint32_t out[2] = {0, 0};         // set in offsets past the end of L (plain sides)
  const int ld2a = static_cast<int>(a.ld_a) * 2, ld2b = static_cast<int>(a.ld_b) * 2;
  const int64_t adv_a = TA ? int64_t(ld2a) * 64 : 128, adv_b = TB ? int64_t(ld2b) * 64 : 128;
  // (the copies of a wave begin at an even one, so a plain side's chunks alternate between two)
  static_assert(P::CA % 2 == 0 && P::CB % 2 == 0, "");
  const int chunk0 = (lane & 7) ^ ((lane >> 4) & 7);
  auto buffers = [&] {
    const int r = uniform(min(max(iss_rem, 0), 64));
    ra = v4i{uniform(static_cast<int>(ia)), uniform(static_cast<int>(ia >> 32)), TA ? uniform(r * ld2a) : static_cast<int>(kNowhere), 0x00027000};
    rb = v4i{uniform(static_cast<int>(ib)), uniform(static_cast<int>(ib >> 32)), TB ? uniform(r * ld2b) : static_cast<int>(kNowhere), 0x00027000};
    if constexpr (!TA || !TB) {
      out[0] = 8 * chunk0 >= iss_rem ? kNowhere : 0;
      out[1] = 8 * (chunk0 ^ 4) >= iss_rem ? kNowhere : 0;
    }
  };
  auto iss_setup = [&](const TileAt& t) {
    const T* pa = static_cast<const T*>(a.a);
    const T* pb = static_cast<const T*>(a.b);
    const int l0 = t.step0 * 64;
    if constexpr (PASS == Pass::kWeight) {
      ia = uniform(pa + (int64_t(t.lo) + l0) * a.ld_a + t.row0);
      ib = uniform(pb + (int64_t(t.lo) + l0) * a.ld_b + t.col0);
    } else {
      ia = uniform(pa + t.row0 * a.ld_a + l0);
      ib = uniform(pb + t.e * a.mat_b + (PASS == Pass::kForward ? t.col0 * a.ld_b + l0 : l0 * a.ld_b + t.col0));
    }
    iss_left = t.steps;
    const int n = iss_tile++;
    auto put = [&](int field, int v) { tiles_at = lane == (n & 3) * 8 + field ? v : tiles_at; };
    put(kRow0, t.row0);
    put(kRows, t.rows);
    put(kCol0, t.col0);
    put(kMat, t.e);
    put(kSlice, t.slice);
    put(kSteps, t.steps);
    iss_rem = t.l - l0;
    const int cols = a.n - t.col0;
#pragma unroll
    for (int q = 0; q < P::CA; ++q) {
      int row, chunk;
      SA::source(P::CA * wave + q, lane, row, chunk);
      // (rows that are not there come as zeros, which cost the matrix cores the least power)
      oa[q] = (TA ? 8 * chunk : row) < t.rows ? row * ld2a + 16 * chunk : kNowhere;
    }
#pragma unroll
    for (int q = 0; q < P::CB; ++q) {
      int row, chunk;
      SB::source(P::CB * wave + q, lane, row, chunk);
      ob[q] = (TB ? 8 * chunk : row) < cols ? row * ld2b + 16 * chunk : kNowhere;
    }
    buffers();
  };
  // (total and G are at most 2^30: no overflow)
  auto next_pos = [&](int pos) { return pos + G; };
  // copy number m of the step at the issue side
  auto issue = [&](auto mc) {
    constexpr int m = decltype(mc)::value;
    const uint32_t slot = lds0 + iss_slot * P::SLOT;
    if constexpr (m < P::CA) copy16(TA ? oa[m] : oa[m] | out[m % 2], ra, slot + P::A + (P::CA * wave + m) * 1024);
    else copy16(TB ? ob[m - P::CA] : ob[m - P::CA] | out[m % 2], rb, slot + P::B + (P::CB * wave + m - P::CA) * 1024);
  };
  // to the next step; behind the last tile the last one is copied again, into
  // slots that are not read
  auto advance = [&] {
    iss_slot = iss_slot + 1 == S ? 0 : iss_slot + 1;
    if (--iss_left == 0) {
      if (next_pos(iss_pos) < total) iss_pos = next_pos(iss_pos);
      iss_setup(tile_at(iss_pos));
    } else {
      ia += adv_a;
      ib += adv_b;
      iss_rem -= 64;
      buffers();
    }
  };

  // ---- read side: byte offsets in a slot of this lane's fragments
  int fa[TA ? MI : 1], fb[TB ? NI : 1];
  auto set_frags = [&](bool half) {
    const int a0 = half ? 0 : wm * MI, b0 = half ? wave * (NI / 2) : wn * NI;
#pragma unroll
    for (int i = 0; i < (TA ? MI : 1); ++i) fa[i] = P::A + SA::frag(a0 + i, lane);
    // (of half a tile only the first NI/2 are taken)
#pragma unroll
    for (int j = 0; j < (TB ? NI : 1); ++j) fb[j] = P::B + SB::frag((b0 + j) % (kRowsTileN / 32), lane);
  };
  // plain: quarter h of a step is chunks 2h and 2h + 1
  const int sw = (l32 >> 1) & 7;
  const int ch[4] = {16 * (g32 ^ sw), 16 * ((2 + g32) ^ sw), 16 * ((4 + g32) ^ sw), 16 * ((6 + g32) ^ sw)};
  v8s av[2][MI], bv[2][NI];  // the fragments of this quarter and of the next
  auto read_t = [&](const uint8_t* p, int rb) -> v8s {
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
    const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * rb));
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto read_frag = [&](int slot, auto hc, auto jc) {
    constexpr int H = decltype(hc)::value, j = decltype(jc)::value;
    uint8_t* p = lds + slot * P::SLOT;
    if constexpr (j < NI) {
      if constexpr (TB) bv[H % 2][j] = read_t(p + fb[j] + H * 16 * SB::RB, SB::RB);
      else bv[H % 2][j] = *reinterpret_cast<const v8s*>(p + fb[0] + ch[H] + j * 4096);
    } else {
      constexpr int i = j - NI;
      if constexpr (TA) av[H % 2][i] = read_t(p + fa[i] + H * 16 * SA::RB, SA::RB);
      else av[H % 2][i] = *reinterpret_cast<const v8s*>(p + fa[0] + ch[H] + i * 4096);
    }
  };

  int slot = 0;
  // One step of four quarters.  FIRST: the tile's first, its products start
  // from zero.  after_stores: the last tile's stores may still be on their way
  // (operations finish in the order in which they were issued).
  // acc: the sums, MI x NI blocks or half as many.  last: the last of tile n.
  auto step = [&](auto first_c, auto& acc, bool after_stores, bool last, int n) {
    constexpr bool FIRST = decltype(first_c)::value != 0;
    constexpr int NE = sizeof(acc[0]) / sizeof(v16f), NM = MI * NE;
    // The products so far stay before this point (without it the compiler moves
    // them past the branches below, to where the sums are next used).
    auto settle = [&] {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NE; ++j) asm volatile("" : "+a"(acc[i][j]));
    };
    const int nslot = slot + 1 == S ? 0 : slot + 1;
    // the copies of step s + S - 1, begun in the last quarter of step s - 1,
    // go on over the quarters before the barrier (with two slots: the first)
    constexpr int QI = S == 2 ? 1 : 3;
    unrolled<0, 4>([&](auto qc) {
      constexpr int q = decltype(qc)::value;
      constexpr bool LAST = q == 3;
      if constexpr (q == QI) {
        settle();
        advance();
      }
      if constexpr (LAST) {
        settle();
        wait_lds();
        // outstanding: the copies of steps s + 1 .. s + S - 1, of which
        // s + 1's have to be done (with more than two slots all of them were
        // issued before the stores)
        constexpr int left = P::C * (S - 2);
        if (S > 2 && after_stores) wait_vm<(left + P::STORES < 63 ? left + P::STORES : 63)>();
        else wait_vm<left>();
        tile_barrier();
        if constexpr (HALVES)
          if (last) set_frags(get(n + 1, kRows) <= 128);
      }
      unrolled<0, NM>([&](auto kc) {
        constexpr int k = decltype(kc)::value, i = k / NE, j = k % NE;
        acc[i][j] = mfma32<T>(bv[q % 2][j], av[q % 2][i], FIRST && q == 0 ? v16f{} : acc[i][j]);
        // the next quarter's reads, in the first three quarters of this one
        constexpr int R = MI + NI, lo = k * R / (NM * 3 / 4), hi = (k + 1) * R / (NM * 3 / 4);
        unrolled<(lo < R ? lo : R), (hi < R ? hi : R)>(
            [&](auto jc) { read_frag(LAST ? nslot : slot, Int<LAST ? 0 : q + 1>{}, jc); });
        if constexpr (q < QI) {
          constexpr int n = NM * QI, x = q * NM + k;
          unrolled<P::C0 + x * (P::C - P::C0) / n, P::C0 + (x + 1) * (P::C - P::C0) / n>([&](auto mc) { issue(mc); });
        }
        if constexpr (LAST) unrolled<k * P::C0 / NM, (k + 1) * P::C0 / NM>([&](auto mc) { issue(mc); });
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    settle();
    slot = nslot;
  };

  // ---- results: acc[i][j] of this wave; lane (l32, g32) register r is column
  // 8(r/4) + 4 g32 + r%4 of row l32 of the block.  WIDE: buffer stores with
  // the tile's first row as base: a lane whose row or columns are not there
  // takes an offset past the buffer's end and stores nothing, so there are no
  // branches (which would cost copies of the accumulators).  Otherwise the
  // same 16-byte pieces at any address, and only a row's last one by elements.
  auto store_tile = [&](int n, auto& acc) {
    constexpr int NE = sizeof(acc[0]) / sizeof(v16f);
    constexpr bool HALF = NE < NI;
    constexpr int SZ = sizeof(TO), PER = 16 / SZ;
    const int rows = get(n, kRows), col0 = get(n, kCol0), cols = a.n - col0;
    const uint64_t base = uniform(static_cast<TO*>(a.c) + get(n, kSlice) * a.slice_c +
                                  (PASS == Pass::kWeight ? get(n, kMat) * a.mat_c : 0) + get(n, kRow0) * a.ld_c + col0);
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, kNowhere, 0x00027000);
    const uint32_t ld = static_cast<uint32_t>(a.ld_c) * SZ;
    // the last MFMA's results take 16 passes (18 wait states); the compiler
    // counts them for its own reads, not for the assembly's below
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    // this lane's rows: with 16-bit results lane l stores rows l%16 and
    // 16 + l%16 of each block of 32, otherwise row l%32
    constexpr bool ROWS16 = SZ == 2;
    constexpr int NR = ROWS16 ? 2 : 1;
    uint32_t at[MI][NR];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int h = 0; h < NR; ++h) {
        const int row = ((HALF ? 0 : wm * MI) + i) * 32 + (ROWS16 ? 16 * h + (lane & 15) : l32);
        at[i][h] = row < rows ? row * ld : kNowhere;
      }
    unrolled<0, MI * NE>([&](auto bc) {
      constexpr int i = decltype(bc)::value / NE, j = decltype(bc)::value % NE;
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
      const int col = (HALF ? wave * NE + j : wn * NI + j) * 32;
      if constexpr (ROWS16) {
        // lane (l32, g32) has columns 8q + 4 g32 .. + 3 of row l32, q = 0..3.
        // Lanes l and l + 32 exchange halves, and it has 8 columns (16 bytes),
        // 16p + 8 g32 .., p = 0, 1; then the 16-lane rows of the wave do, and
        // four lanes have the 64 bytes of a row of the block.
        uint32_t v[2][4];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const auto e = __builtin_amdgcn_permlane32_swap(pack2<TO>(c(8 * p + 2 * x), c(8 * p + 2 * x + 1)),
                                                            pack2<TO>(c(8 * p + 4 + 2 * x), c(8 * p + 5 + 2 * x)), false, false);
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

  if (first < total) {
    // ---- the stream of steps: the first S - 1 and the first part of the next
    // are on their way before the first product
    iss_setup(tile_at(first));
    unrolled<0, S - 1>([&](auto) {
      unrolled<0, P::C>([&](auto mc) { issue(mc); });
      advance();
    });
    unrolled<0, P::C0>([&](auto mc) { issue(mc); });
    set_frags(HALVES && get(0, kRows) <= 128);
    wait_vm<P::C*(S - 2) + P::C0>();
    tile_barrier();
    unrolled<0, MI + NI>([&](auto jc) { read_frag(0, Int<0>{}, jc); });

    bool stored = false;
    int n = 0;
    for (int pos = first; pos < total; pos = next_pos(pos), ++n) {
      // without WIDE the number of stores is not known here: wait for all
      if (!WIDE && stored) wait_vm<0>();
      stored &= WIDE;
      auto run = [&](auto ne) {
        v16f acc[MI][decltype(ne)::value];
        int left = get(n, kSteps) - 1;
        step(Int<1>{}, acc, stored, left == 0, n);
        while (left > 0) step(Int<0>{}, acc, false, --left == 0, n);
        store_tile(n, acc);
      };
      if (HALVES && get(n, kRows) <= 128) run(Int<HALVES ? NI / 2 : NI>{});
      else run(Int<NI>{});
      stored = true;
    }
    // the copies still on their way land in this workgroup's LDS
    wait_vm<0>();
  }

  // ---- rows of no matrix are zero (of partial sums the joining kernel does it)
  if constexpr (PASS != Pass::kWeight) {
    if (!a.offsets || a.slices > 1) return;
    __syncthreads();  // all waves are done with the LDS
    zero_uncovered<kThreads, TO>(a, reinterpret_cast<int*>(lds));
  }
}

template <typename T, typename TO, Pass PASS, int BM>
hipError_t launch_tile_bm(const RowsArgs& a, bool wide, int64_t tiles, hipStream_t st) {
  const unsigned grid = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(tiles, a.num_cus)));
  if (wide) k_rows_tile<T, TO, PASS, BM, true><<<grid, kThreads, 0, st>>>(a);
  else if constexpr (sizeof(TO) == 2) k_rows_tile<T, TO, PASS, BM, false><<<grid, kThreads, 0, st>>>(a);
  else return hipErrorInvalidValue;  // (partial sums and fp32 gradients are laid out on 16 bytes)
  return hipGetLastError();
}

template <typename T, typename TO, Pass PASS>
hipError_t launch_tile(const RowsArgs& a, const RowsChoice& c, hipStream_t st) {
  if constexpr (PASS != Pass::kWeight)  // (a transposed side of 64 columns has no four pieces to exchange)
    if (c.bm == 64) return launch_tile_bm<T, TO, PASS, 64>(a, c.wide, c.tiles, st);
  return c.bm == 128 ? launch_tile_bm<T, TO, PASS, 128>(a, c.wide, c.tiles, st) : launch_tile_bm<T, TO, PASS, 256>(a, c.wide, c.tiles, st);
}

template <Pass PASS>
hipError_t launch_pass(const RowsArgs& a, const RowsChoice& c, RowType in, RowType out, hipStream_t st) {
  if (in == RowType::kBf16) return out == RowType::kFp32 ? launch_tile<bf16_t, float, PASS>(a, c, st) : launch_tile<bf16_t, bf16_t, PASS>(a, c, st);
  return out == RowType::kFp32 ? launch_tile<_Float16, float, PASS>(a, c, st) : launch_tile<_Float16, _Float16, PASS>(a, c, st);
}

}  // namespace rows
}  // namespace mxmoe
