// Internal interface between the C-ABI layer (api.cpp) and the HIP kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace mxmoe {

// One unit of grouped-GEMM work: rows [row_begin, row_end) of expert `ex`
// (ex < E: routed expert; ex >= E: shared expert ex - E).
struct Tile {
  int32_t ex, row_begin, row_end, pad;
};

// Everything the kernels of one forward need; all pointers are device memory.
struct FwdArgs {
  // shape
  int T, d, dff, E, k, S;
  int R;         // permuted rows: T*k routed + S*T shared
  int Rr;        // routed rows T*k
  // inputs
  const uint16_t* x;    // bf16 [T][d]
  const float* wr;      // [E][d]
  const float* br;      // [E] or null
  const uint8_t *gu_c, *gu_s, *dn_c, *dn_s;      // routed weights
  const uint8_t *sgu_c, *sgu_s, *sdn_c, *sdn_s;  // shared weights
  // outputs
  uint16_t* y;  // bf16 [T][d]
  // workspace buffers (or caller taps substituted for them)
  float* logits;        // [T][E]
  float* router_part;   // [router_ks][T][E] split-K partial logits (router_ks > 1)
  int32_t* topk_ids;    // [T][k]
  float* topk_w;        // [T][k]
  uint8_t* x_codes;     // [T][d]
  uint8_t* x_scales;    // [T][d/32]
  int32_t* counts;      // [E]
  int32_t* offsets;     // [E+1]
  int32_t* row_src;     // [Rr]   pair index
  int32_t* row_token;   // [Rr]   token of each routed row
  int32_t* token_row;   // [T][k]
  uint64_t* chunk_mask; // [nchunks][E]
  int32_t* chunk_base;  // [E][nchunks]
  Tile* tiles;          // [max_tiles], grouped by expert (routed ascending, then shared)
  int32_t* tile_count;  // [1]
  int32_t* ex_tiles;    // [E+S+1] first tile of each expert (prefix over tile counts)
  uint8_t* h_codes;     // [R][dff]
  uint8_t* h_scales;    // [R][dff/32]
  uint16_t* h16;        // [R][dff] bf16 h (A16W4 variant), else unused
  int a16;              // 1: A16W4 variant (bf16 x and h, no MXFP8 activations)
  uint16_t* o16;        // [R][d] bf16 down outputs: permuted-row order after the
                        // decode kernels, (token, slot) order after the prefill ones
  // optional taps (null = skip)
  float* gu_acc;        // [R][2*dff]
  float* y_routed;      // [T][d]
  float* y_shared;      // [T][d]
  // launch-time choices
  int router_ks;        // K slices of the MFMA router (1: no partials)
  int bm;               // rows per tile: 8 (decode kernels) or 256 (prefill kernels)
  int num_cus;          // compute units of the device (persistent decode grid)
  int max_tiles;
  int nchunks;          // 64-token chunks
  // the prefill down GEMM's K split (LatentMoE tail only): > 1 cuts K into
  // ksplit equal slices (multiples of 512) and writes fp32 partials
  // kpart[slice][R][d] in row order instead of bf16 o rows
  int ksplit;
  float* kpart;
  // 1: expert weights in the canonical layout ([N][K/2] codes, [N][K/32]
  // scales) instead of the packed one
  int wcanon;
};

// Everything the kernels of one LatentMoE tail call need (device pointers).
struct TailArgs {
  int T, latent, hidden, bm;
  float eps;
  const float* z;        // [T][latent] routed experts' weighted sum
  const float* gamma;    // [latent]
  const float* s;        // [T][hidden] shared experts' output, or null
  const uint8_t *up_c, *up_s;  // MXFP4 W_up [hidden][latent], packed or canonical
  int wcanon;                  // 1: canonical layout
  uint16_t* y;           // bf16 [T][hidden]
  uint8_t* codes;        // [T][latent] MXFP8 of the normalised rows
  uint8_t* scales;       // [T][latent/32]
  float* inv_rms;        // [T] tap, or null
  uint16_t* o16;         // [T][hidden] projection (y itself when s is null)
  int32_t* row_src;      // [T] identity
  Tile* tiles;           // [ceil(T/bm)]
  int32_t* tile_count;   // [1]
  int32_t* ex_tiles;     // [2]
  float* part;           // [slices][T][hidden] split-K partials (T <= kTailGemvMaxT)
};

// The tail's projection for at most kTailGemvMaxT rows runs split along K:
// each wave takes at most kTailGemvSteps of the 128-wide K steps.
constexpr int kTailGemvMaxT = 16;
constexpr int kTailGemvSteps = 4;
inline int tail_gemv_slices(int latent) {
  const int ns = latent / 128;
  return (ns + 4 * kTailGemvSteps - 1) / (4 * kTailGemvSteps);
}

// Rows per tile of the decode (weight-streaming) kernels; larger tiles go to
// the prefill kernels.
constexpr int kDecodeMaxRows = 8;

// Rows per tile of the LatentMoE tail's projection: the weight-streaming
// kernel for a few rows; from 24 rows on the prefill kernel, on 64-row tiles
// up to 512 rows (more tiles per column block, so fewer K slices and fp32
// partials are needed to fill the chip) and 256-row tiles above.
inline int tail_tile_rows(int64_t T) { return T < 24 ? kDecodeMaxRows : T <= 512 ? 64 : 256; }
// K slices of the tail's projection on those tiles, when its tiles x
// 256-column blocks alone would give fewer workgroups than three quarters of
// the 256 CUs: the smallest divisor of latent/512 (at most 8) that reaches
// 192 workgroups, else the largest.  Each slice adds one fp32 partial of the
// output, summed in order (with s) by the tail's reduction.
inline int tail_ksplit(int64_t T, int64_t latent, int64_t hidden, int64_t bm) {
  if (T < 24 || latent % 512 != 0) return 1;
  const int64_t base = ((T + bm - 1) / bm) * ((hidden + 255) / 256);
  const int64_t g = latent / 512;
  int best = 1;
  for (int d = 1; d <= 8 && d <= g; ++d) {
    if (g % d != 0) continue;
    best = d;
    if (base * d >= 192) break;
  }
  return best;
}

// Launchers (kernels_*.hip).  Each returns hipSuccess or the launch error.
hipError_t launch_tail(const TailArgs& a, int num_cus, hipStream_t st);
hipError_t launch_quantize(const void* src, int src_fp32, int64_t rows, int64_t cols, int64_t ld,
                           uint8_t* codes, uint8_t* scales, hipStream_t st);

// Tokens up to which the per-expert GEMV router (with the x quantisation
// fused) runs; above it, the bf16 MFMA router.
constexpr int kRouterSmallMaxT = 32;
inline bool router_small(int64_t T, int64_t d, int64_t E) { return T <= kRouterSmallMaxT && T * (d / 32) <= 32 * E; }

// K slices of the MFMA router for T tokens: few 128x128 output tiles are
// spread over the GPU by cutting d into up to 16 slices of at least 512.
inline int router_splits(int64_t T, int64_t E, int64_t d) {
  const int64_t tiles = ((T + 127) / 128) * ((E + 127) / 128);
  if (tiles >= 256) return 1;
  int64_t ks = (256 + tiles - 1) / tiles;
  if (ks > d / 512) ks = d / 512;
  if (ks > 16) ks = 16;
  return ks < 1 ? 1 : static_cast<int>(ks);
}

// The few-token forward splits its gate_up in two launches (top-k +
// permutation + shared experts, then the routed experts) when routing runs in
// one workgroup and every tile is a weight-streaming one, with the K split.
inline bool stream_split_phases(const FwdArgs& a) {
  return router_small(a.T, a.d, a.E) && a.bm <= kDecodeMaxRows && a.S > 0;
}

hipError_t launch_router_bias_update(const int32_t* offsets, int E, int64_t tk, float rate, float* b,
                                     hipStream_t st);
hipError_t launch_router(const FwdArgs& a, hipStream_t st);
hipError_t launch_topk_shared_gate_up(const FwdArgs& a, hipStream_t st);
hipError_t launch_topk_quant(const FwdArgs& a, hipStream_t st);
hipError_t launch_permute(const FwdArgs& a, hipStream_t st);
hipError_t launch_gemm_gate_up(const FwdArgs& a, hipStream_t st);
hipError_t launch_gemm_down(const FwdArgs& a, hipStream_t st);
hipError_t launch_combine(const FwdArgs& a, hipStream_t st);
hipError_t launch_pack_mx4(const uint8_t* codes, const uint8_t* scales, int64_t mats, int64_t rows,
                           int64_t k, int interleave, uint8_t* codes_p, uint8_t* scales_p, hipStream_t st);

// ---- the standalone pieces: MXFP4 conversion and product, token order

// element types of rows (row_types.h has their arithmetic)
enum class RowType { kBf16, kFp16, kFp32 };

hipError_t launch_quantize_mx4(const void* src, RowType dt, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                               uint8_t* scales, hipStream_t st);
hipError_t launch_dequantize_mx4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* dst,
                                 RowType dt, int64_t ld, hipStream_t st);

// y[r] = A[r] W[e(r)]^T, both MXFP4 in canonical layout (all device pointers)
struct LinearArgs {
  const uint8_t *a_c, *a_s;  // [rows][k/2], [rows][k/32]
  const uint8_t *w_c, *w_s;  // [mats][n][k/2], [mats][n][k/32]
  const int* offsets;        // [mats+1] first row of each matrix, or null: all rows to one matrix
  int64_t rows;
  int mats, n, k;
  void* y;                   // [rows][ld_y]
  int64_t ld_y;
  int num_cus;
};
hipError_t launch_linear_mx4(const LinearArgs& a, RowType dt, hipStream_t st);
// Output tiles that a launch counts to, and how many a product may have: in
// tiles of 64 rows (the lowest) x 256 columns, one more per matrix for its end.
constexpr int64_t kMaxLinearTiles = int64_t(1) << 30;
inline int64_t linear_tiles_max(int64_t rows, int64_t mats, int64_t n) { return ((rows + 63) / 64 + mats) * ((n + 255) / 256); }

// pairs sorted by one workgroup in one launch
constexpr int kSortSmallPairs = 4096;
// pairs per workgroup above that: at most kSortSmallPairs, and half of them
// while that fills the chip better
inline int sort_chunk(int64_t pairs) { return pairs <= (int64_t(1) << 20) ? kSortSmallPairs / 2 : kSortSmallPairs; }
// chunks up to which every ranking workgroup sums all chunks' counts itself
constexpr int kSortFusedChunks = 128;
hipError_t launch_sort_tokens(const void* ids, bool ids64, int64_t pairs, int E, int* offsets, int* row_src,
                              int* token_row, int* counts, hipStream_t st);
hipError_t launch_dispatch_rows(const void* x, int64_t row_bytes, int64_t ld_x, const int* token_row, int64_t T, int k,
                                int64_t R, const int* num_rows, void* out, int64_t ld_out, hipStream_t st);

struct CombineArgs {
  int64_t T, R, d;           // tokens, rows that there are, columns
  int k;
  const void* rows;          // [R][ld]
  int64_t ld;
  const int* token_row;      // [T][k]
  const float* w;            // [T][k], or null: ones
  void* y;                   // forward: [T][ld_y]
  const void* dy;            // backward: [T][ld_y]
  int64_t ld_y;
  void* drows;               // backward: [R][ld_d], or null
  int64_t ld_d;
  float* dw;                 // backward: [T][k], or null
  const int* num_rows;       // backward: first row of drows to zero-fill, or null
};
hipError_t launch_combine_rows(const CombineArgs& a, RowType dt, hipStream_t st);
hipError_t launch_combine_rows_backward(const CombineArgs& a, RowType dt, hipStream_t st);

// ---- 16-bit products of rows sorted by expert (rows_choice.h, rows_tile.h)
namespace rows {
enum class Pass;
struct RowsChoice;

struct RowsArgs {
  const void* a;             // the side of C's rows: x [rows][ld_a], dy [rows][ld_a]
  int64_t ld_a;
  const void* b;             // the side of C's columns: W [mats][mat_b], its rows ld_b apart, or x [rows][ld_b]
  int64_t ld_b, mat_b;
  const int* offsets;        // [mats+1] first row of each matrix, or null: all rows to one matrix
  int64_t rows;
  int mats;
  int m, n, l;               // C's rows (weights' gradient), its columns, the length of the sums (else)
  void* c;                   // [rows][ld_c], or [mats][mat_c] with rows of ld_c; slice s from s * slice_c on
  int64_t ld_c, mat_c, slice_c;
  int slices;
  int num_cus;
};
// for few products, operands and their rows anywhere
hipError_t launch_stream(const RowsArgs& a, const RowsChoice& c, RowType in, hipStream_t st);
// both operands on 16 bytes with rows on 16 bytes, what they hold between a
// row's end and its next 16 bytes zero
hipError_t launch_forward(const RowsArgs& a, const RowsChoice& c, RowType in, RowType out, hipStream_t st);
hipError_t launch_input(const RowsArgs& a, const RowsChoice& c, RowType in, RowType out, hipStream_t st);
hipError_t launch_weight(const RowsArgs& a, const RowsChoice& c, RowType in, RowType out, hipStream_t st);

// dst [rows][ld_dst] = src [rows][ld_src] (16-bit elements), zeros from cols to
// ld_dst, for at most three matrices
struct PadMatrix {
  const void* src;
  int64_t rows, cols, ld_src;
  void* dst;
  int64_t ld_dst;
};
constexpr int kMaxPads = 3;
hipError_t launch_pad_rows(const PadMatrix* m, int count, hipStream_t st);
// out[r] = sum of the slices' row r, rounded once; with offsets, rows of no matrix are zero
hipError_t launch_join(const float* part, int slices, int64_t rows, int64_t cols, int64_t ld, const int* offsets, int mats,
                       void* out, RowType out_t, int64_t ld_out, hipStream_t st);
}  // namespace rows

// ---- activations in 8 bits, the gated activation
hipError_t launch_quantize_mx8(const void* src, RowType dt, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                               uint8_t* scales, hipStream_t st);
// pad (cols <= pad < cols + 8) columns of dst are written, zeros from cols on
hipError_t launch_dequantize_mx8(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* dst,
                                 RowType dt, int64_t ld, int64_t pad, hipStream_t st);
// forward (dh null): a from h, and codes of h where they are given; backward:
// dh, and a where it is given, from da and h, or from its codes
struct SwigluArgs {
  int64_t rows, f;
  const void* h;
  int64_t ld_h;
  void* a;
  int64_t ld_a;
  uint8_t *codes, *scales;
  const void* da;
  int64_t ld_da;
  void* dh;
  int64_t ld_dh;
};
hipError_t launch_swiglu(const SwigluArgs& s, RowType dt, hipStream_t st);

// bytes of one packed scale matrix [rows/16][ceil(k/512)][64][4]
__host__ __device__ inline int64_t packed_scale_bytes(int64_t rows, int64_t k) { return rows * (k / 32); }

// token counts at or below which the single-workgroup permutation is used
constexpr int kPermSmallMaxTokens = 1024;

}  // namespace mxmoe
