// Which kernel a 16-bit product of rows sorted by expert takes, and what its
// workspace holds: the rules alone, plain host code without a device.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace mxmoe {
namespace rows {

// y = x W^T; dx = dy W; dW = dy^T x
enum class Pass { kForward, kInput, kWeight };

constexpr int kMaxRowMats = 1024;
constexpr int kRowsTileN = 256;  // columns of a tile
// Output tiles that a launch counts to, and how many a product may have: in
// tiles of 64 rows (the lowest) x 256 columns, one more per matrix for its end.
constexpr int64_t kMaxRowTiles = int64_t(1) << 30;
constexpr int kCus = 256;        // compute units that the estimates below count with
constexpr int kMaxSlices = 64;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round8(int64_t v) { return (v + 7) & ~int64_t(7); }

// The product as the tile kernel sees it: C [m x n], sums over l
struct RowsShape {
  Pass pass;
  int64_t rows, n, k;   // of the operator: rows, W [mats][n][k]
  int mats;
  bool grouped;         // rows go to the matrices by offsets, else all to the one
  int out_size;         // bytes of an element of C
  int64_t laid_out;     // elements of operands that are laid out before the tile kernel
  bool pieces;          // a row of C is a whole number of 16-byte pieces, on 16 bytes

  int64_t cols() const { return pass == Pass::kForward ? n : k; }
  // for the weights' gradient that of an average matrix, since the host does not
  // know the offsets.  Small matrices of uneven rows are slow for it: 32768 rows of 32
  // matrices 256 x 128 take 14 us if they are even and 138 us if one has half of
  // them, as its two tiles then sum on two compute units.
  int64_t length() const { return pass == Pass::kForward ? k : pass == Pass::kInput ? n : rows / std::max(1, mats); }
  // row tiles of bm rows: known for one matrix and for the weights' gradient,
  // otherwise an estimate (the offsets are on the device): half a tile more per
  // matrix than full ones, and at least one for every row or matrix
  int64_t row_tiles(int64_t bm) const {
    if (pass == Pass::kWeight) return mats * ceil_div(n, bm);
    if (!grouped) return ceil_div(rows, bm);
    return std::max<int64_t>(ceil_div(rows, bm) + mats / 2, std::min<int64_t>(rows, mats));
  }
  // at most so many
  int64_t row_tiles_max(int64_t bm) const {
    if (pass == Pass::kWeight || !grouped) return row_tiles(bm);
    return std::min<int64_t>(rows, ceil_div(rows, bm) + mats);
  }
};

struct RowsChoice {
  bool stream;     // k_rows_stream, which reads operands where they are, else k_rows_tile:
  int bm;          // rows of a tile, 64 (not for the weights' gradient), 128 or 256
  int slices;      // parts of L, joined from fp32 sums in the workspace
  bool join;       // through the workspace (slices > 1, or rows that the tile kernel cannot write)
  bool wide;       // rows of C in whole pieces
  int64_t tiles;   // at most so many, slices counted
};

// Tiles of the smallest kind, with the most that the groups' ends can add.
inline int64_t least_tiles(const RowsShape& s) {
  const int64_t tn = ceil_div(s.cols(), kRowsTileN);
  return (s.pass == Pass::kWeight ? s.mats * ceil_div(s.n, 128) : ceil_div(s.rows, 64) + s.mats) * tn;
}

// fp32 sums of a slice: rows of C as the tile kernel writes them
inline int64_t join_rows(const RowsShape& s) { return s.pass == Pass::kWeight ? s.mats * s.n : s.rows; }
inline int64_t join_ld(const RowsShape& s) { return (s.cols() + 3) & ~int64_t(3); }

// Tiles of 256 rows do the most products for what they read, smaller ones fill
// the chip and a matrix's end better (captured calls in a row on the same
// operands; 4096 columns, sums of 7168: 1024 rows 66 us in tiles of 64 and 79 in
// tiles of 128, 2048 rows 98 us in tiles of 128 and 125 in tiles of 256, 8192 rows
// 340 us in tiles of 256 and 381 in tiles of 128; 32768 rows of 64 matrices 1.83
// ms in tiles of 256 and 1.91 in tiles of 128).  Few tiles of long sums are cut
// into slices (64 rows: 20 us with 8 of them, 23 us with the 16 that are taken, 40
// us without; the gradient of one matrix 128 x 256 from 30000 rows 21 us with 64,
// 98 us with one).  Few products take k_rows_stream (1 row: 13 us, 16 us in tiles
// with 8 or 16 slices; 64 rows of 64 matrices, one each, 632 against 605 us in
// tiles, which is why the estimates are close to each other there).
inline RowsChoice choose_rows(const RowsShape& s) {
  const int64_t ntn = ceil_div(s.cols(), kRowsTileN), steps = std::max<int64_t>(1, ceil_div(s.length(), 64));
  // By estimates of their times in units of 0.1 us: a step, and a tile's end.
  // What is not on 16 bytes is laid out first: read and written, at 4 TB/s.
  const int64_t lay = (s.laid_out * 4 + (s.laid_out ? 800000 : 0)) / 400000;
  static const int kBm[3] = {256, 128, 64}, kStep[3] = {12, 8, 6}, kEnd[3] = {60, 40, 30};
  int64_t best = -1;
  RowsChoice c{};
  for (int i = 0; i < (s.pass == Pass::kWeight ? 2 : 3); ++i) {
    for (int slices = 1; slices <= kMaxSlices && (slices == 1 || slices * 4 <= steps); slices *= 2) {
      const int64_t tiles = s.row_tiles(kBm[i]) * ntn;
      if (slices > 1 && tiles * slices > 2 * kCus) break;
      const int64_t join = slices == 1 ? 0 : 50 + join_rows(s) * join_ld(s) * 8 * slices / 450000;
      const int64_t cost = ceil_div(tiles * slices, kCus) * (ceil_div(steps, slices) * kStep[i] + kEnd[i]) + join;
      if (best < 0 || cost < best) {
        best = cost;
        c.bm = kBm[i];
        c.slices = slices;
      }
    }
  }
  if (s.pass == Pass::kForward) {
    // 2 us, and 0.18 us per 256 units of 16 x 16 and 128 products
    const int64_t units = s.row_tiles(16) * ceil_div(s.n, 16);
    const int64_t stream = 20 + units * ceil_div(s.k, 128) * 18 / 2560;
    if (stream < best + lay) {
      c.stream = true;
      c.slices = 1;
      c.join = false;
      c.wide = false;
      c.tiles = s.row_tiles_max(16) * ceil_div(s.n, 16);
      return c;
    }
  }
  c.join = c.slices > 1 || (s.out_size == 4 && !s.pieces);
  c.wide = c.join || s.pieces;
  c.tiles = s.row_tiles_max(c.bm) * ntn * c.slices;
  return c;
}

}  // namespace rows
}  // namespace mxmoe
