// Which kernel of kernels_linear.hip a product of MXFP4 matrices takes: the
// rule alone, plain host code without a device.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace mxmoe {

struct LinearShape {
  int64_t rows, n, k;
  int mats;
  bool grouped;         // rows go to the matrices by offsets, else all to the one
  int size;             // bytes of an element of y
  int64_t row_bytes;    // from a row of y to the next
  bool pieces;          // a row of y is a whole number of 16-byte pieces, on 16 bytes
  int scale_align;      // bytes on which every row of scales begins: 16, 4 or 1
  int num_cus;
};

struct LinearChoice {
  int bm;               // k_linear_tile: rows of a tile, 64, 128 or 256; 0: k_linear_stream
  int scales;           // k_linear_tile's GS or k_linear_stream's SCALES
  bool wide, once;      // of k_linear_tile
  int mt, nb, waves;    // of k_linear_stream
};

constexpr int kTileN = 256;  // columns of a tile

// Row tiles of bm rows: known for one matrix, otherwise an estimate (the
// offsets are on the device): half a tile more per matrix than full ones, and
// at least one for every row or matrix.
inline int64_t row_tiles(const LinearShape& a, int64_t bm) {
  if (!a.grouped) return (a.rows + bm - 1) / bm;
  return std::max<int64_t>((a.rows + bm - 1) / bm + a.mats / 2, std::min<int64_t>(a.rows, a.mats));
}
// at most so many
inline int64_t row_tiles_max(const LinearShape& a, int64_t bm) {
  return a.grouped ? std::min<int64_t>(a.rows, (a.rows + bm - 1) / bm + a.mats) : (a.rows + bm - 1) / bm;
}

inline LinearChoice choose_stream(const LinearShape& a) {
  const bool one = row_tiles_max(a, 16) * ((a.n + 15) / 16) <= a.num_cus;
  if (a.k % 512 == 0 && a.scale_align >= 16) return {0, 0, false, false, 1, 1, one ? 8 : 4};
  if (a.k % 128 == 0 && a.scale_align >= 4) return {0, 1, false, false, 1, 1, one ? 8 : 4};
  // what the tile kernel does not take comes here at every size: many rows in
  // units of 64 x 32, which read half as much per product
  return a.rows > 32 * a.mats ? LinearChoice{0, 2, false, false, 4, 2, 8} : LinearChoice{0, 2, false, false, 1, 1, 4};
}

inline LinearChoice choose_tile(const LinearShape& a, int bm) {
  if (!a.pieces) {
    // (256 rows of fp32 and partial pieces need more registers than there are;
    // with 16-bit results they fit: 8192 x 4095, k = 7168, 160 us against 197 us
    // in tiles of 128 rows)
    return {bm == 256 && a.size == 4 ? 128 : bm, 0, false, false, 0, 0, 0};
  }
  const bool whole = a.k % 512 == 0 && a.scale_align >= 16;
  const bool once = bm == 64 && a.rows <= (a.grouped ? 32 * a.mats : 64);
  return {bm, !whole ? 0 : bm == 64 && a.k % 1024 == 0 ? 4 : 2, true, once, 0, 0, 0};
}

// By estimates of their times in units of 0.1 us.
// Tiles: a tile on every CU takes 2 us and, per step of 256 of K,
// 0.6, 0.8 and 1.3 us for 64, 128 and 256 rows when few CUs are busy; a full
// chip takes about twice that for each (measured with k = 7168: 256 rows x
// 4096 columns in 64 tiles of 64 rows 23 us, in 16 of 256 rows 38 us; 131072
// rows over 64 matrices in 256-row tiles 314 us, in 64-row tiles 465 us), so
// the same weights rank them in both cases.
// Stream: 2 us, and 0.25 us per 256 units and 512 of K (measured: 64 rows x
// 4096 columns, k = 7168, 16.8 us against 19.6 us in tiles; 128 rows 30
// against 22 us; 16 rows 10 against 18 us).
inline LinearChoice choose_linear(const LinearShape& a) {
  // (the tile kernel's stores reach 2^31 bytes from a tile's first row)
  if (a.k % 128 || a.scale_align < 4 || a.row_bytes * 256 > (int64_t(1) << 31)) return choose_stream(a);
  const int64_t cblocks = (a.n + kTileN - 1) / kTileN, steps = (a.k + 255) / 256;
  auto tile_cost = [&](int64_t bm, int64_t step) {
    return (row_tiles(a, bm) * cblocks + a.num_cus - 1) / a.num_cus * (20 + steps * step);
  };
  const int64_t c64 = tile_cost(64, 6), c128 = tile_cost(128, 8), c256 = tile_cost(256, 13);
  const int64_t units = row_tiles(a, 16) * ((a.n + 15) / 16);
  const int64_t stream = 20 + units * ((a.k + 511) / 512) * 25 / 2560;
  const int64_t least = std::min(c64, std::min(c128, c256));
  if (stream < least) return choose_stream(a);
  return choose_tile(a, least == c64 ? 64 : least == c128 ? 128 : 256);
}

}  // namespace mxmoe
