// Which kernel multiplies a block-scaled fp8 linear: host arithmetic on the sizes alone.
#pragma once

#include <cstdint>

namespace qpl {

// A few rows in one launch (k_fp8b_token): up to 16, of up to FP8B_TOKEN_PARTS parts of 512 channels together.
constexpr int FP8B_TOKEN_PARTS = 32;
inline bool fp8b_token_fits(int64_t M, int64_t K) { return M <= 16 && M * ((K + 511) / 512) <= FP8B_TOKEN_PARTS; }

// rows and cols: outputs of a workgroup (a gated product makes cols / 2 of them from as many rows of each
// weight); piece and tile: microseconds for 128 channels, and for a tile.
struct Fp8bShape {
  int rows, cols;
  double piece, tile;
};
constexpr Fp8bShape kFp8bShapes[] = {{16, 32, 0, 0.5},      {32, 32, 0, 0.5},      {64, 64, 0.28, 0.5},
                                     {64, 128, 0.46, 1.0},  {128, 128, 0.62, 2.0}, {256, 256, 1.8, 8}};
constexpr int kFp8bShapeCount = 6;

// Shape of a product of M rows by N columns (of all weights together) over `pieces` pieces of K.  A gated product
// has no 64 x 64 shape: a wavefront there has one column tile, and needs one of each weight.
constexpr int FP8B_UNGATED = 2;
inline int fp8b_shape(int64_t M, int64_t pieces, int64_t N, bool gated) {
  int best = 0;
  double least = 0;
  for (int v = 0; v < kFp8bShapeCount; ++v) {
    if (gated && v == FP8B_UNGATED) continue;
    const Fp8bShape& s = kFp8bShapes[v];
    const double tiles = (double)((M + s.rows - 1) / s.rows) * (double)((N + s.cols - 1) / s.cols) / 256;
    const double left = tiles - __builtin_floor(tiles);
    const double last = left == 0 ? 0 : s.rows >= 256 && left <= 0.25 ? 0.6 : s.rows >= 128 && left <= 0.5 ? 0.8 : 1;
    const double piece = s.piece > 0 ? s.piece : ((M < s.rows ? M : s.rows) + s.cols) * 128 / 42e3;
    const double t = (tiles - left + last) * ((double)pieces * piece + s.tile);
    if (v == 0 || t < least) {
      best = v;
      least = t;
    }
  }
  return best;
}

}  // namespace qpl
