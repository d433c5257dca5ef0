// Which kernel multiplies a block-scaled fp8 linear: host arithmetic on the sizes alone.
#pragma once

#include <cstdint>

namespace qpl {

// A few rows in one launch (k_fp8b_token): up to 16, of up to FP8B_TOKEN_PARTS parts of 512 channels together, which is
// two for each wavefront.  us in one launch and in two (quantizer, product): 1 x 4096 x 4096 4.7 and 8.8, 4 x 4096 x
// 4096 6.0 and 9.4, 16 x 1024 x 4096 5.0 and 6.6, 2 x 8192 x 8192 15.4 and 20.5, gated 4 x 4096 x 10752 18.7 and 23.5.
constexpr int FP8B_TOKEN_PARTS = 32;
inline bool fp8b_token_fits(int64_t M, int64_t K) { return M <= 16 && M * ((K + 511) / 512) <= FP8B_TOKEN_PARTS; }

// ---------------------------------------------------------------------------
// Which kernel multiplies otherwise.  A workgroup's time is about
//   (pieces of 128 channels) * piece + tile   microseconds
// with the constants below, and the 256 CUs take the tiles in rounds; the shape with the least time is taken.
// The direct kernel's piece is its bytes at 40 KB/us, and several of its workgroups share a CU, so its rounds need
// not be whole.  Measured, us in a graph with the quantizer's launch (4 to 5 us):
//   M    K    N      16x16 16x32 32x32 64x64 64x128 128x128 128x256 256x256
//   17   4096 4096   15.1  12.9  13.8  17.4  20.8   24.5
//   48   4096 12288  51.6  35.0  28.6  19.0  21.9   25.7
//   64   8192 1024   14.7  17.8  21.2  27.6  33.9   40.8
//   256  1024 6144   61.0  26.4  20.9  11.6  11.0   12.5    13.8    16.5
//   256  4096 4096   84.9  50.7  37.4  19.3  22.4   25.6    27.6    40.2
//   515  2064 5003   127   58.3  40.6  24.7  24.4   25.3    25.0    30.0
//   512  4096 12288  476   263   180   56.2  43.4   43.2    40.4    45.4
//   1536 4096 12288                    158   114    107     103     108
//   4096 4096 12288                    406   296    245     227     205
// gated, N the columns of both weights:
//   17   4096 21504        35.8  26.6        22.0   35.9
//   515  2048 5632         69.2  50.3        19.4   23.2    19.6    26.3
//   1024 4096 8192                           53.9   46.9    43.9    47.1
//   4096 4096 21504                          472    392     368     343
// two segments (the gated backward, with its first launch), K of both:
//   16   21504 4096  28.4  36.8  39.4  61.4  76.8
//   130  5472 1040   22.4  18.6  15.7  23.0  27.4           37.9    53.4
//   515  11264 2048  199   143   106   51.7  50.4           63.0    100
// Of 108 such sizes, most of them random, the shape taken was within 9 % of the best for 107.  A 128 x 128
// shape (the table's column) was the best for one of them, by 4 %, and is not built.
// ---------------------------------------------------------------------------
// rows and cols: outputs of a workgroup (a gated product makes cols / 2 of them from as many rows of each weight).
struct Fp8bShape {
  int rows, cols;
  double piece, tile;
};
constexpr Fp8bShape kFp8bShapes[] = {{16, 16, 0, 1.9},    {16, 32, 0, 1.7},    {32, 32, 0, 2.0},     {64, 64, 0.3, 1.9},
                                     {64, 128, 0.41, 2.7}, {128, 256, 1.18, 3.4}, {256, 256, 2.05, 6.3}};
constexpr int kFp8bShapeCount = 7;
// A gated product has no 16 x 16 shape (its 16 x 32 is as fine) and no 64 x 64 shape, where a wavefront has too few
// column tiles for two weights.
constexpr bool fp8b_gated_shape(int v) { return v != 0 && v != 3; }

// Shape of a product of M rows by N columns (of all weights together) over `pieces` pieces of K.
inline int fp8b_shape(int64_t M, int64_t pieces, int64_t N, bool gated) {
  int best = -1;
  double least = 0;
  for (int v = 0; v < kFp8bShapeCount; ++v) {
    if (gated && !fp8b_gated_shape(v)) continue;
    const Fp8bShape& s = kFp8bShapes[v];
    const bool direct = s.piece == 0;
    const double tiles = (double)((M + s.rows - 1) / s.rows) * (double)((N + s.cols - 1) / s.cols) / 256;
    const double left = tiles - __builtin_floor(tiles);  // of the last round; staged tiles are cut in it
    const double last = left == 0 ? 0 : s.rows >= 256 && left <= 0.25 ? 0.6 : s.rows >= 128 && left <= 0.5 ? 0.8 : 1;
    const double rounds = direct ? (tiles > 1 ? tiles + 0.2 : 1) : tiles - left + last;
    const double piece = direct ? ((M < s.rows ? M : s.rows) + s.cols) * 128 / 40e3 : s.piece;
    const double t = rounds * (double)pieces * piece + (rounds > 1 ? rounds : 1) * s.tile;
    if (best < 0 || t < least) {
      best = v;
      least = t;
    }
  }
  return best;
}

}  // namespace qpl
