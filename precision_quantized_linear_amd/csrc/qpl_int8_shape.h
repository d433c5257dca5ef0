// Which kernel multiplies an 8-bit integer linear: host arithmetic on the sizes alone.
#pragma once

#include <cmath>
#include <cstdint>

namespace qpl {

// A few rows in one launch (k_int8_token): up to 16, of up to TOKEN_PARTS parts of 512 elements
// together.  Half as many elements again would lose: with four parts per wavefront
// 16 x 2048 x 6144 took 10.6 us, its two launches 8.3 us; with two, 16 x 1024 x 4096 takes
// 6.1 us either way.
constexpr int TOKEN_PARTS = 32;
inline bool token_fits(int64_t M, int64_t K) { return M <= 16 && M * ((K / 8 + 63) / 64) <= TOKEN_PARTS; }

// The row quantizer: a workgroup per row (true) or a wavefront per row.  A wavefront holds rows of up to
// 12288 elements in registers and would read longer ones twice; below that, a workgroup per row pays
// while rows are too few to fill the chip, up to more of them the longer they are.  Gathered rows come
// from the caches and pay sooner by the wavefront.  Measured (us in a graph, wavefront / workgroup):
//   rows     K 512    1024     2048     4096       8192       16384
//   16       2.4/2.6  2.7/2.7  3.0/2.7  3.6/2.8    5.0/3.2    14.8/4.0
//   256      2.6/2.8  3.1/3.1  3.1/2.8  4.1/3.3    6.2/3.8    22.7/5.4
//   1024     2.7/3.4  2.9/3.4  3.5/3.6  5.3/4.7    8.5/7.4    38.3/11.6
//   2048     2.8/3.8  3.4/3.9  5.2/5.2  7.8/7.0    12.9/10.8  45.7/19.0
//   4096     3.6/5.5  4.9/6.4  7.3/8.0  11.5/11.4  21.4/18.6  58.4/35.1
//   8192     4.8/8.9  7.3/10.5 10.9/13.0 19.0/18.8 36.4/34.0  110.6/62.9
// gathered, each row four times:
//   256      2.7/2.9  2.9/2.9  3.2/3.0  3.9/3.2    5.3/3.7    15.6/5.5
//   1024     2.8/3.2  3.1/3.3  3.5/3.8  4.3/5.1    6.2/7.3    22.1/11.3
//   4096     3.5/5.6  4.3/6.4  5.4/7.4  9.0/11.4   13.2/17.5  29.7/32.1
// Smoothed rows take the plain rows' rule: 4096 elements 9.9/6.5 for 1024 rows, 17.8/16.4 for 4096.
inline bool split_rows(int64_t rows, int64_t K, bool gathered) {
  if (K > 12288) return true;
  return K > 512 && rows <= (gathered ? K / 8 : K / 2);
}

// ---------------------------------------------------------------------------
// Which kernel multiplies.  A workgroup's time is about
//   (pieces of 128 bytes of K) * piece + tile   microseconds
// with the constants below, and the 256 CUs take the tiles in rounds; the shape with the least
// time is taken.  The direct kernel's piece is its bytes at 42 KB/us (operand rows that do not
// exist cost nothing), the staged kernel's was measured for each tile: about 60 KB/us of
// operands up to 128 x 128, MFMAs and LDS reads above.  Measured (us):
//   M    K    N      16x16 16x32 32x32 64x64 64x128 128x128 128x256 256x256
//   1    4096 4096   5.9   7.6   7.9   13.2  15.0   17.5
//   1    2048 6144   7.3   5.4   5.7   8.6   9.6    11.1
//   16   4096 12288  19.3  17.8  18.9  14.5  19.4   19.1
//   64   4096 4096   21.0  13.7  10.5  13.2  15.4   17.6
//   64   8192 1024   10.2  13.4  17.1  22.5  26.4   29.8
//   256  1024 6144   50.6  25.5  17.2  8.5   7.4    8.5     10.5    13.2
//   515  2080 5003   114   56    39.7  18.6  18.6   16.4    19.8    25.0
//   512  4096 12288  456   258   176   54.5  43.7   41.9    35.6    48.2
//   1025 4096 4096                     39.4  35.2   31.2    32.0    38.9
//   1536 4096 12288                    157   109    97.4    93.9    95.5
//   4096 4096 12288                    381   284    216     207     188
//   4608 4096 12288                    429   313    249     239     222
// (a launch in a graph, the weight from HBM where it is larger than the caches).  Of 65 random sizes, dense and grouped, the one taken was
// within 9 % of the best for 55, and 10 to 23 % behind it for ten.
// ---------------------------------------------------------------------------
struct Shape {
  int rows, cols;
  double piece, tile;
};
constexpr Shape kShapes[] = {{16, 16, 0, 0.25},    {16, 32, 0, 0.5},      {32, 32, 0, 0.5},      {64, 64, 0.28, 0.5},
                             {64, 128, 0.46, 1.0}, {128, 128, 0.62, 2.0}, {128, 256, 1.0, 3.7}, {256, 256, 1.6, 8}};
constexpr int kNumShapes = 8;

// tiles_m(rows): row tiles of that height; rows_each: rows that a row tile has at most; part:
// workgroups end at different times (grouped tiles differ in rows), so rounds are not whole.
template <class F>
int pick_shape(const F& tiles_m, double rows_each, int64_t K, int64_t N, bool part) {
  int best = 0;
  double least = 0;
  for (int v = 0; v < kNumShapes; ++v) {
    const Shape& s = kShapes[v];
    const double tiles = tiles_m(s.rows) * (double)((N + s.cols - 1) / s.cols) / 256;
    const double left = tiles - __builtin_floor(tiles);  // of the last round; staged tiles are cut in it
    const double last = left == 0 ? 0 : s.rows >= 256 && left <= 0.25 ? 0.6 : s.rows >= 128 && left <= 0.5 ? 0.8 : 1;
    const double rounds = part ? (tiles + 0.4 > 1 ? tiles + 0.4 : 1) : tiles - left + last;
    const double piece = s.piece > 0 ? s.piece : ((rows_each < s.rows ? rows_each : s.rows) + s.cols) * 128 / 42e3;
    const double t = rounds * ((double)((K + 127) / 128) * piece + s.tile);
    if (v == 0 || t < least) {
      best = v;
      least = t;
    }
  }
  return best;
}

// Shape of a product of M rows.
inline int dense_shape(int64_t M, int64_t K, int64_t N) {
  return pick_shape([&](int rows) { return (double)((M + rows - 1) / rows); }, (double)M, K, N, false);
}

// The shape of a grouped product.  The host knows the number of rows, not how the experts share
// them: of E experts that R rows are dealt to, E (1 - (1 - 1/E)^R) have any, and half a tile more
// than R / rows for each of them is a fair guess.
inline int grouped_shape(int64_t R, int64_t K, int64_t N, int64_t E) {
  const double used = (double)E * -std::expm1((double)R * std::log1p(-1.0 / (double)(E > 1 ? E : 2)));
  const double some = E > 1 ? (used > 1 ? used : 1) : 1;
  return pick_shape(
      [&](int rows) {
        const double t = (double)R / rows + some / 2;
        return t > some ? t : some;
      },
      (double)R / some, K, N, true);
}

// Row tiles of a grouped product: every expert with rows has at most one that is not full.
inline int64_t row_tile_bound(int64_t R, int64_t E, int rows) { return R / rows + (E < R ? E : R); }

// 128 x 128 tiles: one workgroup per CU with four stages, or past 256 tiles two with two stages:
// 192 tiles of K = 2048 take 13.5 against 15.6 us, 384 of them 24.6 against 19.1 us.
inline bool four_stages(int64_t row_tiles, int64_t N) { return row_tiles * ((N + 127) / 128) <= 256; }

}  // namespace qpl
