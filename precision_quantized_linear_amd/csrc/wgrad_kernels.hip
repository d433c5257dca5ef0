// Gradient of a linear's weight for gfx950: dW [N, K] (fp32) = dy^T x of bf16 dy [M, N] and x [M, K].
#include "qpl_dma_lane.h"
#include "qpl_internal.h"

namespace qpl {

namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// The sum runs over tokens, the slow axis of both operands, so both come through LDS as they lie and are turned
// over on the way to the registers: ds_read_b64_tr_b16 takes 4 tokens x 16 channels from 16 lanes (lane l gives the
// address of token l / 4, channels 4 (l % 4) ..) and returns channel l's 4 tokens to lane l.
//
// A workgroup of four wavefronts (2 x 2) owns 64 T channels of x by 64 T of dy; a wavefront T x T tiles of 32 x 32
// (V_MFMA_F32_32X32X16_BF16).  x is the first operand, so a lane holds four consecutive channels of x for one of
// dy: 16 bytes of a row of dW.  S stages of 32 tokens ring through LDS, filled by buffer_load_dwordx4 ... lds between
// the MFMAs.  16-byte chunk c of a stage row r sits at chunk c ^ 4 (r % 4): the four rows that a read takes, whose
// distance is a multiple of 256 bytes, hit different banks.
//
// A piece is multiplied in two halves of 16 tokens.  Under the first half's MFMAs the second's fragments are read and
// the piece S - 1 ahead is loaded; then comes the sync, and under the second half's the next piece's first fragments
// are read.  The order of issue is pinned MFMA by MFMA: a wavefront has its SIMD for itself, so what is not issued
// beside an MFMA leaves the matrix unit idle.
//
// 4096 x 4096 x 10752 takes 316 us (1.14 PFLOP/s; a third round of tiles is 0.6 full), 4096 x 4096 x 8192 224 us (1.23
// PFLOP/s): bound by the matrix unit, the sync of each piece and power.  With a half's fragments read at its start
// they took 331 and 234 us, with eight wavefronts for a tile 333 and more.
// ---------------------------------------------------------------------------
struct GradArgs {
  const uint16_t* dy;
  const uint16_t* x;
  float* dw;
  int64_t M, N, K;
  int tiles_n, tiles_k;
};

template <int T, int S>
__global__ __launch_bounds__(256) void k_weight_grad(GradArgs p) {
  constexpr int C = 64 * T, ROW = 2 * C, TOK = 32, OP = TOK * ROW, STAGE = 2 * OP;  // bytes
  constexpr int L = OP / 1024 / 4;                       // loads per wavefront and operand
  constexpr int RPL = 1024 / ROW;                        // rows of a load
  constexpr int CH = ROW / 16;                           // chunks of a row
  __shared__ __attribute__((aligned(16))) uint8_t lds[S * STAGE];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wk = wv >> 1, wn = wv & 1;
  const uint32_t lbase = lds_address(lds);
  // workgroups of one XCD take neighbouring tiles
  const int nwg = gridDim.x, b = blockIdx.x;
  const int each = (nwg + 7) >> 3, at = (b & 7) * each + (b >> 3);
  const int t = (nwg & 7) == 0 ? at : b;
  const int tn = t / p.tiles_k, tk = t % p.tiles_k;
  const int64_t n0 = (int64_t)tn * C, k0 = (int64_t)tk * C;
  const int np = (int)((p.M + TOK - 1) / TOK);

  // lane l of load q: row RPL (L wv + q) + l / CH of the stage, its chunk l % CH holds the row's chunk ^ 4 (row % 4)
  uint32_t vo[2 * L];
#pragma unroll
  for (int d = 0; d < 2 * L; ++d) {
    const bool isx = d < L;
    const int row = RPL * (L * wv + (isx ? d : d - L)) + lane / CH;
    const int ch = (lane % CH) ^ (4 * (row & 3));
    const int64_t width = isx ? p.K : p.N, c0 = isx ? k0 : n0;
    vo[d] = c0 + 8 * ch < width ? (uint32_t)((row * width + c0 + 8 * ch) * 2) : kOutOfRange;
  }
  // rows past the last token, and pieces past the last, are past the descriptor's end
  auto source = [&](int piece, bool isx) {
    const int64_t m = (int64_t)piece * TOK, width = isx ? p.K : p.N;
    const int64_t rows = p.M - m < TOK ? (p.M - m > 0 ? p.M - m : 0) : TOK;
    return make_desc((isx ? p.x : p.dy) + (rows > 0 ? m * width : 0), rows * width * 2);
  };
  auto issue = [&](int stage, int d, const u32x4& desc) {
    dma16(lbase + stage * STAGE + (d < L ? 0 : OP) + 1024 * (L * wv + (d < L ? d : d - L)), vo[d], desc);
  };
  // Fragment of 32 channels, tokens 16 u .. 16 u + 15 (lane l: channel l % 32, tokens 8 (l / 32) ..), in two reads.
  // The swizzle moves whole fragments, so each has an address of its own, and the tokens are offsets from it.
  uint32_t ax[T], ay[T];
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int r = (lane & 15) >> 2;
    const int row = 8 * (lane >> 5) + r, lo = 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
    ax[i] = row * ROW + 64 * ((T * wk + i) ^ r) + lo;
    ay[i] = OP + row * ROW + 64 * ((T * wn + i) ^ r) + lo;
  }
  i16x4 f[2][2 * T][2];  // of both halves of a piece: x's, then dy's
  auto read = [&](int stage, int u, int t) {  // t: one of 4 T reads
    const int i = t >> 1, h = t & 1;
    const uint8_t* at = lds + stage * STAGE + (i < T ? ax[i] : ay[i - T]) + (16 * u + 4 * h) * ROW;
    f[u][i][h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)at);
  };
  auto frag = [&](int u, int i) {
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(f[u][i][0], f[u][i][1], 0, 1, 2, 3, 4, 5, 6, 7));
  };
  f32x16 acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[i][j] = f32x16{};
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    const u32x4 sx = source(s, true), sy = source(s, false);
#pragma unroll
    for (int d = 0; d < 2 * L; ++d) issue(s, d, d < L ? sx : sy);
  }
  QPL_WAIT_VMCNT((S - 2) * 2 * L);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int t = 0; t < 4 * T; ++t) read(0, 0, t);
  for (int k = 0; k < np; ++k) {
    const u32x4 sx = source(k + S - 1, true), sy = source(k + S - 1, false);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) {
          const int s = T * i + j;
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(u, i), frag(u, T + j), acc[i][j], 0, 0, 0);
#pragma unroll
          for (int t = 0; t < 4 * T; ++t)
            if (s == t / 2) read(u == 0 ? k % S : (k + 1) % S, 1 - u, t);
          if (u == 0)
#pragma unroll
            for (int d = 0; d < 2 * L; ++d)
              if (s == d * T * T / (2 * L)) issue((k + S - 1) % S, d, d < L ? sx : sy);
          __builtin_amdgcn_sched_barrier(0);
        }
      if (u == 0) {
        QPL_WAIT_LGKM0();  // this wavefront is done with the stage that the next piece's loads fill
        QPL_WAIT_VMCNT((S - 2) * 2 * L);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
    }
  }
#pragma unroll
  for (int j = 0; j < T; ++j) {
    const int64_t n = n0 + 32 * (T * wn + j) + (lane & 31);
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t k = k0 + 32 * (T * wk + i) + 8 * g + 4 * (lane >> 5);
        if (n < p.N && k < p.K)
          *reinterpret_cast<f32x4*>(p.dw + n * p.K + k) =
              f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
      }
  }
  QPL_WAIT_VMCNT(0);
}

template <int T, int S>
hipError_t launch_grad(GradArgs p, hipStream_t stream) {
  p.tiles_n = (int)((p.N + 64 * T - 1) / (64 * T));
  p.tiles_k = (int)((p.K + 64 * T - 1) / (64 * T));
  hipLaunchKernelGGL((k_weight_grad<T, S>), dim3((unsigned)(p.tiles_n * p.tiles_k)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_weight_grad(const uint16_t* dy, const uint16_t* x, int64_t M, int64_t N, int64_t K, float* dw,
                              hipStream_t stream) {
  GradArgs p{dy, x, dw, M, N, K, 0, 0};
  // 256 x 256 tiles read half as much, and a CU takes one at a time; of 128 x 128 tiles it takes two, so that 128
  // large tiles' outputs are one round.  us for 4096 tokens at 64 large tiles 51 small, 84 large; at 128 83 and 87; at
  // 224 158 and 108; at 256 163 and 114; at 672 457 and 316
  const int64_t big = ((N + 255) / 256) * ((K + 255) / 256);
  if (big > 128) return launch_grad<4, 4>(p, stream);
  return launch_grad<2, 4>(p, stream);
}

}  // namespace qpl
