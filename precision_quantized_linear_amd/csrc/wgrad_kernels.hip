// Gradient of a linear's weight for gfx950: dW [N, K] (fp32) = dy^T x of bf16 dy [M, N] and x [M, K].
#include "qpl_dma.h"
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
// 4096 x 4096 x 10752 takes 331 us (1.09 PFLOP/s; a third round of tiles is 0.6 full), 4096 x 4096 x 8192 234 us (1.17
// PFLOP/s), with the matrix unit busy for half of the time and half of a wavefront's time spent on waits to issue.
// Fragments read one step ahead, eight wavefronts for a tile and loads spread further apart took 333 to 367 us.
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
  const int lrow = lane / CH, lch = lane % CH;
  auto issue = [&](int piece, int d) {
    const bool isx = d < L;
    const int q = isx ? d : d - L;
    const int row = RPL * (L * wv + q) + lrow;
    const int ch = lch ^ (4 * (row & 3));
    const int64_t width = isx ? p.K : p.N, c0 = isx ? k0 : n0;
    const int64_t m = (int64_t)piece * TOK;
    const int64_t rows = p.M - m < TOK ? (p.M - m > 0 ? p.M - m : 0) : TOK;
    const u32x4 desc = make_desc((isx ? p.x : p.dy) + m * width, rows * width * 2);
    const uint32_t vo = c0 + 8 * ch < width ? (uint32_t)((row * width + c0 + 8 * ch) * 2) : kOutOfRange;
    const int stage = piece % S;
    dma16(lbase + stage * STAGE + (isx ? 0 : OP) + 1024 * (L * wv + q), piece < np ? vo : kOutOfRange, desc, 0);
  };
  // fragment of 32 channels from `c` on, tokens 16 u .. 16 u + 15 (lane l: channel l % 32, tokens 8 (l / 32) ..)
  auto frag = [&](const uint8_t* op, int c, int u) {
    i16x4 r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 16 * u + 8 * (lane >> 5) + 4 * i + ((lane & 15) >> 2);
      const int col = c + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
      const uint8_t* a = op + row * ROW + (((col >> 3) ^ (4 * (row & 3))) << 4) + (col & 7) * 2;
      r[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)a);
    }
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(r[0], r[1], 0, 1, 2, 3, 4, 5, 6, 7));
  };
  f32x16 acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[i][j] = f32x16{};
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
#pragma unroll
    for (int d = 0; d < 2 * L; ++d) issue(s, d);
  for (int k = 0; k < np; ++k) {
    QPL_WAIT_LGKM0();  // this wavefront is done with the stage that the next loads fill
    QPL_WAIT_VMCNT((S - 2) * 2 * L);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const uint8_t* st = lds + (k % S) * STAGE;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      bf16x8 fx[T], fy[T];
#pragma unroll
      for (int i = 0; i < T; ++i) fx[i] = frag(st, 32 * (T * wk + i), u);
#pragma unroll
      for (int j = 0; j < T; ++j) fy[j] = frag(st + OP, 32 * (T * wn + j), u);
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fx[i], fy[j], acc[i][j], 0, 0, 0);
          const int s = u * T * T + T * i + j;
#pragma unroll
          for (int d = 0; d < 2 * L; ++d)
            if (s == d * 2 * T * T / (2 * L)) issue(k + S - 1, d);
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
  // large tiles' outputs are one round.  us for 4096 tokens at 64 large tiles 53 small, 95 large; at 128 84 and 98; at
  // 224 160 and 121; at 256 167 and 126; at 672 457 and 328
  const int64_t big = ((N + 255) / 256) * ((K + 255) / 256);
  if (big > 128) return launch_grad<4, 4>(p, stream);
  return launch_grad<2, 4>(p, stream);
}

}  // namespace qpl
