// Block-scaled fp8 linears for gfx950: y[m, n] = sum_b s_x[m, b] s_w[n / 128, b] sum_{k in b} q_x q_w with E4M3
// codes, a scale for every 128 channels of a row of x and for every 128 x 128 block of the weight.
//
// A block's scale is s = max |v| times fp32(1 / 448), its codes E4M3(v / s) of the correctly rounded quotient; a zero
// block has s = 0 and signed-zero codes.  A block's products are summed by the FP8 matrix instructions, which cut each
// product of a group of eight below 2^-13 of the group's largest (measured with constructed operands for this form,
// the 32 x 32 x 64 one and the unscaled one), and each sum is folded into fp32 accumulators as acc += P (s_x s_w): one
// product and one fma per output and block.
#include "qpl_dma_lane.h"
#include "qpl_fp8b_shape.h"
#include "qpl_fp8.h"
#include "qpl_piece.h"

namespace qpl {

namespace {

constexpr int EPI_SILU = 4;  // gated: SiLU of the gate (else EPI_GELU)

// ---------------------------------------------------------------------------
// Row quantizer.  16 lanes hold a block, 8 channels each; a wavefront takes one row's 2048 channels, all its
// loads in flight together.  Scales [M, blocks], or (SLAB) [blocks, M], where a piece of a product finds those
// of consecutive rows in one run.  Takes `rows` of the M rows (row_slices).  HBM: 4096 x 4096 in 10.7 us, 4096 x
// 10752 in 26.8 (4.9 TB/s).
// ---------------------------------------------------------------------------
constexpr int QV = 4;  // vectors of 8 channels per lane

// Largest magnitudes (two packed bf16) of the 16 lanes that share a block, in all of them.
__device__ __forceinline__ uint32_t block_absmax(uint32_t m) {
  m = absmax_acc(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x128, 0xF, 0xF, true));  // row_ror:8
  m = absmax_acc(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x124, 0xF, 0xF, true));
  m = absmax_acc(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x122, 0xF, 0xF, true));
  return absmax_acc(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x121, 0xF, 0xF, true));
}

template <bool SLAB>
__global__ __launch_bounds__(256) void k_quant_fp8b(const uint16_t* __restrict__ x, int64_t rows, int64_t M, int64_t K,
                                                    int64_t pitch, uint32_t chunks, uint8_t* __restrict__ xq,
                                                    float* __restrict__ xs) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)(blockIdx.x / chunks) * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int64_t nv = K >> 3, nb = (K + 127) >> 7;
  const int64_t j0 = (int64_t)(blockIdx.x % chunks) * (64 * QV) + lane;
  const u32x4* xr = reinterpret_cast<const u32x4*>(x + row * K);
  u32x4 v[QV];
#pragma unroll
  for (int i = 0; i < QV; ++i)
    v[i] = j0 + 64 * i < nv ? __builtin_nontemporal_load(xr + j0 + 64 * i) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < QV; ++i) {
    const int64_t j = j0 + 64 * i;
    const RowDiv d = block_div(absmax_value(block_absmax(vec_absmax(v[i], 0u))));
    if (j < (SLAB ? 16 * nb : nv)) {  // the products' rows end with a whole block, zeros behind K
      reinterpret_cast<u32x2*>(xq + row * pitch)[j] = fp8_vec(v[i], d);
      if ((lane & 15) == 0) xs[SLAB ? (j >> 4) * M + row : row * nb + (j >> 4)] = d.s;
    }
  }
}

// Weight quantizer: a workgroup per 128 x 128 block.  HBM: 10752 x 4096 in 23.6 us (5.6 TB/s, part of it from caches).
__global__ __launch_bounds__(256) void k_quant_weight_fp8b(const uint16_t* __restrict__ w, int64_t N, int64_t K,
                                                           uint8_t* __restrict__ wq, float* __restrict__ ws) {
  __shared__ float part[4];
  const int64_t nv = K >> 3, kb = (K + 127) >> 7, nb = (N + 127) >> 7;
  const int64_t j = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
  for (int64_t bn = blockIdx.y; bn < nb; bn += gridDim.y) {
    const int64_t r0 = bn * 128 + (threadIdx.x >> 4);
    u32x4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + 16 * i;
      v[i] = r < N && j < nv ? reinterpret_cast<const u32x4*>(w + r * K)[j] : u32x4{0u, 0u, 0u, 0u};
      m = vec_absmax(v[i], m);
    }
    const float a = wave_max(absmax_value(m));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
    __syncthreads();
    const RowDiv d = block_div(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + 16 * i;
      if (r < N && j < nv) reinterpret_cast<u32x2*>(wq + r * K)[j] = fp8_vec(v[i], d);
    }
    if (threadIdx.x == 0) ws[bn * kb + blockIdx.x] = d.s;
    __syncthreads();
  }
}

// Transposed codes [K, N] and scales [K / 128, N / 128] of a weight [N, K]: a workgroup per 128 x 128 block, its
// bytes turned over in LDS.  A thread reads 16 channels of four rows and writes 16 rows of four channels.  HBM:
// 10752 x 4096 in 18.3 us (4.8 TB/s).
__global__ __launch_bounds__(256) void k_transpose_fp8b(const uint8_t* __restrict__ w, const float* __restrict__ ws,
                                                        int64_t N, int64_t K, uint8_t* __restrict__ wt,
                                                        float* __restrict__ wst) {
  constexpr int P = 132;  // bytes between rows: four rows' words of a column fall into different banks
  __shared__ __attribute__((aligned(16))) uint8_t t[128 * P];
  const int64_t kb = (K + 127) >> 7, nb = (N + 127) >> 7;
  const int64_t k0 = (int64_t)blockIdx.x * 128;
  for (int64_t bn = blockIdx.y; bn < nb; bn += gridDim.y) {
    const int64_t n0 = bn * 128;
    const int c = (threadIdx.x & 7) * 16, r0 = threadIdx.x >> 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 32 * i;
      u32x4 v{0u, 0u, 0u, 0u};
      if (n0 + r < N && k0 + c < K) v = *reinterpret_cast<const u32x4*>(w + (n0 + r) * K + k0 + c);
#pragma unroll
      for (int d = 0; d < 4; ++d) *reinterpret_cast<uint32_t*>(t + r * P + c + 4 * d) = v[d];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = r0 + 32 * i;  // row of the transposed block; columns c .. c + 15
      if (k0 + k < K && n0 + c < N) {
        u32x4 v;
#pragma unroll
        for (int d = 0; d < 4; ++d)
          v[d] = (uint32_t)t[(c + 4 * d) * P + k] | (uint32_t)t[(c + 4 * d + 1) * P + k] << 8 |
                 (uint32_t)t[(c + 4 * d + 2) * P + k] << 16 | (uint32_t)t[(c + 4 * d + 3) * P + k] << 24;
        *reinterpret_cast<u32x4*>(wt + (k0 + k) * N + n0 + c) = v;
      }
    }
    if (threadIdx.x == 0) wst[blockIdx.x * nb + bn] = ws[bn * kb + blockIdx.x];
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Backward of h = act(g) u: dg = dh u act'(g), du = dh act(g), rounded to bf16 (what a caller keeps for the
// weights' gradients), and the codes of both, side by side in a row: dg's blocks, then du's, as one product
// multiplies them by the two transposed weights.  One pass: 6 bytes read and 2 to 6 written per element.
// The products run in 8 bits like the forward's; the scheme's rule keeps 4 significant bits of each gradient.
// HBM and the vector unit alike: 4096 x 10752 with dg and du kept in 85 us (528 MB, 6.2 TB/s, part of it from caches).
// ---------------------------------------------------------------------------
constexpr float GELU_LINEAR = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float GELU_CUBE = 0.134145f;              // 3 * 0.044715

__device__ __forceinline__ float sigmoid2(float t) {  // 1 / (1 + 2^t)
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}
constexpr float LOG2E = 0x1.715476p+0f;

// act(v) and act'(v).  SiLU: v s and s (1 + v (1 - s)) with s = sigma(v).  GELU (tanh form): v s and
// s + 2 v s (1 - s) sqrt(2/pi) (1 + 3 * 0.044715 v^2) with s = sigma(2 u); past |v| = 12, where s is 0 or 1 in
// fp32, the slope is taken at 12, so that no product of an infinity and a zero arises.
template <bool SILU>
__device__ __forceinline__ void act_and_slope(float v, float& a, float& d) {
  if constexpr (SILU) {
    const float s = sigmoid2(-LOG2E * v), o = sigmoid2(LOG2E * v);
    a = v * s;
    d = __builtin_fmaf(a, o, s);
  } else {
    a = gelu_tanh(v);
    const float c = __builtin_amdgcn_fmed3f(v, -12.0f, 12.0f);
    const float t = c * __builtin_fmaf(GELU_C3, c * c, GELU_C1);
    const float s = sigmoid2(t), o = sigmoid2(-t);
    d = __builtin_fmaf(2.0f * GELU_LINEAR * c * (s * o), __builtin_fmaf(GELU_CUBE, c * c, 1.0f), s);
  }
}

template <bool SILU>
__device__ __forceinline__ void gate_gradients(uint32_t dh, uint32_t g, uint32_t u, uint32_t& dg, uint32_t& du) {
  float a[2], d[2], og[2], ou[2];
  act_and_slope<SILU>(bf16_lo(g), a[0], d[0]);
  act_and_slope<SILU>(bf16_hi(g), a[1], d[1]);
  const float h[2] = {bf16_lo(dh), bf16_hi(dh)}, w[2] = {bf16_lo(u), bf16_hi(u)};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    og[k] = h[k] * w[k] * d[k];
    ou[k] = h[k] * a[k];
  }
  dg = pack_bf16(og[0], og[1]);
  du = pack_bf16(ou[0], ou[1]);
}

constexpr int GV = 2;  // vectors of 8 channels per lane

template <bool SILU>
__global__ __launch_bounds__(256) void k_gated_backward(const uint16_t* dh, const uint16_t* g, const uint16_t* u,
                                                        int64_t rows, int64_t M, int64_t H, int64_t pitch, uint32_t chunks,
                                                        uint16_t* dg, uint16_t* du, uint8_t* __restrict__ q,
                                                        float* __restrict__ s) {
  // a lane has read all of its vectors before it writes the first: dg and du may be dh, g or u themselves
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)(blockIdx.x / chunks) * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int64_t nv = H >> 3, nb = (H + 127) >> 7;
  const int64_t j0 = (int64_t)(blockIdx.x % chunks) * (64 * GV) + lane;
  u32x4 v[GV][3];
#pragma unroll
  for (int i = 0; i < GV; ++i) {
    const bool in = j0 + 64 * i < nv;
    const int64_t at = row * nv + j0 + 64 * i;
    const u32x4 zero{0u, 0u, 0u, 0u};
    v[i][0] = in ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(dh) + at) : zero;
    v[i][1] = in ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(g) + at) : zero;
    v[i][2] = in ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(u) + at) : zero;
  }
#pragma unroll
  for (int i = 0; i < GV; ++i) {
    const int64_t j = j0 + 64 * i;
    u32x4 o[2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t a, b;
      gate_gradients<SILU>(v[i][0][k], v[i][1][k], v[i][2][k], a, b);
      o[0][k] = a;
      o[1][k] = b;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const RowDiv d = block_div(absmax_value(block_absmax(vec_absmax(o[w], 0u))));
      if (j < 16 * nb) {  // zeros behind H
        reinterpret_cast<u32x2*>(q + row * pitch + w * nb * 128)[j] = fp8_vec(o[w], d);
        if ((lane & 15) == 0) s[(w * nb + (j >> 4)) * M + row] = d.s;
        if (dg && j < nv) reinterpret_cast<u32x4*>(w == 0 ? dg : du)[row * nv + j] = o[w];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// What the products share.
// ---------------------------------------------------------------------------
struct Fp8bArgs {
  const uint8_t* x;    // codes [M, segs pieces of 128 bytes], rows px apart
  const float* xs;     // scales [segs pieces, M]
  const uint8_t* w[2]; // weight [N, K]; gated: of the gate and of up; two segments: of the first and second half of x
  const float* ws[2];  // [ceil(N / 128), pieces]
  int64_t M, N;
  int K, px, pieces, segs;
  uint16_t* save[2];   // gated: bf16 [M, N] of both projections, or nullptr
};

template <int EPI>
__device__ __forceinline__ float gate_act(float v) {
  if constexpr ((EPI & EPI_SILU) != 0) return v * sigmoid2(-LOG2E * v);
  return gelu_tanh(v);
}

__device__ __forceinline__ f32x4 mfma16(const i32x4 (&a)[2], const i32x4 (&b)[2]) {
  const i32x8 va = __builtin_shufflevector(a[0], a[1], 0, 1, 2, 3, 4, 5, 6, 7);
  const i32x8 vb = __builtin_shufflevector(b[0], b[1], 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, f32x4{}, 0, 0, 0, 127, 0, 127);
}

__device__ __forceinline__ void fold4(f32x4& acc, const f32x4& p, float s) {
#pragma unroll
  for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(p[r], s, acc[r]);
}

__device__ __forceinline__ void put_four(uint16_t* dst, const float (&o)[4], int64_t n, int64_t N) {
  const uint32_t w0 = pack_bf16(o[0], o[1]), w1 = pack_bf16(o[2], o[3]);
  if (n + 4 <= N) {
    reinterpret_cast<Segment4*>(dst)->v = u32x2{w0, w1};
  } else {
    dst[0] = (uint16_t)w0;
    if (n + 1 < N) dst[1] = (uint16_t)(w0 >> 16);
    if (n + 2 < N) dst[2] = (uint16_t)w1;
  }
}

// Outputs (m, n .. n + 3), if m < m1, as far as n < N; gated: of the projections a (gate) and b (up).
template <bool GATED, int EPI>
__device__ __forceinline__ void store_four(const Fp8bArgs& p, uint16_t* __restrict__ y, int64_t m, int64_t m1,
                                           int64_t n, const f32x4& a, const f32x4& b, const EpiArgs& e) {
  if (m >= m1 || n >= p.N) return;
  float o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    o[k] = a[k];
    if constexpr (GATED) {
      o[k] = gate_act<EPI>(a[k]) * b[k];
    } else if constexpr ((EPI & EPI_GELU) != 0) {
      o[k] = gelu_tanh(a[k]);
    }
  }
  put_four(out_ptr<EPI>(y, m, n, p.N, e), o, n, p.N);
  if constexpr (GATED) {
    if (p.save[0]) {
      const float g[4] = {a[0], a[1], a[2], a[3]}, u[4] = {b[0], b[1], b[2], b[3]};
      put_four(p.save[0] + m * p.N + n, g, n, p.N);
      put_four(p.save[1] + m * p.N + n, u, n, p.N);
    }
  }
}

// ---------------------------------------------------------------------------
// The product without LDS staging, for few rows.  A workgroup of W wavefronts owns 16 MT rows of x and 16 NT
// columns (gated: of each weight).  Its wavefronts take the pieces of K in turn, each lane loading its MFMA
// operands (V_MFMA_SCALE_F32_16X16X128_F8F6F4, 32 bytes per lane) straight from memory, and their sums meet in
// LDS, in the order of the wavefronts.  Operands are swapped (the MFMA computes y^T): a lane holds four
// consecutive columns of one row.  Lane l has bytes 16 (l / 16) and 64 + 16 (l / 16) of the piece of row l % 16.
// Bound by the latency of its loads, about 40 KB/us for a workgroup: 130 x 5472 x 1040 in two segments 10.0 to 11.2 us
// (32 x 32); 17 x 4096 x 4096 12.9 us with the quantizer's launch (16 x 32).
// ---------------------------------------------------------------------------
template <int MT, int NT, int W, int U, bool GATED, int EPI>
__global__ __launch_bounds__(64 * W) void k_fp8b_direct(Fp8bArgs p, uint16_t* __restrict__ Y, EpiArgs e) {
  constexpr int G = GATED ? 2 : 1, T = G * MT * NT;
  __shared__ f32x4 red[W][T][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r16 = lane & 15, q = lane >> 4;
  const int all = p.pieces * p.segs;
  const int64_t tiles_m = (p.M + 16 * MT - 1) / (16 * MT), tiles_n = (p.N + 16 * NT - 1) / (16 * NT);
  for (int64_t tm = blockIdx.y; tm < tiles_m; tm += gridDim.y) {
    for (int64_t tn = blockIdx.x; tn < tiles_n; tn += gridDim.x) {
      const int64_t m0 = tm * 16 * MT, n0 = tn * 16 * NT;
      const int64_t m1 = p.M - m0 < 16 * MT ? p.M : m0 + 16 * MT;
      const int64_t nr = p.N - n0 < 16 * NT ? p.N - n0 : 16 * NT;
      const __amdgpu_buffer_rsrc_t dx = make_rsrc(p.x + m0 * p.px, (m1 - m0) * p.px);
      f32x4 acc[G][MT][NT] = {};
      for (int c0 = wv; c0 < all; c0 += W * U) {
        i32x4 fx[U][MT][2], fw[U][G][NT][2];
        float sx[U][MT], sw[U][G];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * W;
          const bool second = c >= p.pieces;  // of two segments
          const int kc = second ? c - p.pieces : c;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const int which = GATED ? g : second ? 1 : 0;
            const __amdgpu_buffer_rsrc_t dw = make_rsrc(p.w[which] + n0 * p.K, nr * p.K);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const int k = kc * 128 + 64 * s + 16 * q;
              const bool in = c < all && k < p.K;
#pragma unroll
              for (int j = 0; j < NT; ++j)
                fw[u][g][j][s] = load16(dw, in ? (uint32_t)((16 * j + r16) * p.K + k) : kOutOfRange);
            }
            sw[u][g] = c < all ? p.ws[which][(n0 >> 7) * p.pieces + kc] : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const int k = kc * 128 + 64 * s + 16 * q;
              const bool in = c < all && k < p.K;
              fx[u][i][s] = load16(dx, in ? (uint32_t)((16 * i + r16) * p.px + c * 128 + 64 * s + 16 * q) : kOutOfRange);
            }
            const int64_t m = m0 + 16 * i + r16;
            sx[u][i] = c < all && m < m1 ? p.xs[(int64_t)c * p.M + m] : 0.0f;
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int j = 0; j < NT; ++j)
                fold4(acc[g][i][j], mfma16(fw[u][g][j], fx[u][i]), sx[u][i] * sw[u][g]);
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j) red[wv][(g * MT + i) * NT + j][lane] = acc[g][i][j];
      __syncthreads();
      // vector v: tile v / 64 (row block, column block), lane v % 64's four columns
      for (int v = threadIdx.x; v < MT * NT * 64; v += 64 * W) {
        const int tile = v >> 6, l = v & 63;
        f32x4 sum[2] = {};
#pragma unroll
        for (int g = 0; g < G; ++g) {
          sum[g] = red[0][g * MT * NT + tile][l];
#pragma unroll
          for (int k = 1; k < W; ++k) sum[g] += red[k][g * MT * NT + tile][l];
        }
        store_four<GATED, EPI>(p, Y, m0 + 16 * (tile / NT) + (l & 15), m1, n0 + 16 * (tile % NT) + 4 * (l >> 4), sum[0],
                               sum[1], e);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// A few rows (single tokens) in one launch: as the direct kernel, but every workgroup quantizes the M <= 16 rows
// itself, into LDS, while its first weight bytes are on their way.  A row is parts of 512 channels (four blocks);
// wavefront w takes the parts w, w + 16, ... of all rows.  1 x 4096 x 4096 in 4.7 us (3.6 TB/s: latency, 64 KB of
// weight per CU), gated 4 x 4096 x 10752 in 18.5 us (4.8 TB/s: HBM).
// ---------------------------------------------------------------------------
constexpr int TOKEN_W = 16, TOKEN_SLOTS = FP8B_TOKEN_PARTS / TOKEN_W;
constexpr int TOKEN_BYTES = FP8B_TOKEN_PARTS * 512 + 16 * 16;  // rows 16 bytes further apart than they are long

template <bool GATED, int EPI>
__global__ __launch_bounds__(64 * TOKEN_W) void k_fp8b_token(const uint16_t* __restrict__ x, Fp8bArgs p,
                                                             uint16_t* __restrict__ Y, EpiArgs e) {
  constexpr int W = TOKEN_W, U = 2, G = GATED ? 2 : 1;
  __shared__ __attribute__((aligned(16))) uint8_t codes[TOKEN_BYTES];  // [M, K + 16]
  __shared__ f32x4 red[W][G][64];
  __shared__ float scale[FP8B_TOKEN_PARTS * 4];  // [M, 4 parts]
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r16 = lane & 15, q = lane >> 4;
  const int M = (int)p.M, nv = p.K >> 3, pitch = p.K + 16;
  const int parts = (nv + 63) >> 6;
  const int rcp = (65536 + parts - 1) / parts;  // part / parts, exact for the numbers up to 32 that occur
  int64_t n0 = (int64_t)blockIdx.x * 16;
  i32x4 fw[U][G][2];
  float sw[U][G];
  auto load_w = [&](int c0, int64_t n) {
    const int64_t nr = p.N - n < 16 ? p.N - n : 16;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const __amdgpu_buffer_rsrc_t dw = make_rsrc(p.w[g] + n * p.K, nr * p.K);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * W;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int k = c * 128 + 64 * s + 16 * q;
          fw[u][g][s] = load16(dw, k < p.K ? (uint32_t)(r16 * p.K + k) : kOutOfRange);
        }
        sw[u][g] = c < p.pieces ? p.ws[g][(n >> 7) * p.pieces + c] : 0.0f;
      }
    }
  };
  // the rows' vectors, then (behind them, so that they do not wait for it) the first weight bytes
  u32x4 v[TOKEN_SLOTS];
#pragma unroll
  for (int t = 0; t < TOKEN_SLOTS; ++t) {
    const int u = wv + W * t, row = (u * rcp) >> 16, j = (u - row * parts) * 64 + lane;
    v[t] = row < M && j < nv ? reinterpret_cast<const u32x4*>(x + (int64_t)row * p.K)[j] : u32x4{0u, 0u, 0u, 0u};
  }
  load_w(wv, n0);
#pragma unroll
  for (int t = 0; t < TOKEN_SLOTS; ++t) {
    const int u = wv + W * t, row = (u * rcp) >> 16, sub = u - row * parts, j = sub * 64 + lane;
    if (row >= M) break;
    const RowDiv d = block_div(absmax_value(block_absmax(vec_absmax(v[t], 0u))));
    if (r16 == 0) scale[4 * u + q] = d.s;
    if (j < nv) reinterpret_cast<u32x2*>(codes + row * pitch)[j] = fp8_vec(v[t], d);
  }
  __syncthreads();
  for (;;) {
    f32x4 acc[G] = {};
    for (int c0 = wv; c0 < p.pieces; c0 += W * U) {
      if (c0 != wv) load_w(c0, n0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * W;
        i32x4 fx[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int k = c * 128 + 64 * s + 16 * q;
          fx[s] = i32x4{0, 0, 0, 0};
          if (r16 < M && k < p.K) fx[s] = *reinterpret_cast<const i32x4*>(codes + r16 * pitch + k);
        }
        const float sx = r16 < M && c < p.pieces ? scale[4 * r16 * parts + c] : 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) fold4(acc[g], mfma16(fw[u][g], fx), sx * sw[u][g]);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) red[wv][g][lane] = acc[g];
    // the next columns' first weight bytes
    const int64_t next = n0 + (int64_t)gridDim.x * 16;
    if (next < p.N) load_w(wv, next);
    __syncthreads();
    if (threadIdx.x < 64) {
      f32x4 sum[2] = {};
#pragma unroll
      for (int g = 0; g < G; ++g) {
        sum[g] = red[0][g][lane];
#pragma unroll 3
        for (int k = 1; k < W; ++k) sum[g] += red[k][g][lane];  // a few at a time: next to the weight in flight
      }
      store_four<GATED, EPI>(p, Y, r16, M, n0 + 4 * q, sum[0], sum[1], e);
    }
    n0 = next;
    if (n0 >= p.N) break;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// The product through LDS, for enough rows to reuse the weight.  A workgroup of WM x WN wavefronts owns 16 WM NJM
// rows of x by 16 WN NI rows of the weight; a wavefront 16 NJ x 16 NI of them: one V_MFMA_SCALE_F32_16X16X128_F8F6F4
// per block and 16 x 16 tile, from a zero accumulator, and four fmas that fold its sums, so the accumulators stay in
// vector registers.  Gated: half of a wavefront's NI column tiles belong to the gate, the other half to the same
// columns of up, so that both projections of an output meet in one lane.
//
// Workgroups are persistent; K is walked in pieces of 128 bytes (a block) of both operands, S stages of them in
// LDS, filled by buffer_load_dwordx4 ... lds together with the piece's scales.  The pieces of all of a workgroup's
// tiles form one stream.  A tile with at most half (a quarter) of its rows present runs with NJ = NJM / 2 (/ 4); the
// tiles of a last round that is at most half (a quarter) full are cut into such parts, one for each workgroup.
//
// A piece is multiplied row tile by row tile; a tile's sums are folded two MFMAs later.  The sync stands before its
// last row tile, when all of its operands are in registers: every wavefront waits for its own loads of the next
// piece, then all meet; the next piece is then in LDS and this piece's stage is free.  Behind it the loads of piece
// P + S are issued between MFMAs, into the first half of the next piece's, and the next piece's first operands are
// read, each column tile's as soon as the last row tile is done with the register.  A wavefront's vector memory
// operations retire in issue order, so the sync's wait names how many later ones may be in flight: the loads of the
// pieces behind the next and the output stores of an epilogue issued after its loads.  A smaller number than that only
// waits longer.
//
// Bound by the matrix unit and the instructions beside it, power and the tile ends: 4096 x 4096 x 12288 to q, k, v 208
// us of 219 with the quantizer's (2.0 PFLOP/s), gated 4096 x 4096 x 2 * 10752 with both projections kept 355 of 366 (2.0
// PFLOP/s), two segments 4096 x 21504 x 4096 310 us (2.3 PFLOP/s: few tile ends).  4096 x K x 12288, three tiles for
// each workgroup, takes 43, 104, 188, 361 and 704 us at K = 512, 2048, 4096, 8192 and 16384: 1.7 to 1.8 us a piece and
// 20 us for the launch and the three tiles' first pieces and ends.  To q, k, v it takes 17 to 32 us more at any of
// them: the stores' addresses, of three tensors in 64 bits.  The same on 32 x 32 x 64 tiles, two
// of them and sixteen fmas for a block, with the sync at a piece's end took 246, 425 and 370 us.
// ---------------------------------------------------------------------------
struct Fp8bStagedArgs {
  Fp8bArgs g;
  int tiles_m, tiles_n, nwg;
  uint16_t* y;
  EpiArgs e;
};

template <int WM, int WN, int NI, int NJM, int S>
struct StagedShape {
  static constexpr int W = WM * WN, XR = 16 * WM * NJM, WR = 16 * WN * NI;
  // a stage: scales (XR of x, 64 of each weight), rows of x, rows of W
  static constexpr int XB = 4 * XR + 512, WB = XB + XR * PR_ROW, STAGE = WB + WR * PR_ROW;
  static constexpr int LDS = S * STAGE + 256;         // and a spare area
  static constexpr int per_cu() { return (160 << 10) / LDS < 16 / W ? (160 << 10) / LDS : 16 / W; }
  static constexpr int per_simd() { return per_cu() * W / 4; }
};

// Epilogue of a wavefront's tile: y = bf16 of the accumulators (EPI_GELU: of their GELU).  acc[i][j] holds y^T:
// element r at lane l is row m0 + 16 j + l % 16, column n0 + 16 i + 4 (l / 16) + r.  Lanes of neighbouring rows of 16
// exchange words of column tiles i and i + 1 (V_PERMLANE16_SWAP), so that each holds eight consecutive columns: 8 (l /
// 32) .. of tile i + (l / 16) % 2.  Returns the number of stores left in flight (0 on the edge path, which checks
// every element and drains its stores).
template <int NJ, int NI, int EPI, bool ANY, bool FAST, class Acc>
__device__ __forceinline__ void store16_path(const Acc& acc, int lane, int64_t m0, int64_t n0, int64_t M, int64_t N,
                                             uint16_t* __restrict__ y, const EpiArgs& e) {
  const int q = lane >> 4;
  // loops expanded at compile time, as in store_tile; values, because a choice among an array's elements would become an
  // index into memory
  uint16_t *const oq = e.qkv[0], *const ok = e.qkv[1], *const ov = e.qkv[2];
  const int64_t d = e.d, tokens = e.tokens, off = e.off;
  const int lg_hd = e.lg_hd;
  static_for<0, NJ>([&](auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    const int64_t m = m0 + 16 * j + (lane & 15);
    static_for<0, NI / 2>([&](auto ic) __attribute__((always_inline)) {
      constexpr int i = 2 * decltype(ic)::value;
      uint32_t w[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float o[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = (EPI & EPI_GELU) != 0 ? gelu_tanh(acc[i + t][j][r]) : acc[i + t][j][r];
        w[t][0] = pack_bf16(o[0], o[1]);
        w[t][1] = pack_bf16(o[2], o[3]);
      }
      const auto a = __builtin_amdgcn_permlane16_swap(w[0][0], w[1][0], false, false);
      const auto b = __builtin_amdgcn_permlane16_swap(w[0][1], w[1][1], false, false);
      const u32x4 v{a[0], b[0], a[1], b[1]};
      const int64_t n = n0 + 16 * (i + (q & 1)) + 8 * (q >> 1);
      uint16_t* dst = y + m * N + n;
      if constexpr ((EPI & EPI_QKV) != 0) {  // as out_ptr, without an array indexed by the part; eight columns are of one head
        const bool k = n >= d, v2 = n >= 2 * d;
        const int64_t c = n - (v2 ? 2 * d : k ? d : 0), hd = c >> lg_hd;
        dst = (v2 ? ov : k ? ok : oq) + (((hd * tokens + off + m) << lg_hd) + (c & ((int64_t{1} << lg_hd) - 1)));
      }
      if constexpr (FAST && !ANY) {
        *reinterpret_cast<u32x4*>(dst) = v;
      } else if constexpr (FAST) {
        reinterpret_cast<Segment*>(dst)->v = v;
      } else if (m < M) {
        if (n + 8 <= N) {
          reinterpret_cast<Segment*>(dst)->v = v;
        } else {
          const uint32_t el[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (n + c < N) dst[c] = (uint16_t)(el[c >> 1] >> (16 * (c & 1)));
        }
      }
    });
    __builtin_amdgcn_sched_barrier(0);  // a row tile at a time: registers
  });
}

// This lane's number in its wavefront, made anew at each call: one that is kept costs a register all along.
__device__ __forceinline__ int lane_id() {
  int lane;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(lane));
  return lane;
}

template <int NJ, int NI, int EPI, bool ANY, class Acc>
__device__ __forceinline__ int store16(const Acc& acc, int64_t m0, int64_t n0, int64_t M, int64_t N,
                                       uint16_t* __restrict__ y, const EpiArgs& e) {
  const int lane = lane_id();  // what follows is not to be computed before the products, where registers are scarce
  if (m0 + 16 * NJ <= M && n0 + 16 * NI <= N) {
    store16_path<NJ, NI, EPI, ANY, true>(acc, lane, m0, n0, M, N, y, e);
    return NJ * NI / 2;
  }
  store16_path<NJ, NI, EPI, ANY, false>(acc, lane, m0, n0, M, N, y, e);
  QPL_WAIT_VMCNT(0);
  return 0;
}

template <int WM, int WN, int NI, int NJM, int S, bool GATED, int EPI>
__global__ __launch_bounds__(64 * WM * WN)
__attribute__((amdgpu_waves_per_eu((StagedShape<WM, WN, NI, NJM, S>::per_simd()),
                                   (StagedShape<WM, WN, NI, NJM, S>::per_simd())))) void
k_fp8b_staged(Fp8bStagedArgs) {
  using C = StagedShape<WM, WN, NI, NJM, S>;
  constexpr int W = C::W, XR = C::XR, WR = C::WR, XB = C::XB, WB = C::WB, STAGE = C::STAGE;
  constexpr int NO = GATED ? NI / 2 : NI;              // column tiles of outputs per wavefront
  constexpr int COLS = 16 * WN * NO;                   // output columns of a tile
  constexpr int XL = XR / 8 / W, WL = WR / 8 / W;      // loads per wavefront per piece: x, W
  constexpr int LOADS = XL + WL + 1;                   // and one of scales
  static_assert(XR / 64 + 2 <= W, "one load of scales per wavefront");
  static_assert((XR / W) % 16 == 0 && (WR / W) % 16 == 0, "the swizzle of a load's rows");
  static_assert(!GATED || (WM == 2 && NO % 2 == 0), "a wavefront loads rows of one weight");
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::LDS];
  // The arguments are read where they are needed, from the kernel's argument block: held in scalar registers through
  // the loop over K they would push its own values out of them.
  using Args = const __attribute__((address_space(4))) Fp8bStagedArgs;
  auto args = []() {
    Args* p = (Args*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
  };
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wv / WN, wn = wv % WN;
  const int q = lane >> 4, r16 = lane & 15;
  const uint32_t lbase = lds_address(lds);
  const int pieces = args()->g.pieces, np = pieces * args()->g.segs;

  struct Tile {
    int m0, n0, rows;
  };
  // This workgroup's i-th unit: a tile, or a part of one of the last round's; rows <= 0 if there is none.
  // Workgroups are dealt to the 8 XCDs in turn; in every round, the last and shorter one too, an XCD's workgroups
  // take a contiguous run of units.
  auto tile = [&](int i) {
    Args* a = args();
    const int nwg = a->nwg, ntiles = a->tiles_m * a->tiles_n, b = blockIdx.x;
    const int full = ntiles - ntiles % nwg, tail = ntiles - full;
    const int parts = NJM >= 8 && 4 * tail <= nwg ? 4 : NJM >= 4 && 2 * tail <= nwg ? 2 : 1;
    const int units = full + tail * parts;
    const int base = i * nwg, left = min(units - base, nwg);
    const int each = (left + 7) >> 3, at = (b & 7) * each + (b >> 3);
    int u = -1;
    if (left > 0) {
      if ((nwg & 7) != 0) {
        u = b < left ? base + b : -1;
      } else {
        u = (b >> 3) < each && at < left ? base + at : -1;
      }
    }
    Tile t{0, 0, 0};
    if (u < 0) return t;
    int tm, tn;
    const bool whole = u < full;
    const int cut = whole ? 0 : (u - full) % parts;
    walk(whole ? u : full + (u - full) / parts, a->tiles_m, a->tiles_n, tm, tn);
    t.n0 = tn * COLS;  // M and N are below 2^31
    t.m0 = tm * XR;
    t.rows = min((int)a->g.M - t.m0, XR);
    if (!whole && parts > 1) {
      const int first = XR / parts * cut;
      t.m0 += first;
      t.rows = min(t.rows - first, XR / parts);
    }
    return t;
  };

  // load n of an operand: stage rows (rows / W) wv + 8 n .. + 7; lane l fills row + l / 8, stage chunk l % 8, with
  // the row's chunk (l % 8) ^ ((row / 2) % 8) = lc ^ 4 (n % 2).  Gated: the rows of a wavefront's share all belong to
  // the gate (even wavefronts) or to up.
  const int lc = (lane & 7) ^ (lane >> 4);
  uint32_t vx, vw;
  {
    const int wrow = GATED ? (wv >> 1) * (WR / W) : wv * (WR / W);
    vx = (uint32_t)((XR / W * wv + (lane >> 3)) * args()->g.px + 16 * lc);
    vw = (uint32_t)((wrow + (lane >> 3)) * args()->g.K + 16 * lc);
  }
  const int job = wv < XR / 64 ? 0 : wv - XR / 64 + 1;  // scales: of x, of the first weight, of the second
  const bool scales = job <= (GATED ? 2 : 1);
  // a lane's scale lies vs_step bytes behind the lane's before it: the next row's of x, the next 128 rows' of a weight
  const uint32_t vs_step = job == 0 ? 4 : (uint32_t)pieces * 4, vs0 = !scales ? kOutOfRange : job == 0 ? 256u * wv : 0;

  // The stream of pieces: what the loads of the next one need.  Past the last tile the operands have no rows, and
  // zeros are loaded.
  int s_i = 0, s_k = 0, s_stage = 0;  // tile, piece, stage
  const uint8_t *xp = nullptr, *wp = nullptr;
  const float* sp = nullptr;
  int x_bytes = 0, w_bytes = 0, sp_bytes = 0, sp_step = 0, kx = 0, kw = 0;
  int s_n0 = 0;
  auto weight = [&](int which) {  // rows and scales of the tile in one of the weights
    Args* a = args();
    const int rn = min((int)a->g.N - s_n0, COLS);
    const int row_part = GATED ? wv & 1 : which;
    wp = (row_part ? a->g.w[1] : a->g.w[0]) + (int64_t)s_n0 * a->g.K;
    w_bytes = rn * a->g.K;
    if (job == 0) return;
    // one scale for every 128 rows of the weight, whose rows of scales are `pieces` long
    const int scale_part = GATED ? job - 1 : which;
    const int nb0 = s_n0 >> 7, nb = min((int)((a->g.N + 127) >> 7) - nb0, (COLS + 127) / 128);
    sp = (scale_part ? a->g.ws[1] : a->g.ws[0]) + (int64_t)nb0 * pieces;
    sp_bytes = ((nb - 1) * pieces + 1) * 4;
    sp_step = 1;
  };
  // moves the stream to the piece to load next; its loads have to be issued before the following call
  int l_stage = 0;
  auto next_piece = [&]() {
    l_stage = s_stage;
    s_stage = s_stage == S - 1 ? 0 : s_stage + 1;
    kx += PR_ROW;
    kw += PR_ROW;
    sp += sp_step;
    if (s_k == 0 || s_k == pieces) {  // a tile, or the second of two segments
      if (s_k == 0) {
        const Tile t = tile(s_i);
        kx = 0;
        x_bytes = w_bytes = sp_bytes = 0;
        if (t.rows > 0) {
          Args* a = args();
          s_n0 = t.n0;
          xp = a->g.x + (int64_t)t.m0 * a->g.px;
          x_bytes = t.rows * a->g.px;
          weight(0);
          if (job == 0) {
            sp = a->g.xs + t.m0;
            sp_bytes = t.rows * 4;
            sp_step = (int)a->g.M;
          }
        }
      } else if (x_bytes > 0) {
        weight(1);
      }
      kw = 0;
    }
    if (++s_k == np) {
      s_k = 0;
      ++s_i;
    }
  };
  // px, pw: pitches of x and W.  A lane's whole offset is in voff: rows past the operand's last, and everything where
  // there is no tile, are past the descriptor's end by it.  With the rows' and K's part moving the descriptor's start
  // and size instead (five scalar instructions a load) the gated 4096 x 4096 x 2 * 10752 took 375 us for 369.
  auto issue = [&](int d, int px, int pw) {
    const uint32_t st = lbase + l_stage * STAGE;
    if (d < XL) {
      dma16(st + XB + (XR / W * wv + 8 * d) * PR_ROW, (d & 1 ? vx ^ 64 : vx) + (uint32_t)(kx + 8 * d * px),
            make_desc(xp, x_bytes));
    } else if (d < XL + WL) {
      const int n = d - XL;
      dma16(st + WB + (WR / W * wv + 8 * n) * PR_ROW,
            (n & 1 ? vw + (lane & 4 ? -64 : 64) : vw) + (uint32_t)(kw + 8 * n * pw), make_desc(wp, w_bytes));
    } else {
      dma4(scales ? st + (job == 0 ? 256 * wv : 4 * XR + 256 * (job - 1)) : lbase + S * STAGE,
           __umul24((uint32_t)lane_id(), vs_step) + vs0, make_desc(sp, sp_bytes));
    }
  };

  // fragment of 16 rows: lane l has chunks l / 16 and 4 + l / 16 of row l % 16
  const int at0 = r16 * PR_ROW + ((q ^ (r16 >> 1)) << 4), at1 = at0 ^ 64;
  auto frag = [&](const uint8_t* a, const uint8_t* b) {
    return __builtin_shufflevector(*reinterpret_cast<const i32x4*>(a), *reinterpret_cast<const i32x4*>(b), 0, 1, 2, 3, 4,
                                   5, 6, 7);
  };
  auto mma = [&](const i32x8& w, const i32x8& x) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{}, 0, 0, 0, 127, 0, 127);
  };

  constexpr int LATER = (S - 2) * LOADS;        // loads of the pieces behind the next
  constexpr int STORES = NO * NJM / 2;          // output stores of a whole tile
  static_assert(LATER + STORES < 64, "vmcnt holds 63");
  int stores[S - 1] = {};  // left in flight by the epilogue after each of the last S - 1 pieces
  int cur = 0;             // stage of the piece being multiplied
  i32x8 fw[NI], fx[2];     // operands: the weight's column tiles, row tile j in fx[j % 2]
  float sw[2], sx[2];      // their scales

  auto sync = [&]() {
    QPL_WAIT_LGKM0();
    int n = 0;
#pragma unroll
    for (int i = 0; i < S - 1; ++i) n += stores[i];
    if (n >= STORES) {
      QPL_WAIT_VMCNT(LATER + STORES);
    } else {
      QPL_WAIT_VMCNT(LATER);
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = S - 2; i > 0; --i) stores[i] = stores[i - 1];
    stores[0] = 0;
  };
  // where a wavefront that owns nj row tiles finds its operands in stage st
  struct Source {
    const uint8_t *x0, *x1, *w0, *w1;
    const float *sx, *sw;
  };
  auto source = [&](int st, int nj) {
    const uint8_t* s = lds + st * STAGE;
    const uint8_t* x = s + XB + wm * 16 * nj * PR_ROW;
    const uint8_t* w = s + WB + wn * 16 * NI * PR_ROW;
    const float* f = reinterpret_cast<const float*>(s);
    return Source{x + at0, x + at1, w + at0, w + at1, f + wm * 16 * nj + r16, f + XR + ((wn * 16 * NO) >> 7)};
  };
  auto read_x = [&](const Source& s, int j) {
    fx[j & 1] = frag(s.x0 + 16 * PR_ROW * j, s.x1 + 16 * PR_ROW * j);
    sx[j & 1] = s.sx[16 * j];
  };
  auto read_w = [&](const Source& s, int i) { fw[i] = frag(s.w0 + 16 * PR_ROW * i, s.w1 + 16 * PR_ROW * i); };
  auto read_scales = [&](const Source& s) {
    sw[0] = s.sw[0];
    sw[1] = GATED ? s.sw[64] : sw[0];
  };

#pragma unroll
  for (int ahead = 0; ahead < S; ++ahead) {
    next_piece();
#pragma unroll
    for (int d = 0; d < LOADS; ++d) issue(d, args()->g.px, args()->g.K);
  }
  QPL_WAIT_VMCNT((S - 1) * LOADS);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

  // loads issued behind the sync, one after each of a piece's last MFMAs; the others follow between the first half of
  // the next piece's
  constexpr int EARLY = (LOADS + 2) / 3, LATE = LOADS - EARLY;
  // One piece, its first operands in registers.  first: of a tile, whose loads have been issued; last: of a tile, whose
  // next piece's operands are read when the accumulators have been stored and the registers are free.
  auto piece = [&](auto& acc, auto nj, auto first, auto last, int px, int pw) {
    constexpr int NJ = decltype(nj)::value, T = NI * NJ;
    constexpr bool FIRST = decltype(first)::value, LAST = decltype(last)::value;
    constexpr int LAG = 2;  // MFMAs between a tile's own and the fold of its sums
    // a tile's only piece keeps code of its own: merged with the first of several, the two parted between an MFMA and
    // the fold of its sums, with one wait state too few on one of the ways
    if constexpr (FIRST && LAST) asm volatile("; one piece" : "+v"(fx[0]));
    const int nxt = cur == S - 1 ? 0 : cur + 1;
    const Source now = source(cur, NJ);
    // a load's offset is made when it is issued: kept for all loads they would not fit the registers, and a reload
    // from memory would wait for every load in flight
    asm volatile("" : "+s"(px), "+s"(pw));
    f32x4 pr[3];
    float f[2][2];  // scales of row tile j and of either weight's column tiles
    auto fold = [&](auto tc) __attribute__((always_inline)) {
      constexpr int t = decltype(tc)::value, i = t % NI, j = t / NI;
      fold4(acc[i][j], pr[t % 3], f[j & 1][i >= NO ? 1 : 0]);
      // kept where it stands: the compiler would move all folds behind the sync's branches, and keep every sum till then
      asm volatile("" : "+v"(acc[i][j]));
    };
    static_for<0, NJ>([&](auto jc) __attribute__((always_inline)) {
      constexpr int j = decltype(jc)::value;
      f[j & 1][0] = sx[j & 1] * sw[0];
      f[j & 1][1] = GATED ? sx[j & 1] * sw[1] : f[j & 1][0];
      Source next;
      if constexpr (j + 1 < NJ) {
        read_x(now, j + 1);
      } else {
        sync();
        next_piece();
        if constexpr (!LAST) {
          next = source(nxt, NJ);
          read_x(next, 0);
          read_scales(next);
        }
      }
      static_for<0, NI>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value, t = NI * j + i;
        pr[t % 3] = mma(fw[i], fx[j & 1]);
        if constexpr (t >= LAG) fold(std::integral_constant<int, t - LAG>{});
        if constexpr (j + 1 == NJ) {
          if constexpr (!LAST) read_w(next, i);
#pragma unroll
          for (int d = 0; d < EARLY; ++d)
            if (d * NI / EARLY == i) issue(d, px, pw);
        } else if constexpr (!FIRST) {
#pragma unroll
          for (int d = 0; d < LATE; ++d)
            if (d * (T / 2) / LATE == t) issue(EARLY + d, px, pw);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    static_for<T - LAG, T>(fold);
    cur = nxt;
  };
  using Yes = std::integral_constant<bool, true>;
  using No = std::integral_constant<bool, false>;
  auto run_tile = [&](const Tile& t, auto nj) {
    constexpr int NJ = decltype(nj)::value;
    f32x4 acc[NI][NJ];
#pragma unroll
    for (int x = 0; x < NI; ++x)
#pragma unroll
      for (int y = 0; y < NJ; ++y) acc[x][y] = f32x4{};
    const int px = args()->g.px, pw = args()->g.K;
    const Source s = source(cur, NJ);
#pragma unroll
    for (int i = 0; i < NI; ++i) read_w(s, i);
    read_x(s, 0);
    read_scales(s);
    if (np == 1) {
      piece(acc, nj, Yes{}, Yes{}, px, pw);
    } else {
      piece(acc, nj, Yes{}, No{}, px, pw);
      for (int k = 2; k < np; ++k) piece(acc, nj, No{}, No{}, px, pw);
      piece(acc, nj, No{}, Yes{}, px, pw);
    }
    // before the output stores, because a load behind them could not be waited for without them
#pragma unroll
    for (int d = EARLY; d < LOADS; ++d) issue(d, px, pw);
    Args* a = args();
    const int64_t m0 = (int64_t)t.m0 + wm * 16 * NJ, n0 = (int64_t)t.n0 + wn * 16 * NO, m1 = (int64_t)t.m0 + t.rows,
                  N = a->g.N;
    EpiArgs e{};
    if constexpr ((EPI & EPI_QKV) != 0) {
#pragma unroll
      for (int i = 0; i < 3; ++i) e.qkv[i] = a->e.qkv[i];
      e.d = a->e.d;
      e.tokens = a->e.tokens;
      e.off = a->e.off;
      e.lg_hd = a->e.lg_hd;
    }
    uint16_t* y = a->y;
    int left = 0;
    if constexpr (GATED) {
      uint16_t *g = a->g.save[0], *u = a->g.save[1];
      if (g) {
        left += store16<NJ, NO, 0, false>(acc, m0, n0, m1, N, g, e);
        left += store16<NJ, NO, 0, false>(acc + NO, m0, n0, m1, N, u, e);
      }
#pragma unroll
      for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = gate_act<EPI>(acc[i][j][r]) * acc[i + NO][j][r];
          __builtin_amdgcn_sched_barrier(0);
        }
      left += store16<NJ, NO, 0, false>(acc, m0, n0, m1, N, y, e);
    } else {
      left = store16<NJ, NO, EPI, true>(acc, m0, n0, m1, N, y, e);
    }
    stores[0] = __builtin_amdgcn_readfirstlane(left);
  };
  for (int i = 0;; ++i) {
    const Tile t = tile(i);
    if (t.rows <= 0) break;  // none, or a part behind its tile's last row
    if (NJM <= 2 || t.rows > XR / 2) {
      run_tile(t, std::integral_constant<int, NJM>{});
    } else if (NJM <= 4 || t.rows > XR / 4) {
      if constexpr (NJM >= 4) run_tile(t, std::integral_constant<int, NJM / 2>{});
    } else {
      if constexpr (NJM >= 8) run_tile(t, std::integral_constant<int, NJM / 4>{});
    }
  }
  QPL_WAIT_VMCNT(0);
  QPL_WAIT_LGKM0();
}

// ---------------------------------------------------------------------------
// Launchers.
// ---------------------------------------------------------------------------
// The kernel for this epilogue: L::run<GATED, EPI>().
template <class L>
hipError_t with_epilogue(const L& l, bool gated, int kind) {
  if (gated) return kind == EPI_SILU ? l.template run<true, EPI_SILU>() : l.template run<true, EPI_GELU>();
  switch (kind) {
    case 0: return l.template run<false, 0>();
    case EPI_GELU: return l.template run<false, EPI_GELU>();
    case EPI_QKV: return l.template run<false, EPI_QKV>();
    default: return hipErrorInvalidValue;
  }
}

// Workgroups stride over column and row tiles past these numbers.
constexpr int64_t kDirectColumns = int64_t(1) << 21, kDirectRows = 65535;

template <int MT, int NT, int W, int U>
struct Direct {
  const Fp8bArgs& p;
  uint16_t* y;
  const EpiArgs& e;
  hipStream_t stream;
  template <bool GATED, int EPI>
  hipError_t run() const {
    if constexpr (GATED && NT == 1) return hipErrorInvalidValue;
    constexpr int N_T = GATED && NT > 1 ? NT / 2 : NT;
    const int64_t tn = (p.N + 16 * N_T - 1) / (16 * N_T), tm = (p.M + 16 * MT - 1) / (16 * MT);
    const dim3 grid((unsigned)(tn < kDirectColumns ? tn : kDirectColumns), (unsigned)(tm < kDirectRows ? tm : kDirectRows));
    hipLaunchKernelGGL((k_fp8b_direct<MT, N_T, W, U, GATED, EPI>), grid, dim3(64 * W), 0, stream, p, y, e);
    return hipGetLastError();
  }
};

struct Token {
  const uint16_t* x;
  const Fp8bArgs& p;
  uint16_t* y;
  const EpiArgs& e;
  hipStream_t stream;
  template <bool GATED, int EPI>
  hipError_t run() const {
    // one workgroup per CU at most, which quantizes once and takes 16 columns in each of its turns
    const int64_t n = (p.N + 15) / 16;
    hipLaunchKernelGGL((k_fp8b_token<GATED, EPI>), dim3((unsigned)(n < 256 ? n : 256)), dim3(64 * TOKEN_W), 0, stream, x,
                       p, y, e);
    return hipGetLastError();
  }
};

template <int WM, int WN, int NI, int NJM, int S>
struct Staged {
  using C = StagedShape<WM, WN, NI, NJM, S>;
  const Fp8bArgs& p;
  uint16_t* y;
  const EpiArgs& e;
  hipStream_t stream;
  template <bool GATED, int EPI>
  hipError_t run() const {
    if constexpr (GATED && NI == 2) {
      return hipErrorInvalidValue;
    } else {
      constexpr int COLS = GATED ? C::WR / 2 : C::WR;
      Fp8bStagedArgs a;
      a.g = p;
      a.tiles_m = (int)((p.M + C::XR - 1) / C::XR);
      a.tiles_n = (int)((p.N + COLS - 1) / COLS);
      const int64_t n = (int64_t)a.tiles_m * a.tiles_n * (NJM / 2), most = 256 * C::per_cu();
      a.nwg = (int)(n < most ? n : most);
      a.y = y;
      a.e = e;
      hipLaunchKernelGGL((k_fp8b_staged<WM, WN, NI, NJM, S, GATED, EPI>), dim3((unsigned)a.nwg), dim3(64 * C::W), 0, stream,
                         a);
      return hipGetLastError();
    }
  }
};

hipError_t launch_product(const Fp8bArgs& p, bool gated, int kind, uint16_t* y, const EpiArgs& e, hipStream_t stream) {
  switch (fp8b_shape(p.M, (int64_t)p.pieces * p.segs, gated ? 2 * p.N : p.N, gated)) {
    case 0: return with_epilogue(Direct<1, 1, 16, 2>{p, y, e, stream}, gated, kind);
    case 1: return with_epilogue(Direct<1, 2, 8, 2>{p, y, e, stream}, gated, kind);
    case 2: return with_epilogue(Direct<2, 2, 8, 2>{p, y, e, stream}, gated, kind);
    case 3: return with_epilogue(Staged<2, 2, 2, 2, 4>{p, y, e, stream}, gated, kind);
    case 4: return with_epilogue(Staged<2, 2, 4, 2, 3>{p, y, e, stream}, gated, kind);
    case 5: return with_epilogue(Staged<2, 4, 4, 4, 3>{p, y, e, stream}, gated, kind);
    default: return with_epilogue(Staged<2, 4, 4, 8, 2>{p, y, e, stream}, gated, kind);
  }
}

Fp8bArgs product_args(const Fp8bWeight* w, int n, int64_t M, int64_t K, int64_t N) {
  Fp8bArgs p{};
  for (int i = 0; i < 2; ++i) {
    p.w[i] = w[i < n ? i : 0].codes;
    p.ws[i] = w[i < n ? i : 0].scales;
  }
  p.M = M;
  p.N = N;
  p.K = (int)K;
  p.pieces = (int)((K + 127) / 128);
  p.segs = 1;
  return p;
}

// A grid's threads are counted in 32 bits, and the runtime launches what is left of more without an error: kernels with
// a workgroup for every four rows and chunk run on slices of so many rows, f(first row, rows, grid).
constexpr int64_t kMostBlocks = int64_t(1) << 23;

template <class F>
hipError_t row_slices(int64_t M, int64_t chunks, const F& f) {
  const int64_t each = kMostBlocks / chunks * 4;  // chunks: at most 2^20, of rows below 2^31
  for (int64_t r0 = 0; r0 < M; r0 += each) {
    const int64_t rows = M - r0 < each ? M - r0 : each;
    f(r0, rows, dim3((unsigned)((rows + 3) / 4 * chunks)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_quant_fp8b(const uint16_t* x, int64_t M, int64_t K, int64_t pitch, bool slab, uint8_t* xq, float* xs,
                             hipStream_t stream) {
  const int64_t chunks = (pitch / 8 + 64 * QV - 1) / (64 * QV);
  return row_slices(M, chunks, [&](int64_t r0, int64_t rows, dim3 grid) {
    if (slab) {
      hipLaunchKernelGGL(k_quant_fp8b<true>, grid, dim3(256), 0, stream, x + r0 * K, rows, M, K, pitch, (uint32_t)chunks,
                         xq + r0 * pitch, xs + r0);
    } else {
      hipLaunchKernelGGL(k_quant_fp8b<false>, grid, dim3(256), 0, stream, x + r0 * K, rows, M, K, pitch,
                         (uint32_t)chunks, xq + r0 * pitch, xs + r0 * ((K + 127) / 128));
    }
  });
}

hipError_t launch_quant_weight_fp8b(const uint16_t* w, int64_t N, int64_t K, uint8_t* wq, float* ws,
                                    hipStream_t stream) {
  const int64_t nb = (N + 127) / 128;
  const dim3 grid((unsigned)((K + 127) / 128), (unsigned)(nb < 65535 ? nb : 65535));
  hipLaunchKernelGGL(k_quant_weight_fp8b, grid, dim3(256), 0, stream, w, N, K, wq, ws);
  return hipGetLastError();
}

hipError_t launch_transpose_fp8b(const uint8_t* w, const float* ws, int64_t N, int64_t K, uint8_t* wt, float* wst,
                                 hipStream_t stream) {
  const int64_t nb = (N + 127) / 128;
  const dim3 grid((unsigned)((K + 127) / 128), (unsigned)(nb < 65535 ? nb : 65535));
  hipLaunchKernelGGL(k_transpose_fp8b, grid, dim3(256), 0, stream, w, ws, N, K, wt, wst);
  return hipGetLastError();
}

hipError_t launch_gated_backward(const uint16_t* dh, const uint16_t* g, const uint16_t* u, int64_t M, int64_t H,
                                 bool silu, uint16_t* dg, uint16_t* du, uint8_t* q, float* s, hipStream_t stream) {
  const int64_t chunks = ((H + 127) / 128 * 16 + 64 * GV - 1) / (64 * GV), pitch = 2 * ((H + 127) / 128 * 128);
  return row_slices(M, chunks, [&](int64_t r0, int64_t rows, dim3 grid) {
    const int64_t at = r0 * H;
    uint16_t* const og = dg ? dg + at : nullptr;
    uint16_t* const ou = du ? du + at : nullptr;
    if (silu) {
      hipLaunchKernelGGL(k_gated_backward<true>, grid, dim3(256), 0, stream, dh + at, g + at, u + at, rows, M, H, pitch,
                         (uint32_t)chunks, og, ou, q + r0 * pitch, s + r0);
    } else {
      hipLaunchKernelGGL(k_gated_backward<false>, grid, dim3(256), 0, stream, dh + at, g + at, u + at, rows, M, H, pitch,
                         (uint32_t)chunks, og, ou, q + r0 * pitch, s + r0);
    }
  });
}

bool fp8b_one_launch(int64_t M, int64_t K) { return fp8b_token_fits(M, K); }

hipError_t launch_fp8b_token(const uint16_t* x, const Fp8bWeight& w, int64_t M, int64_t K, int64_t N,
                             const Epilogue& ep, uint16_t* y, hipStream_t stream) {
  EpiArgs e;
  const int kind = epi_kind(ep, e);
  return with_epilogue(Token{x, product_args(&w, 1, M, K, N), y, e, stream}, false, kind);
}

hipError_t launch_gemm_fp8b(const uint8_t* xq, const float* xs, const Fp8bWeight& w, int64_t M, int64_t K, int64_t N,
                            const Epilogue& ep, uint16_t* y, hipStream_t stream) {
  EpiArgs e;
  const int kind = epi_kind(ep, e);
  Fp8bArgs p = product_args(&w, 1, M, K, N);
  p.x = xq;
  p.xs = xs;
  p.px = (int)fp8b_pitch(K);
  return launch_product(p, false, kind, y, e, stream);
}

hipError_t launch_fp8b_gated(const uint16_t* x, const uint8_t* xq, const float* xs, const Fp8bWeight (&w)[2], int64_t M,
                             int64_t K, int64_t H, bool silu, uint16_t* h, uint16_t* const (&save)[2],
                             hipStream_t stream) {
  const EpiArgs e{};
  Fp8bArgs p = product_args(w, 2, M, K, H);
  p.save[0] = save[0];
  p.save[1] = save[1];
  const int kind = silu ? EPI_SILU : EPI_GELU;
  if (fp8b_token_fits(M, K)) return with_epilogue(Token{x, p, h, e, stream}, true, kind);
  p.x = xq;
  p.xs = xs;
  p.px = (int)fp8b_pitch(K);
  return launch_product(p, true, kind, h, e, stream);
}

hipError_t launch_gemm_fp8b_pair(const uint8_t* xq, const float* xs, const Fp8bWeight (&w)[2], int64_t M, int64_t K,
                                 int64_t N, uint16_t* y, hipStream_t stream) {
  Fp8bArgs p = product_args(w, 2, M, K, N);
  p.x = xq;
  p.xs = xs;
  p.segs = 2;
  p.px = 2 * 128 * p.pieces;
  return launch_product(p, false, 0, y, EpiArgs{}, stream);
}

}  // namespace qpl
