// Pieces that the tiled GEMMs share: the order in which workgroups take tiles, the
// swizzle of an LDS stage and the epilogue that scales, activates, rounds and stores
// a tile.
#pragma once

#include <type_traits>

#include "qpl_dma.h"
#include "qpl_internal.h"

namespace qpl {

namespace {

// Rows of a 256-row tile that lie inside the matrix (rows_left = rows from the
// tile's first row to the matrix end).
__device__ __forceinline__ int64_t M_rows(int64_t rows_left) { return rows_left < 256 ? rows_left : 256; }

// Tile order.  The tile sequence walks groups of GROUP_M tile-rows column by column.
// Workgroups are dispatched round-robin over the 8 XCDs and each XCD has its own
// L2, so in every round of the persistent loop the 32 workgroups of one XCD take a
// contiguous run of 32 tiles of the sequence: a 4 x 8 block that shares 4
// activation slabs and 8 weight slabs in that XCD's L2.
constexpr int GROUP_M = 4;

// tm: rows of x per tile (256, or 128 for the INT4 GEMM); tiles are 256 columns wide.
__device__ __forceinline__ void tile_coords(int s, int tiles_m, int tiles_n, int64_t& m0, int64_t& n0,
                                            int tm = 256) {
  const int per_group = GROUP_M * tiles_n;
  const int g = s / per_group;
  const int first_m = g * GROUP_M;
  const int gm = min(tiles_m - first_m, GROUP_M);
  const int r = s - g * per_group;
  m0 = (int64_t)(first_m + r % gm) * tm;
  n0 = (int64_t)(r / gm) * 256;
}

// Position in the tile sequence of workgroup b's i-th tile (nwg workgroups).
__device__ __forceinline__ int tile_seq(int i, int b, int nwg) {
  return (nwg & 7) == 0 ? i * nwg + (b & 7) * (nwg >> 3) + (b >> 3) : i * nwg + b;
}

// A stage row of the paired-slab rings is one 128-byte line; its 16-byte chunk c sits
// at chunk c ^ (r % 8).
constexpr int PR_ROW = 128;                      // bytes per row per stage (two slabs)
__device__ __forceinline__ int proff(int r, int c) { return r * PR_ROW + ((c ^ (r & 7)) << 4); }

// f(integral_constant<int, I>) for I = B .. E - 1, expanded at compile time.
template <int B, int E, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for<B + 1, E>(f);
  }
}

// Epilogue kinds (bit flags; the Nunchaku post, "Introducing Nunchaku Lite", names
// fused QKV projections and fused GELU/MLP kernels as the model-specific paths of
// its original engine):
// * EPI_GELU: the tanh form of GELU on each fp32 result before the bf16 rounding;
// * EPI_QKV: the output row's three parts (columns [0, d), [d, 2d), [2d, 3d)) go to
//   three tensors [heads, tokens, head_dim] at a token offset, the layout attention
//   reads, instead of the row-major y.
constexpr int EPI_GELU = 1, EPI_QKV = 2;

struct EpiArgs {
  uint16_t* qkv[3];  // EPI_QKV: q, k, v
  int64_t d;         // EPI_QKV: columns per part (heads * head_dim)
  int64_t tokens;    // EPI_QKV: tokens per head
  int64_t off;       // EPI_QKV: token of output row 0
  int lg_hd;         // EPI_QKV: log2(head_dim)
};
// GELU, tanh form: v sigma(2u) with u = sqrt(2/pi) (v + 0.044715 v^3), since
// (1 + tanh u) / 2 = 1 / (1 + exp(-2u)).  exp2 and the reciprocal run on the
// transcendental unit; the exponent is t = -2 u log2(e) = v (C1 + C3 v^2).  Large
// negative v gives t = +inf and a result of -0; large positive v gives v.
constexpr float GELU_C1 = -0x1.26aec2p+1f;  // -2 sqrt(2/pi) log2(e), -2.3022082
constexpr float GELU_C3 = -0x1.a5a7d0p-4f;  // GELU_C1 * 0.044715, -0.10294324
__device__ __forceinline__ float gelu_tanh(float v) {
  const float t = v * __builtin_fmaf(GELU_C3, v * v, GELU_C1);
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}

// Destination of output element (m, n): y[m, n], or under EPI_QKV element
// n mod head_dim of head (n mod d) / head_dim of part n / d at token off + m.
template <int EPI>
__device__ __forceinline__ uint16_t* out_ptr(uint16_t* __restrict__ y, int64_t m, int64_t n, int64_t N,
                                             const EpiArgs& e) {
  if constexpr ((EPI & EPI_QKV) != 0) {
    const int part = (n >= e.d) + (n >= 2 * e.d);
    const int64_t c = n - part * e.d;
    const int64_t h = c >> e.lg_hd;
    return e.qkv[part] + (((h * e.tokens + e.off + m) << e.lg_hd) + (c & ((int64_t{1} << e.lg_hd) - 1)));
  } else {
    return y + m * N + n;
  }
}

// An accumulator element as fp32 (the integer GEMM's sums are rounded to 24 bits here,
// two orders of magnitude finer than the bf16 result).
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(int v) { return (float)v; }

// Epilogue of one tile: y = bf16(act((acc * rs(m)) * cs(n))), then the EPI output
// transform.  acc[i][j] holds y^T: its
// element r at lane l is row m = m0 + 128 wm + 32 j + l % 32, column
// n = n0 + 128 wn + 32 i + 8 (r / 4) + 4 (l / 32) + r % 4.  Lanes l and l + 32
// exchange halves (V_PERMLANE32_SWAP) so that each lane holds eight consecutive
// columns of one row and stores them as one 16-byte segment.  NJ: 32-row blocks
// per wavefront (4 for a 256-row tile, 2 for a 128-row half tile, whose rows are
// m0 + 64 wm + 32 j + l % 32); NI: 32-column blocks per wavefront (4: columns
// n0 + 128 wn + ..., wn in 0..1; 2: n0 + 64 wn + ..., wn in 0..3).  Returns the
// number of store instructions left in flight: 2 NJ NI on the interior path, 0 on
// the edge path (which checks every element and drains its stores).  ANY: rows of y may
// start at any element, and 16-byte segments are stored at 2-byte alignment.
struct __attribute__((packed, aligned(2))) Segment {
  u32x4 v;
};
template <int NJ, int NI, int EPI, bool FAST, bool ANY, class Acc, class RowScale, class ColScale>
__device__ __forceinline__ void store_tile_path(const Acc& acc, int wm, int wn, int lane, int64_t m0, int64_t n0,
                                                int64_t M, int64_t N, uint16_t* __restrict__ y, const RowScale& rs,
                                                const ColScale& cs, const EpiArgs& e) {
  // unrolled at compile time: with a heavy epilogue the body exceeds what the
  // unroll pragma accepts, and a rolled loop would index acc dynamically (scratch)
  static_for<0, NJ>([&](auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    const int mr = wm * 32 * NJ + j * 32 + (lane & 31);
    const float fr = rs(mr);
    const int64_t m = m0 + mr;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int gp = 0; gp < 2; ++gp) {
        uint32_t w[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int g = 2 * gp + h;
          const f32x4 fc = cs(wn * 32 * NI + i * 32 + g * 8 + (lane >> 5) * 4);
          const auto& a = acc[i][j];
          float o[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            o[c] = (to_f32(a[g * 4 + c]) * fr) * fc[c];
            if constexpr ((EPI & EPI_GELU) != 0) o[c] = gelu_tanh(o[c]);
          }
          w[h][0] = pack_bf16(o[0], o[1]);
          w[h][1] = pack_bf16(o[2], o[3]);
        }
        const auto r0 = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
        const auto r1 = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
        const u32x4 v = u32x4{r0[0], r1[0], r0[1], r1[1]};
        const int64_t n = n0 + wn * 32 * NI + i * 32 + (2 * gp + (lane >> 5)) * 8;
        // the segment's eight columns stay inside one head (head_dim >= 8, n % 8 == 0)
        uint16_t* dst = out_ptr<EPI>(y, m, n, N, e);
        if constexpr (FAST && !ANY) {
          *reinterpret_cast<u32x4*>(dst) = v;
        } else if constexpr (FAST) {
          reinterpret_cast<Segment*>(dst)->v = v;
        } else if (m < M) {
          const uint32_t el[4] = {v.x, v.y, v.z, v.w};
          if (!ANY && (N & 7) == 0 && n + 8 <= N) {
            *reinterpret_cast<u32x4*>(dst) = v;
          } else if (ANY && n + 8 <= N) {
            reinterpret_cast<Segment*>(dst)->v = v;
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (n + c < N) dst[c] = (uint16_t)(el[c >> 1] >> (16 * (c & 1)));
          }
        }
      }
  });
}

template <int NJ, int NI = 4, int EPI = 0, bool ANY = false, class Acc, class RowScale, class ColScale>
__device__ __forceinline__ int store_tile(const Acc& acc, int wm, int wn, int lane, int64_t m0, int64_t n0,
                                          int64_t M, int64_t N, uint16_t* __restrict__ y, const RowScale& rs,
                                          const ColScale& cs, const EpiArgs& e = EpiArgs{}) {
  // interior: the wavefront's rows and columns all inside the matrix; the two paths
  // are separate code, so the interior one has no per-segment branches
  const bool fast = m0 + (wm + 1) * 32 * NJ <= M && n0 + (wn + 1) * 32 * NI <= N && (ANY || (N & 7) == 0);
  if (fast) {
    store_tile_path<NJ, NI, EPI, true, ANY>(acc, wm, wn, lane, m0, n0, M, N, y, rs, cs, e);
    return 2 * NJ * NI;
  }
  store_tile_path<NJ, NI, EPI, false, ANY>(acc, wm, wn, lane, m0, n0, M, N, y, rs, cs, e);
  QPL_WAIT_VMCNT(0);
  return 0;
}

}  // namespace

// Kernel-side epilogue arguments and kind (EPI flags) of a launch.
static int epi_kind(const Epilogue& ep, EpiArgs& e) {
  e = EpiArgs{};
  int k = ep.gelu ? EPI_GELU : 0;
  if (ep.qkv[0]) {
    k |= EPI_QKV;
    for (int i = 0; i < 3; ++i) e.qkv[i] = ep.qkv[i];
    e.d = ep.d;
    e.tokens = ep.tokens;
    e.off = ep.off;
    e.lg_hd = ep.lg_hd;
  }
  return k;
}

}  // namespace qpl
