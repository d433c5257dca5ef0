// 8-bit integer linears for gfx950: y = act((q_x q_w^T) s_x s_w) with a scale for each
// row of x (token) and each row of W (output channel), dense or grouped by expert.
//
// Quantizer.  a = max_k |x[m, k]|, s = fp32(a / 127), q = rint(127 x / a), ties to even.
// The sums of products are int32 and exact for K <= 2^17 (127 * 128 * 2^17 < 2^31), so a
// result does not depend on how K is split over wavefronts or workgroups.
#include "qpl_gemm.h"
#include "qpl_int8_shape.h"

namespace qpl {

namespace {

// ---------------------------------------------------------------------------
// Row quantizer: one wavefront per row and four rows per workgroup, or (SPLIT) a workgroup
// per row when there are too few rows to fill the chip; VPT 16-byte vectors per lane stay in
// registers between the two passes (VPT == 0, for rows that SPLIT does not hold either, streams the row twice).
//
// The code is rint of the exact quotient 127 x / a.  x = i 2^p and a = j 2^q have 8-bit
// integers i, j, so 127 x / a either is a tie (k + 1/2, at most 8 significant bits) or
// differs from every tie by more than 1 / (254 * 255) = 1.5e-5 of itself: the numerator
// of the difference is a nonzero integer over 2 * 127 i.  t = x * fp32(127 / a) is off
// by less than 2^-22.9 of itself.  Rounding t to 16 fraction bits (off by at most 2^-17 =
// 7.6e-6) puts a tie back on the tie and moves nothing across one; then adding 1.5 * 2^23
// rounds to the nearest integer, ties to even, and leaves the code in the low byte.
// ---------------------------------------------------------------------------
struct RowCode {
  float s, r;  // scale; 127 / a, or 127 / (a 2^100) for rows whose 127 / a might overflow
  bool tiny;   // those rows
};

__device__ __forceinline__ RowCode row_code(float amax) {
  RowCode d;
  d.s = amax / 127.0f;
  d.tiny = amax < 0x1p-100f;
  d.r = amax > 0.0f ? 127.0f / (d.tiny ? amax * 0x1p100f : amax) : 0.0f;
  return d;
}

// Bits whose low byte is the code of x.
__device__ __forceinline__ uint32_t code_bits(float x, float r) {
  const uint32_t t = (__float_as_uint(x * r) + 0x40u) & 0xFFFFFF80u;
  return __float_as_uint(__uint_as_float(t) + 0x1.8p23f);
}

// Codes of two bf16 pairs, in order.
__device__ __forceinline__ uint32_t code_word(uint32_t a, uint32_t b, const RowCode& d) {
  float x0 = bf16_lo(a), x1 = bf16_hi(a), x2 = bf16_lo(b), x3 = bf16_hi(b);
  if (d.tiny) {
    x0 *= 0x1p100f;
    x1 *= 0x1p100f;
    x2 *= 0x1p100f;
    x3 *= 0x1p100f;
  }
  const uint32_t lo = __builtin_amdgcn_perm(code_bits(x1, d.r), code_bits(x0, d.r), 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(code_bits(x3, d.r), code_bits(x2, d.r), 0x04000C0Cu);
  return lo | hi;
}

__device__ __forceinline__ u32x2 code_vec(const u32x4& v, const RowCode& d) {
  return u32x2{code_word(v.x, v.y, d), code_word(v.z, v.w, d)};
}

__device__ __forceinline__ uint32_t vec_absmax8(const u32x4& v, uint32_t m) {
  return absmax_acc(absmax_acc(absmax_acc(absmax_acc(m, v.x), v.y), v.z), v.w);
}

__device__ __forceinline__ u32x4 smooth_vec(const u32x4& v, const float* __restrict__ lam) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(lam), b = *reinterpret_cast<const f32x4*>(lam + 4);
  return u32x4{smooth_pair(v.x, a[0], a[1]), smooth_pair(v.y, a[2], a[3]), smooth_pair(v.z, b[0], b[1]),
               smooth_pair(v.w, b[2], b[3])};
}

// Codes and scale of the row at `src` (nullptr: a row of zeros) into row `row`, rows `pitch`
// codes apart.  REUSED: other rows are made of the same source, which should stay in the
// caches.  SPLIT: the workgroup's four wavefronts share the row.
template <int VPT, bool SMOOTH, bool REUSED, bool SPLIT>
__device__ __forceinline__ void quant_row(const uint16_t* __restrict__ src, int64_t row, int64_t K, int64_t pitch,
                                          const float* __restrict__ lam, int8_t* __restrict__ xq,
                                          float* __restrict__ xs) {
  constexpr int STEP = SPLIT ? 256 : 64;
  const int first = SPLIT ? threadIdx.x : threadIdx.x & 63;
  const int64_t nv = K >> 3;
  u32x2* qr = reinterpret_cast<u32x2*>(xq + row * pitch);
  if (REUSED && !src) {
    for (int64_t j = first; j < nv; j += STEP) qr[j] = u32x2{0u, 0u};
    if (first == 0) xs[row] = 0.0f;
    return;
  }
  const u32x4* xr = reinterpret_cast<const u32x4*>(src);
  auto load = [&](int64_t j) {
    const u32x4 v = REUSED ? xr[j] : __builtin_nontemporal_load(xr + j);
    return SMOOTH ? smooth_vec(v, lam + 8 * j) : v;
  };
  auto row_max = [&](uint32_t am) {
    float a = wave_max(absmax_value(am));
    if constexpr (SPLIT) {
      __shared__ float part[4];
      __syncthreads();  // the row before is done with part
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
      __syncthreads();
      a = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    }
    return a;
  };
  uint32_t am = 0;
  if constexpr (VPT > 0) {
    u32x4 v[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t j = first + STEP * i;
      v[i] = j < nv ? load(j) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) am = vec_absmax8(v[i], am);
    const RowCode d = row_code(row_max(am));
    if (first == 0) xs[row] = d.s;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t j = first + STEP * i;
      if (j < nv) qr[j] = code_vec(v[i], d);
    }
  } else {
    for (int64_t j = first; j < nv; j += STEP) am = vec_absmax8(load(j), am);
    const RowCode d = row_code(row_max(am));
    if (first == 0) xs[row] = d.s;
    for (int64_t j = first; j < nv; j += STEP) qr[j] = code_vec(load(j), d);
  }
}

// One row tile of a grouped product: rows [m0, m1) of expert e.
struct RowTile {
  int m0, m1, e, pad;
};

// The experts' rows cut into tiles of `tm` rows that never cross an expert, in order;
// count[0] = their number (at most cap).  offsets [E + 1] are clamped into [0, R] and counted in
// 64 bits, so whatever they hold no tile leaves the R rows and no write the array.  One workgroup.
__device__ __forceinline__ void build_row_tiles(const int* offsets, int E, int R, int tm, int cap,
                                                int* __restrict__ count, RowTile* __restrict__ tiles) {
  __shared__ int64_t wsum[4];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int64_t base = 0;
  for (int e0 = 0; e0 < E; e0 += 256) {
    const int e = e0 + (int)threadIdx.x;
    int lo = 0, hi = 0;
    if (e < E) {
      lo = min(max(offsets[e], 0), R);
      hi = min(max(offsets[e + 1], lo), R);
    }
    const int n = (hi - lo) / tm + ((hi - lo) % tm != 0);
    int64_t sum = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up(sum, d, 64);
      if (lane >= d) sum += o;
    }
    if (lane == 63) wsum[wv] = sum;
    __syncthreads();
    int64_t first = base + sum - n;
    for (int w = 0; w < 4; ++w) {
      if (w < wv) first += wsum[w];
      base += wsum[w];
    }
    // each lane the tiles of its expert, or the whole wavefront those of an expert with many
    if (n <= 4) {
      for (int i = 0; i < n && first + i < cap; ++i)
        tiles[first + i] = RowTile{lo + i * tm, i + 1 < n ? lo + (i + 1) * tm : hi, e, 0};
    }
    for (uint64_t many = __ballot(n > 4); many != 0; many &= many - 1) {
      const int l = __ffsll((unsigned long long)many) - 1;
      const int ln = __shfl(n, l, 64), llo = __shfl(lo, l, 64), lhi = __shfl(hi, l, 64), le = __shfl(e, l, 64);
      const int64_t lfirst = __shfl(first, l, 64);
      for (int i = lane; i < ln && lfirst + i < cap; i += 64)
        tiles[lfirst + i] = RowTile{llo + i * tm, i + 1 < ln ? llo + (i + 1) * tm : lhi, le, 0};
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) count[0] = (int)(base < cap ? base : cap);
}

struct TilePlan {
  const int* offsets;
  int E, R, tm, cap;
  int* count;
  RowTile* tiles;
};

// GROUPED: workgroup 0 cuts the experts' rows into tiles.  GATHER: row i is x[row_index[i]] (a row of
// zeros for an index outside x).
template <int VPT, bool SMOOTH, bool GROUPED, bool GATHER, bool SPLIT>
__global__ __launch_bounds__(256) void k_quant_int8(const uint16_t* __restrict__ x, int64_t rows_x, int64_t rows,
                                                    int64_t K, int64_t pitch, const float* __restrict__ lam,
                                                    const int* __restrict__ row_index, int8_t* __restrict__ xq,
                                                    float* __restrict__ xs, TilePlan plan) {
  int64_t blk = blockIdx.x, nblk = gridDim.x;
  if constexpr (GROUPED) {
    // workgroup 0 cuts the experts' rows into tiles for the product that follows
    if (blk == 0) {
      build_row_tiles(plan.offsets, plan.E, plan.R, plan.tm, plan.cap, plan.count, plan.tiles);
      return;
    }
    blk -= 1;
    nblk -= 1;
  }
  constexpr int ROWS = SPLIT ? 1 : 4;  // rows of a workgroup
  for (int64_t row = blk * ROWS + (SPLIT ? 0 : threadIdx.x >> 6); row < rows; row += nblk * ROWS) {
    int64_t from = row;
    if constexpr (GATHER) {
      from = row_index[row];
      if (from >= rows_x) from = -1;
    }
    quant_row<VPT, SMOOTH, GATHER, SPLIT>(from < 0 ? nullptr : x + from * K, row, K, pitch, lam, xq, xs);
  }
}

// ---------------------------------------------------------------------------
// Plan and first quantizer of the MLP of experts for few choices, in one launch: with up to
// FRONT_N of them a workgroup finds the place of its choice by looking at all others, and writes
// that token's codes there.  Workgroup 0 makes the offsets and the row tiles.  The search grows with
// the square of the choices; measured, us in a graph (this launch / plan and quantizer), for 64 experts:
//   choices   28       256      1024     2048       4096
//   K 256     3.3/5.1  3.4/5.5  4.1/6.2  6.0/6.2    11.3/7.3
//   K 2048    3.3/5.3  3.5/5.7  4.4/6.7  7.1/7.9    13.3/9.6
//   K 8192    4.4/5.9  4.7/6.5  6.3/8.6  13.3/13.1  28.1/21.7
// and for 1024 experts 1024 choices of K = 2048 5.9/8.4, 2048 of them 7.0/8.6.  FRONT_E experts are what
// workgroup 0 sums at four per thread.
// ---------------------------------------------------------------------------
constexpr int FRONT_N = 1024, FRONT_E = 1024;

__global__ __launch_bounds__(256) void k_int8_moe_front(const int* __restrict__ ids, int n, int topk,
                                                        const uint16_t* __restrict__ x, int64_t K, int64_t pitch,
                                                        int8_t* __restrict__ xq, float* __restrict__ xs,
                                                        int* __restrict__ slot, int* __restrict__ offsets,
                                                        TilePlan plan) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, E = plan.E;
  if (blockIdx.x == 0) {
    __shared__ int first[FRONT_E + 1];
    __shared__ int sums[4];
    for (int e = threadIdx.x; e <= E; e += 256) first[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += 256)
      if ((uint32_t)ids[i] < (uint32_t)E) atomicAdd(&first[ids[i]], 1);
    __syncthreads();
    // exclusive sums, four experts per thread (FRONT_E = 4 * 256)
    int c[4], mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c[k] = 4 * (int)threadIdx.x + k < E ? first[4 * threadIdx.x + k] : 0;
      mine += c[k];
    }
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d, 64);
      if (lane >= d) sum += o;
    }
    if (lane == 63) sums[wv] = sum;
    __syncthreads();
    int at = sum - mine;
    for (int w = 0; w < wv; ++w) at += sums[w];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (4 * (int)threadIdx.x + k <= E) first[4 * threadIdx.x + k] = at;
      at += c[k];
    }
    if (threadIdx.x == 255 && E == FRONT_E) first[E] = at;
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += 256) offsets[e] = first[e];
    build_row_tiles(first, E, n, plan.tm, plan.cap, plan.count, plan.tiles);
    return;
  }
  __shared__ int below[4];
  const int i = blockIdx.x - 1;
  const uint32_t own = (uint32_t)ids[i];
  if (own >= (uint32_t)E) {
    if (threadIdx.x == 0) slot[i] = -1;
    return;
  }
  int count = 0;
  for (int j = threadIdx.x; j < n; j += 256) {
    const uint32_t v = (uint32_t)ids[j];
    count += v < own || (v == own && j < i);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) count += __shfl_xor(count, d, 64);
  if (lane == 0) below[wv] = count;
  __syncthreads();
  const int place = below[0] + below[1] + below[2] + below[3];
  if (threadIdx.x == 0) slot[i] = place;
  quant_row<0, false, true, true>(x + (int64_t)(i / topk) * K, place, K, pitch, nullptr, xq, xs);
}

constexpr int64_t kQuantBlocks = int64_t(1) << 22;  // workgroups stride over rows past this many

template <bool SMOOTH, bool GROUPED, bool GATHER, bool SPLIT>
hipError_t launch_quant_rows(const uint16_t* x, int64_t rows_x, int64_t rows, int64_t K, int64_t pitch,
                             const float* lam, const int* row_index, int8_t* xq, float* xs, const TilePlan& plan,
                             hipStream_t stream) {
  const int64_t per_lane = SPLIT ? (K / 8 + 255) / 256 : (K / 8 + 63) / 64;
  const int64_t blocks = SPLIT ? rows : (rows + 3) / 4;
  const dim3 grid((unsigned)((blocks < kQuantBlocks ? blocks : kQuantBlocks) + (GROUPED ? 1 : 0))), block(256);
#define QPL_CASE(V)                                                                                                   \
  if (per_lane <= V || V == 0) {                                                                                      \
    hipLaunchKernelGGL((k_quant_int8<V, SMOOTH, GROUPED, GATHER, SPLIT>), grid, block, 0, stream, x, rows_x, rows, K, \
                       pitch, lam, row_index, xq, xs, plan);                                                          \
    return hipGetLastError();                                                                                         \
  }
  if constexpr (SPLIT) {
    QPL_CASE(1) QPL_CASE(2) QPL_CASE(4) QPL_CASE(8) QPL_CASE(0)
  } else {
    QPL_CASE(1) QPL_CASE(2) QPL_CASE(4) QPL_CASE(8) QPL_CASE(16) QPL_CASE(24)  // split_rows takes the longer ones
  }
#undef QPL_CASE
  return hipErrorInvalidValue;
}

template <bool SMOOTH, bool GROUPED, bool GATHER>
hipError_t launch_quant(const uint16_t* x, int64_t rows_x, int64_t rows, int64_t K, int64_t pitch, const float* lam,
                        const int* row_index, int8_t* xq, float* xs, const TilePlan& plan, hipStream_t stream) {
  return split_rows(rows, K, GATHER) ? launch_quant_rows<SMOOTH, GROUPED, GATHER, true>(
                                           x, rows_x, rows, K, pitch, lam, row_index, xq, xs, plan, stream)
                                     : launch_quant_rows<SMOOTH, GROUPED, GATHER, false>(
                                           x, rows_x, rows, K, pitch, lam, row_index, xq, xs, plan, stream);
}

// ---------------------------------------------------------------------------
// The product without LDS staging.  A workgroup of W wavefronts owns 16 NT columns
// of y (rows of the weight) and 16 MT rows; its wavefronts take the 128-byte pieces of K in
// turn, each lane loading its MFMA operands (V_MFMA_I32_16X16X64_I8, 16 bytes per lane)
// straight from memory, and their int32 sums meet in LDS.
//
// The operands are swapped (the MFMA computes y^T), so a lane holds four consecutive
// columns of one row.  Row r of an operand and bytes 64 s + 16 (l / 16) of the piece go
// to lane l with l % 16 = r.  Rows past an operand's end and bytes past K read as zeros.
// ---------------------------------------------------------------------------
struct Int8Args {
  const int8_t* x;  // [rows, K], px apart
  const int8_t* w;  // [N, K], or [E, N, K]
  const float* xs;
  const float* ws;  // [N], or [E, N]
  int64_t M, N;
  int K, px;
  int64_t tiles_m, tiles_n;
  const int* count;      // grouped: number of row tiles
  const RowTile* tiles;  // grouped: the row tiles
};

// Four outputs stored at 2-byte alignment: rows of y may start at any element.
struct __attribute__((packed, aligned(2))) Segment4 {
  u32x2 v;
};

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, (int)kRawBufferWord3);
}

// The wait states between the last MFMAs and the first reader of their results (8 for 16 x 16, 12
// for 32 x 32).  They are spelled out: a build of the direct kernel had none on the path out of its
// loop, and stored sums without the last MFMA's share.  The empty statements take and return the
// accumulators and, like the s_nop, stay in order, so the MFMAs come before it and the readers behind it.
template <int MT, int NT>
__device__ __forceinline__ void settle(i32x4 (&acc)[MT][NT]) {
  auto pass = [&]() {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(acc[i][j]));
  };
  pass();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  pass();
}

// Outputs (m, n .. n + 3) of the sums, if m < m1, as far as n < N.
template <int EPI>
__device__ __forceinline__ void store_four(uint16_t* __restrict__ y, int64_t m, int64_t m1, int64_t n, int64_t N,
                                           const i32x4& sum, float sx, const float* __restrict__ ws,
                                           const EpiArgs& e) {
  if (m >= m1 || n >= N) return;
  float o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    o[k] = ((float)sum[k] * sx) * ws[n + k < N ? n + k : n];
    if constexpr ((EPI & EPI_GELU) != 0) o[k] = gelu_tanh(o[k]);
  }
  uint16_t* dst = out_ptr<EPI>(y, m, n, N, e);
  const uint32_t w0 = pack_bf16(o[0], o[1]), w1 = pack_bf16(o[2], o[3]);
  if (n + 4 <= N) {
    reinterpret_cast<Segment4*>(dst)->v = u32x2{w0, w1};
  } else {
    dst[0] = (uint16_t)w0;
    if (n + 1 < N) dst[1] = (uint16_t)(w0 >> 16);
    if (n + 2 < N) dst[2] = (uint16_t)w1;
  }
}

// U: pieces of a wavefront in flight together.
template <int MT, int NT, int W, int U, int EPI, bool GROUPED>
__global__ __launch_bounds__(64 * W) void k_int8_direct(Int8Args p, uint16_t* __restrict__ Y, EpiArgs e) {
  __shared__ i32x4 red[W][MT * NT][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t tiles_m = GROUPED ? p.count[0] : p.tiles_m;
  const int pieces = (p.K + 127) >> 7;
  for (int64_t tm = blockIdx.y; tm < tiles_m; tm += gridDim.y) {
    for (int64_t tn = blockIdx.x; tn < p.tiles_n; tn += gridDim.x) {
      const int64_t n0 = tn * 16 * NT;
      int64_t m0, m1;
      const int8_t* w = p.w;
      const float* wsc = p.ws;
      if constexpr (GROUPED) {
        const RowTile rt = p.tiles[tm];
        m0 = rt.m0;
        m1 = rt.m1;
        w += (int64_t)rt.e * p.N * p.K;
        wsc += (int64_t)rt.e * p.N;
      } else {
        m0 = tm * 16 * MT;
        m1 = p.M - m0 < 16 * MT ? p.M : m0 + 16 * MT;
      }
      const int64_t nr = p.N - n0 < 16 * NT ? p.N - n0 : 16 * NT;
      const __amdgpu_buffer_rsrc_t dx = make_rsrc(p.x + m0 * p.px, (m1 - m0) * p.px);
      const __amdgpu_buffer_rsrc_t dw = make_rsrc(w + n0 * p.K, nr * p.K);
      i32x4 acc[MT][NT];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
      for (int c = wv; c < pieces; c += W * U) {
        i32x4 fx[U][2][MT], fw[U][2][NT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int k = (c + u * W) * 128 + 64 * s + 16 * q;
            const bool in = k < p.K;
#pragma unroll
            for (int j = 0; j < NT; ++j)
              fw[u][s][j] = load16(dw, in ? (uint32_t)((16 * j + r16) * p.K + k) : kOutOfRange);
#pragma unroll
            for (int i = 0; i < MT; ++i)
              fx[u][s][i] = load16(dx, in ? (uint32_t)((16 * i + r16) * p.px + k) : kOutOfRange);
          }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int j = 0; j < NT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][s][j], fx[u][s][i], acc[i][j], 0, 0, 0);
      }
      settle(acc);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) red[wv][i * NT + j][lane] = acc[i][j];
      __syncthreads();
      // vector v: tile v / 64 (row block i, column block j), lane v % 64's four columns
      for (int v = threadIdx.x; v < MT * NT * 64; v += 64 * W) {
        const int tile = v >> 6, l = v & 63;
        i32x4 sum = red[0][tile][l];
#pragma unroll
        for (int k = 1; k < W; ++k) sum += red[k][tile][l];
        const int64_t m = m0 + 16 * (tile / NT) + (l & 15);
        const int64_t n = n0 + 16 * (tile % NT) + 4 * (l >> 4);
        store_four<EPI>(Y, m, m1, n, p.N, sum, m < m1 ? p.xs[m] : 0.0f, wsc, e);
      }
      __syncthreads();
    }
  }
}

// Workgroups stride over column and row tiles past these numbers.
constexpr int64_t kDirectColumns = int64_t(1) << 21, kDirectRows = 65535;

template <int MT, int NT, int W, int U, bool GROUPED>
hipError_t launch_direct(Int8Args p, int64_t row_tiles, const Epilogue& ep, uint16_t* y, hipStream_t stream) {
  p.tiles_m = row_tiles;
  p.tiles_n = (p.N + 16 * NT - 1) / (16 * NT);
  const dim3 grid((unsigned)(p.tiles_n < kDirectColumns ? p.tiles_n : kDirectColumns),
                  (unsigned)(row_tiles < kDirectRows ? row_tiles : kDirectRows));
  const dim3 block(64 * W);
  EpiArgs e;
  switch (epi_kind(ep, e)) {
    case 0: hipLaunchKernelGGL((k_int8_direct<MT, NT, W, U, 0, GROUPED>), grid, block, 0, stream, p, y, e); break;
    case EPI_GELU:
      hipLaunchKernelGGL((k_int8_direct<MT, NT, W, U, EPI_GELU, GROUPED>), grid, block, 0, stream, p, y, e);
      break;
    case EPI_QKV:
      if constexpr (!GROUPED) {
        hipLaunchKernelGGL((k_int8_direct<MT, NT, W, U, EPI_QKV, false>), grid, block, 0, stream, p, y, e);
        break;
      }
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// A few rows (single tokens) in one launch: as the direct kernel, but every workgroup quantizes
// the M <= 16 rows itself, into LDS, while its first weight bytes are on their way.  The
// quantizer's launch and the wait for it cost more than the repeated work: 1 x 4096 x 4096 takes
// 5.6 us, the two launches 6.1 + 5.5 us.
// A row is parts of 64 vectors of 8 elements; wavefront w takes the parts w, w + 16, ... of all
// rows, up to TOKEN_SLOTS of them.
// ---------------------------------------------------------------------------
constexpr int TOKEN_W = 16, TOKEN_SLOTS = TOKEN_PARTS / TOKEN_W, TOKEN_BYTES = TOKEN_PARTS * 512;

template <bool SMOOTH, int EPI>
__global__ __launch_bounds__(64 * TOKEN_W) void k_int8_token(const uint16_t* __restrict__ x,
                                                             const float* __restrict__ lam, Int8Args p,
                                                             uint16_t* __restrict__ Y, EpiArgs e) {
  constexpr int W = TOKEN_W, U = 2;
  __shared__ __attribute__((aligned(16))) uint8_t codes[TOKEN_BYTES];  // [M, K]
  __shared__ i32x4 red[W][64];
  __shared__ float part[TOKEN_PARTS];
  __shared__ float scale[16];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r16 = lane & 15, q = lane >> 4;
  const int M = (int)p.M, nv = p.K >> 3;
  const int parts = (nv + 63) >> 6;  // of a row
  // part / parts by a reciprocal, exact for the numbers up to 32 that occur
  const int rcp = (65536 + parts - 1) / parts;
  const int pieces = (p.K + 127) >> 7;
  int64_t n0 = (int64_t)blockIdx.x * 16;
  __amdgpu_buffer_rsrc_t dw;
  i32x4 fw[U][2];
  auto rows_of = [&](int64_t n) {
    const int64_t nr = p.N - n < 16 ? p.N - n : 16;
    dw = make_rsrc(p.w + n * p.K, nr * p.K);
  };
  auto load_w = [&](int c) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int k = (c + u * W) * 128 + 64 * s + 16 * q;
        fw[u][s] = load16(dw, k < p.K ? (uint32_t)(r16 * p.K + k) : kOutOfRange);
      }
  };
  // the rows' vectors, then (behind them, so that they do not wait for it) the first weight bytes
  u32x4 v[TOKEN_SLOTS];
#pragma unroll
  for (int t = 0; t < TOKEN_SLOTS; ++t) {
    const int u = wv + W * t, row = (u * rcp) >> 16, j = (u - row * parts) * 64 + lane;
    const bool in = row < M && j < nv;
    v[t] = in ? reinterpret_cast<const u32x4*>(x + (int64_t)row * p.K)[j] : u32x4{0u, 0u, 0u, 0u};
    if (SMOOTH && in) v[t] = smooth_vec(v[t], lam + 8 * (int64_t)j);
  }
  rows_of(n0);
  load_w(wv);
#pragma unroll
  for (int t = 0; t < TOKEN_SLOTS; ++t) {
    const float a = wave_max(absmax_value(vec_absmax8(v[t], 0u)));
    if (lane == 0) part[wv + W * t] = a;
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < TOKEN_SLOTS; ++t) {
    const int u = wv + W * t, row = (u * rcp) >> 16, sub = u - row * parts, j = sub * 64 + lane;
    if (row >= M) break;
    const RowCode rc = row_code(wave_max(lane < parts ? part[row * parts + lane] : 0.0f));
    if (sub == 0 && lane == 0) scale[row] = rc.s;
    if (j < nv) reinterpret_cast<u32x2*>(codes + row * p.K)[j] = code_vec(v[t], rc);
  }
  __syncthreads();
  for (;;) {
    i32x4 acc[1][1] = {{i32x4{0, 0, 0, 0}}};
    for (int c = wv; c < pieces; c += W * U) {
      if (c != wv) load_w(c);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int k = (c + u * W) * 128 + 64 * s + 16 * q;
          i32x4 fx{0, 0, 0, 0};
          if (r16 < M && k < p.K) fx = *reinterpret_cast<const i32x4*>(codes + r16 * p.K + k);
          acc[0][0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][s], fx, acc[0][0], 0, 0, 0);
        }
    }
    settle(acc);
    red[wv][lane] = acc[0][0];
    // the next columns' first weight bytes
    const int64_t next = n0 + (int64_t)gridDim.x * 16;
    if (next < p.N) {
      rows_of(next);
      load_w(wv);
    }
    __syncthreads();
    if (threadIdx.x < 64) {
      i32x4 sum = red[0][lane];
#pragma unroll
      for (int k = 1; k < W; ++k) sum += red[k][lane];
      store_four<EPI>(Y, r16, M, n0 + 4 * q, p.N, sum, r16 < M ? scale[r16] : 0.0f, p.ws, e);
    }
    n0 = next;
    if (n0 >= p.N) break;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// The product through LDS, for enough rows to reuse the weight.  A workgroup of four
// wavefronts (2 x 2) owns 64 NJM rows of x by 64 NI columns; a wavefront
// owns 32 NJ x 32 NI (V_MFMA_I32_32X32X32_I8, int32 accumulators).  Workgroups are
// persistent; K is walked in 128-byte pieces of both operands, S stages of them in
// LDS, filled by buffer_load_dwordx4 ... lds: piece P + S - 1's loads are issued between
// piece P's MFMAs, so they have S - 1 pieces' time to arrive.  The pieces of all of a
// workgroup's tiles form one stream.
//
// A tile with at most half (a quarter) of its rows present, an expert's last one for
// instance, runs with NJ = NJM / 2 (/ 4), so that its MFMAs are mostly on rows that
// exist.  Chunk c of a 128-byte stage row r sits at chunk c ^ ((r / 2) % 8): two rows fill the
// 64 banks, and the 16 lanes that read 16 bytes each in a cycle, 16 rows apart by one, hit each
// bank once (with c ^ (r % 8) rows r and r + 8 meet).
//
// Top of a piece: wait for its loads, then a barrier: the piece is in LDS for every
// wavefront, and every wavefront is done with the piece before, whose stage the next loads fill.
// A wavefront's vector memory operations retire in issue order, so the wait names how many
// later ones may be in flight: the loads of the pieces behind it (LOADS + 2 each) and the output
// stores of epilogues issued after its loads.  A smaller number than that only waits longer.
// ---------------------------------------------------------------------------
struct StagedArgs {
  Int8Args g;
  int tiles_m, tiles_n;  // tiles_m unused when grouped
  int nwg;
};

__device__ __forceinline__ int chunk_at(int r, int c) { return r * PR_ROW + ((c ^ ((r >> 1) & 7)) << 4); }

// Tile (row tile, column tile) at position s of the walk: groups of four row tiles,
// column by column, so that workgroups of one XCD share operand rows in its L2.
// Tiles number below 2^31: y has at most 2^40 elements and a tile 2^12 of them, and the
// grouped weights' columns, E N <= 2^36, bound the tiles of experts with few rows.
__device__ __forceinline__ void walk(int s, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int per_group = GROUP_M * tiles_n;
  const int g = s / per_group;
  const int gm = min(tiles_m - g * GROUP_M, GROUP_M);
  const int r = s - g * per_group;
  tm = g * GROUP_M + r % gm;
  tn = r / gm;
}

// Workgroups that share a CU: as many as its 160 KB of LDS hold.
template <int NI, int NJM, int S>
constexpr int staged_per_cu() { return (160 << 10) / (64 * (NI + NJM) * (PR_ROW + 4) * S + 256); }

template <int NI, int NJM, int S, int EPI, bool GROUPED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(
    (staged_per_cu<NI, NJM, S>()), (staged_per_cu<NI, NJM, S>())))) void k_int8_staged(StagedArgs a, uint16_t* __restrict__ Y, EpiArgs e) {
  constexpr int XR = 64 * NJM, WR = 64 * NI;     // rows of x and of W per stage
  constexpr int STAGE = (XR + WR) * PR_ROW;
  constexpr int XL = 2 * NJM, LOADS = XL + 2 * NI;  // loads per wavefront per piece: x, all
  constexpr int SBUF = (XR + WR) * 4;            // output scales of a tile
  __shared__ __attribute__((aligned(16))) uint8_t lds[S * STAGE];
  // output scales: a tile's are loaded up to S - 1 tiles ahead
  __shared__ __attribute__((aligned(16))) uint8_t lsc[S * SBUF + 256];
  const Int8Args& p = a.g;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wv >> 1, wn = wv & 1;
  const int h = lane >> 5, r32 = lane & 31;
  const int b = blockIdx.x;
  const uint32_t lbase = lds_address(lds), sbase = lds_address(lsc);
  const int tiles_m = GROUPED ? __builtin_amdgcn_readfirstlane(p.count[0]) : a.tiles_m;
  const int ntiles = tiles_m * a.tiles_n;
  const int np = (p.K + PR_ROW - 1) / PR_ROW;

  struct Tile {
    int64_t m0, n0;
    int rows, e;
  };
  // The tiles of a last round that is at most half (a quarter) full are cut into parts of
  // XR / 2 (/ 4) rows, one for each workgroup: units [0, full) are whole tiles, the ones behind them parts.
  const int full = ntiles - ntiles % a.nwg, tail = ntiles - full;
  const int parts = NJM >= 4 && 4 * tail <= a.nwg ? 4 : NJM >= 2 && 2 * tail <= a.nwg ? 2 : 1;
  const int units = full + tail * parts;
  // This workgroup's i-th unit (units: none).  Workgroups are dealt to the 8 XCDs in turn; in
  // every round, the last and shorter one too, an XCD's workgroups take a contiguous run of units.
  auto position = [&](int i) {
    const int base = i * a.nwg, left = min(units - base, a.nwg);
    if (left <= 0) return units;
    const int each = (left + 7) >> 3, at = (b & 7) * each + (b >> 3);
    if ((a.nwg & 7) != 0) return b < left ? base + b : units;
    return (b >> 3) < each && at < left ? base + at : units;
  };
  auto tile = [&](int i) {
    Tile t;
    int tm, tn;
    const int u = position(i);
    const bool whole = u < full;
    const int cut = whole ? 0 : (u - full) % parts;
    walk(whole ? u : full + (u - full) / parts, tiles_m, a.tiles_n, tm, tn);
    t.n0 = (int64_t)tn * WR;
    if constexpr (GROUPED) {
      const RowTile rt = p.tiles[tm];
      t.m0 = rt.m0;
      t.rows = rt.m1 - rt.m0;
      t.e = rt.e;
    } else {
      t.m0 = (int64_t)tm * XR;
      t.rows = (int)(p.M - t.m0 < XR ? p.M - t.m0 : XR);
      t.e = 0;
    }
    if (!whole && parts > 1) {
      const int first = XR / parts * cut;
      t.m0 += first;
      t.rows = min(t.rows - first, XR / parts);
    }
    return t;
  };
  int nt = 0;
  while (position(nt) < units) ++nt;
  if (nt > 0 && tile(nt - 1).rows <= 0) --nt;  // a part behind its tile's last row

  // load q of an operand: rows (rows / 4) wv + 8 q .. + 7; lane l fills row + l / 8, stage chunk
  // l % 8, with the row's chunk (l % 8) ^ ((row / 2) % 8) = lc ^ 4 (q % 2)
  const int lc = (lane & 7) ^ (lane >> 4);
  const uint32_t vx = (uint32_t)((XR / 4 * wv + (lane >> 3)) * p.px);
  const uint32_t vw = (uint32_t)((WR / 4 * wv + (lane >> 3)) * p.K);

  // The stream of pieces: the descriptors change where it enters a tile, from piece to
  // piece only the byte offset along K does.
  struct Piece {
    int koff, stage, buf;
    bool first, valid;
  };
  int s_i = 0, s_k = 0, s_stage = 0, s_buf = 0;
  u32x4 dx{}, dw{}, ds{};
  auto enter = [&](int i) {
    const Tile t = tile(i);
    const int rn = (int)(p.N - t.n0 < WR ? p.N - t.n0 : WR);
    dx = make_desc(p.x + t.m0 * p.px, (int64_t)t.rows * p.px);
    dw = make_desc(p.w + ((int64_t)t.e * p.N + t.n0) * p.K, (int64_t)rn * p.K);
    const bool row = wv < 2;
    ds = make_desc(row ? p.xs + t.m0 : p.ws + (int64_t)t.e * p.N + t.n0, (row ? t.rows : rn) * 4);
  };
  // the piece to load next; its loads have to be issued before the following call
  auto next_piece = [&]() {
    Piece r;
    r.valid = s_i < nt;
    r.first = s_k == 0;
    if (r.first && r.valid) enter(s_i);
    r.stage = s_stage;
    r.buf = s_buf;
    r.koff = s_k * PR_ROW;
    s_stage = s_stage == S - 1 ? 0 : s_stage + 1;
    if (++s_k == np) {
      s_k = 0;
      ++s_i;
      s_buf = s_buf == S - 1 ? 0 : s_buf + 1;
    }
    return r;
  };
  auto issue = [&](const Piece& s, int d) {
    const int q = d < XL ? d : d - XL;
    const int byte = 16 * (lc ^ (4 * (q & 1)));
    const bool in = s.valid && s.koff + byte < p.K;
    const uint32_t dst = lbase + s.stage * STAGE + (d < XL ? XR / 4 * wv + 8 * q : XR + WR / 4 * wv + 8 * q) * PR_ROW;
    const uint32_t vo = in ? (d < XL ? vx : vw) + (uint32_t)(8 * q * (d < XL ? p.px : p.K) + byte) : kOutOfRange;
    dma16(dst, vo, d < XL ? dx : dw, s.koff);
  };
  // the tile's output scales, 64 per load: wavefronts 0 and 1 those of x, 2 and 3 those of W; every
  // piece issues two loads per wavefront (out of range, into a spare area, unless it starts a tile)
  auto issue_scales = [&](const Piece& s, int hh) {
    const int c = 2 * (wv & 1) + hh;
    const bool real = s.valid && s.first && c < (wv < 2 ? NJM : NI);
    const uint32_t dst = sbase + (real ? s.buf * SBUF + (wv < 2 ? 0 : XR * 4) + c * 256 : S * SBUF);
    dma4(dst, real ? (uint32_t)((c * 64 + lane) * 4) : kOutOfRange, ds, 0);
  };

  struct Frag {
    i32x4 lo, hi;
  };
  auto frag = [&](const uint8_t* st, int row, int u) {
    return Frag{*reinterpret_cast<const i32x4*>(st + chunk_at(row, 4 * u + 2 * h)),
                *reinterpret_cast<const i32x4*>(st + chunk_at(row, 4 * u + 2 * h + 1))};
  };
  auto mma = [&](const Frag& w, const Frag& x, i32x16 c) {
    c = __builtin_amdgcn_mfma_i32_32x32x32_i8(w.lo, x.lo, c, 0, 0, 0);
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(w.hi, x.hi, c, 0, 0, 0);
  };
  Frag fw[NI], fx[NJM];

#pragma unroll
  for (int ahead = 0; ahead < S - 1; ++ahead) {
    const Piece s = next_piece();
#pragma unroll
    for (int d = 0; d < LOADS; ++d) issue(s, d);
    issue_scales(s, 0);
    issue_scales(s, 1);
  }
  constexpr int LATER = (S - 2) * (LOADS + 2);  // loads of the pieces behind the current one
  constexpr int STORES = 2 * NI * NJM;          // output stores of a whole tile
  static_assert(LATER + STORES < 64, "vmcnt holds 63");
  int st[S - 1] = {};  // stores issued by the epilogue after each of the last S - 1 pieces
  int cur = 0;         // stage of the piece being multiplied
  auto piece = [&](auto& acc, auto nj) {
    constexpr int NJ = decltype(nj)::value;
    constexpr int T = NI * NJ;  // tiles of 32 x 32 per wavefront
    int stores = 0;
#pragma unroll
    for (int i = 0; i < S - 1; ++i) stores += st[i];
    if (stores == STORES) {
      QPL_WAIT_VMCNT(LATER + STORES);
    } else {
      QPL_WAIT_VMCNT(LATER);
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = S - 2; i > 0; --i) st[i] = st[i - 1];
    st[0] = 0;
    const Piece s = next_piece();
    const uint8_t* cs = lds + cur * STAGE;
    const uint8_t* cw = cs + XR * PR_ROW;
    cur = cur == S - 1 ? 0 : cur + 1;
#pragma unroll
    for (int i = 0; i < NI; ++i) fw[i] = frag(cw, wn * 32 * NI + i * 32 + r32, 0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) fx[j] = frag(cs, wm * 32 * NJ + j * 32 + r32, 0);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        acc[i][j] = mma(fw[i], fx[j], acc[i][j]);
        const int k = NJ * i + j;
        if (i == NI - 1) fx[j] = frag(cs, wm * 32 * NJ + j * 32 + r32, 1);
        if (j == NJ - 1) fw[i] = frag(cw, wn * 32 * NI + i * 32 + r32, 1);
#pragma unroll
        for (int d = 0; d < LOADS; ++d)
          if (k == (d * T) / LOADS) issue(s, d);
        __builtin_amdgcn_sched_barrier(0);
      }
    // x tile rows outermost: the fragments that the first half freed first come first
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        acc[i][j] = mma(fw[i], fx[j], acc[i][j]);
        if (i == 0 && j == 0) {
          issue_scales(s, 0);
          issue_scales(s, 1);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  int buf = 0;
  auto run_tile = [&](const Tile& t, auto nj) {
    constexpr int NJ = decltype(nj)::value;
    i32x16 acc[NI][NJ];
#pragma unroll
    for (int x = 0; x < NI; ++x)
#pragma unroll
      for (int y = 0; y < NJ; ++y) acc[x][y] = i32x16{};
    for (int k = 0; k < np; ++k) piece(acc, nj);
    // as in settle, but 64 to 256 accumulator registers are not passed through a statement: nothing is
    // scheduled across the two barriers, and every reader stands behind the branch into an output path
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const float* ls = reinterpret_cast<const float*>(lsc + buf * SBUF);
    buf = buf == S - 1 ? 0 : buf + 1;
    st[0] = __builtin_amdgcn_readfirstlane(store_tile<NJ, NI, EPI, true>(
        acc, wm, wn, lane, t.m0, t.n0, t.m0 + t.rows, p.N, Y, [&](int r) { return ls[r]; },
        [&](int c) { return *reinterpret_cast<const f32x4*>(&ls[XR + c]); }, e));
  };
  for (int i = 0; i < nt; ++i) {
    const Tile t = tile(i);
    if (NJM == 1 || t.rows > XR / 2) {
      run_tile(t, std::integral_constant<int, NJM>{});
    } else if (NJM == 2 || t.rows > XR / 4) {
      if constexpr (NJM >= 2) run_tile(t, std::integral_constant<int, NJM / 2>{});
    } else {
      if constexpr (NJM >= 4) run_tile(t, std::integral_constant<int, NJM / 4>{});
    }
  }
  QPL_WAIT_VMCNT(0);
  QPL_WAIT_LGKM0();
}

template <int NI, int NJM, int S, bool GROUPED>
hipError_t launch_staged(const Int8Args& g, int64_t row_tiles, const Epilogue& ep, uint16_t* y, hipStream_t stream) {
  StagedArgs a;
  a.g = g;
  a.tiles_m = (int)row_tiles;
  a.tiles_n = (int)((g.N + 64 * NI - 1) / (64 * NI));
  const int64_t n = row_tiles * a.tiles_n * NJM, most = 256 * staged_per_cu<NI, NJM, S>();
  a.nwg = (int)(n < most ? n : most);
  const dim3 grid((unsigned)a.nwg), block(256);
  EpiArgs e;
  switch (epi_kind(ep, e)) {
    case 0: hipLaunchKernelGGL((k_int8_staged<NI, NJM, S, 0, GROUPED>), grid, block, 0, stream, a, y, e); break;
    case EPI_GELU:
      hipLaunchKernelGGL((k_int8_staged<NI, NJM, S, EPI_GELU, GROUPED>), grid, block, 0, stream, a, y, e);
      break;
    case EPI_QKV:
      if constexpr (!GROUPED) {
        hipLaunchKernelGGL((k_int8_staged<NI, NJM, S, EPI_QKV, false>), grid, block, 0, stream, a, y, e);
        break;
      }
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_int8(const uint16_t* x, int64_t M, int64_t K, int64_t pitch, const float* lam, int8_t* xq,
                             float* xs, hipStream_t stream) {
  const TilePlan none{};
  return lam ? launch_quant<true, false, false>(x, M, M, K, pitch, lam, nullptr, xq, xs, none, stream)
             : launch_quant<false, false, false>(x, M, M, K, pitch, nullptr, nullptr, xq, xs, none, stream);
}

namespace {

template <bool GROUPED>
hipError_t launch_shape(int v, const Int8Args& p, int64_t row_tiles, const Epilogue& ep, uint16_t* y,
                        hipStream_t stream) {
  switch (v) {
    case 0:
      // 16 wavefronts share K where one product has few workgroups (16 x 4096 x 4096: 6.8 against 7.2 us);
      // experts bring workgroups enough (28 rows of 16 experts, K = 2048, N = 1408: 8 take 9.8 us)
      return launch_direct<1, 1, GROUPED ? 8 : 16, 2, GROUPED>(p, row_tiles, ep, y, stream);
    case 1: return launch_direct<1, 2, 8, 2, GROUPED>(p, row_tiles, ep, y, stream);
    case 2: return launch_direct<2, 2, 8, 2, GROUPED>(p, row_tiles, ep, y, stream);
    case 3: return launch_staged<1, 1, 4, GROUPED>(p, row_tiles, ep, y, stream);
    case 4: return launch_staged<2, 1, 3, GROUPED>(p, row_tiles, ep, y, stream);
    case 5:
      if (four_stages(row_tiles, p.N)) return launch_staged<2, 2, 4, GROUPED>(p, row_tiles, ep, y, stream);
      return launch_staged<2, 2, 2, GROUPED>(p, row_tiles, ep, y, stream);
    case 6: return launch_staged<4, 2, 3, GROUPED>(p, row_tiles, ep, y, stream);
    default: return launch_staged<4, 4, 2, GROUPED>(p, row_tiles, ep, y, stream);
  }
}

}  // namespace

namespace {

template <bool SMOOTH>
hipError_t launch_token(const uint16_t* x, const float* lam, const Int8Args& p, const Epilogue& ep, uint16_t* y,
                        hipStream_t stream) {
  // one workgroup per CU at most, which quantizes once and takes 16 columns in each of its turns
  // (1 x 4096 x 12288: 13.2 us, 16.4 us with a workgroup for every 16 or 32 columns)
  const int64_t n = (p.N + 15) / 16;
  const dim3 grid((unsigned)(n < 256 ? n : 256)), block(64 * TOKEN_W);
  EpiArgs e;
  switch (epi_kind(ep, e)) {
    case 0: hipLaunchKernelGGL((k_int8_token<SMOOTH, 0>), grid, block, 0, stream, x, lam, p, y, e); break;
    case EPI_GELU:
      hipLaunchKernelGGL((k_int8_token<SMOOTH, EPI_GELU>), grid, block, 0, stream, x, lam, p, y, e);
      break;
    case EPI_QKV:
      hipLaunchKernelGGL((k_int8_token<SMOOTH, EPI_QKV>), grid, block, 0, stream, x, lam, p, y, e);
      break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

bool int8_token_fits(int64_t M, int64_t K) { return token_fits(M, K); }

hipError_t launch_int8_token(const uint16_t* x, int64_t M, int64_t K, int64_t N, const int8_t* w, const float* ws,
                             const float* lam, const Epilogue& ep, uint16_t* y, hipStream_t stream) {
  Int8Args p{};
  p.w = w;
  p.ws = ws;
  p.M = M;
  p.N = N;
  p.K = (int)K;
  return lam ? launch_token<true>(x, lam, p, ep, y, stream) : launch_token<false>(x, lam, p, ep, y, stream);
}

hipError_t launch_gemm_int8(const int8_t* xq, const float* xs, const int8_t* w, const float* ws, int64_t M, int64_t K,
                            int64_t N, const Epilogue& ep, uint16_t* y, hipStream_t stream) {
  Int8Args p{};
  p.x = xq;
  p.w = w;
  p.xs = xs;
  p.ws = ws;
  p.M = M;
  p.N = N;
  p.K = (int)K;
  p.px = (int)int8_pitch(K);
  const int v = dense_shape(M, K, N);
  return launch_shape<false>(v, p, (M + kShapes[v].rows - 1) / kShapes[v].rows, ep, y, stream);
}

int64_t grouped_row_tiles(int64_t R, int64_t E) { return row_tile_bound(R, E, kShapes[0].rows); }

static TilePlan tile_plan(const int32_t* offsets, int64_t R, int64_t K, int64_t N, int64_t E, int32_t* tiles) {
  TilePlan t;
  t.offsets = offsets;
  t.E = (int)E;
  t.R = (int)R;
  t.tm = kShapes[grouped_shape(R, K, N, E)].rows;
  t.cap = (int)row_tile_bound(R, E, t.tm);
  t.count = tiles;
  t.tiles = reinterpret_cast<RowTile*>(tiles) + 1;
  return t;
}

hipError_t launch_quant_int8_grouped(const uint16_t* x, int64_t rows_x, int64_t R, int64_t K, int64_t N,
                                     const int32_t* row_index, const int32_t* offsets, int64_t E, int8_t* xq,
                                     float* xs, int32_t* tiles, hipStream_t stream) {
  const TilePlan t = tile_plan(offsets, R, K, N, E, tiles);
  const int64_t pitch = int8_pitch(K);
  return row_index ? launch_quant<false, true, true>(x, rows_x, R, K, pitch, nullptr, row_index, xq, xs, t, stream)
                   : launch_quant<false, true, false>(x, rows_x, R, K, pitch, nullptr, nullptr, xq, xs, t, stream);
}

bool moe_front_fits(int64_t n, int64_t E) { return n <= FRONT_N && E <= FRONT_E; }

hipError_t launch_int8_moe_front(const int32_t* ids, int64_t n, int64_t topk, const uint16_t* x, int64_t K, int64_t N,
                                 int64_t E, int8_t* xq, float* xs, int32_t* slot, int32_t* offsets, int32_t* tiles,
                                 hipStream_t stream) {
  const TilePlan t = tile_plan(offsets, n, K, N, E, tiles);
  hipLaunchKernelGGL(k_int8_moe_front, dim3((unsigned)(n + 1)), dim3(256), 0, stream, ids, (int)n, (int)topk, x, K,
                     int8_pitch(K), xq, xs, slot, offsets, t);
  return hipGetLastError();
}

hipError_t launch_gemm_int8_grouped(const int8_t* xq, const float* xs, const int8_t* w, const float* ws, int64_t R,
                                    int64_t K, int64_t N, int64_t E, const int32_t* tiles, const Epilogue& ep,
                                    uint16_t* y, hipStream_t stream) {
  Int8Args p{};
  p.x = xq;
  p.w = w;
  p.xs = xs;
  p.ws = ws;
  p.M = R;
  p.N = N;
  p.K = (int)K;
  p.px = (int)int8_pitch(K);
  p.count = tiles;
  p.tiles = reinterpret_cast<const RowTile*>(tiles) + 1;
  const int v = grouped_shape(R, K, N, E);
  return launch_shape<true>(v, p, row_tile_bound(R, E, kShapes[v].rows), ep, y, stream);
}

}  // namespace qpl
