// Routing of tokens to experts for gfx950: the sort of the router's choices by expert
// and the weighted sum that brings the experts' rows back to their tokens.
#include "qpl_device.h"
#include "qpl_internal.h"

namespace qpl {

namespace {

// ---------------------------------------------------------------------------
// Plan: a stable counting sort of n choices ids[i] in [0, E) without atomics or a
// workspace.  Workgroup e serves expert e: it counts the choices below e (the
// expert's first place) and lists its own, then hands out its places in order of i.
// Each wavefront owns a contiguous run of choices, so a place is the expert's first +
// the counts of earlier wavefronts + a ballot prefix.  A wavefront lists up to LIST
// choices in LDS; one that finds more reads its run again.  Workgroup E serves the ids
// outside [0, E): slot -1, and row_index -1 behind the last place.  Every workgroup
// reads all choices (from L2), which costs less than a second launch.
// ---------------------------------------------------------------------------
constexpr int LIST = 512;

// i / topk for 0 <= i < 2^31: mul is ceil(2^shift / topk) with shift = 31 + ceil(log2 topk), so
// mul topk exceeds 2^shift by at most topk and the quotient is exact.
struct Divider {
  uint64_t mul;
  int shift;
  __device__ __forceinline__ int operator()(int i) const { return (int)(((uint64_t)(uint32_t)i * mul) >> shift); }
};

template <int W, int B>
__global__ __launch_bounds__(64 * W) void k_expert_plan(const int* __restrict__ ids, int n, Divider token, int E,
                                                        int* __restrict__ row_index, int* __restrict__ slot,
                                                        int* __restrict__ offsets) {
  __shared__ int below_s[W], own_s[W];
  __shared__ int list[W][LIST];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int run = (n / (64 * W) + 1) * 64;  // choices per wavefront, a multiple of 64
  const int64_t first = (int64_t)wv * run;
  const int lo = first < n ? (int)first : n;
  const int hi = first + run < n ? (int)(first + run) : n;
  const uint64_t before = (1ull << lane) - 1ull;
  // use(v, i) with choice i of the run for each lane, 64 at a time in order: batches of B loads
  // in flight together, then single ones.  Behind the end stands an id that is nobody's (INT_MIN
  // is outside [0, E)).
  auto each = [&](auto use) {
    int i0 = lo + lane;
    for (; i0 - lane + 64 * B <= hi; i0 += 64 * B) {
      int v[B];
#pragma unroll
      for (int u = 0; u < B; ++u) v[u] = ids[i0 + 64 * u];
#pragma unroll
      for (int u = 0; u < B; ++u) use(v[u], i0 + 64 * u);
    }
    for (; i0 - lane < hi; i0 += 64) use(i0 < hi ? ids[i0] : INT32_MIN, i0);
  };
  // found(i, r) for the run's r-th choice i of expert e, in order; returns their number
  auto scan = [&](int e, auto count, auto found) {
    int own = 0;
    each([&](int v, int i) {
      count(v);
      const uint64_t b = __ballot(v == e);
      if (b != 0) {
        if (v == e) found(i, own + __popcll(b & before));
        own += __popcll(b);
      }
    });
    return own;
  };
  for (int e = blockIdx.x; e <= E; e += gridDim.x) {
    int below = 0;
    const int own = scan(
        e, [&](int v) { below += (uint32_t)v < (uint32_t)e; },
        [&](int i, int r) {
          if (r < LIST) list[wv][r] = i;
        });
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) below += __shfl_xor(below, d, 64);
    if (lane == 0) {
      below_s[wv] = below;
      own_s[wv] = own;
    }
    __syncthreads();
    int base = 0;
    for (int w = 0; w < W; ++w) base += below_s[w];
    if (threadIdx.x == 0) offsets[e] = base;
    if (e < E) {
      int place = base;
      for (int w = 0; w < wv; ++w) place += own_s[w];
      if (own <= LIST) {
        for (int r = lane; r < own; r += 64) {
          const int i = list[wv][r];
          slot[i] = place + r;
          row_index[place + r] = token(i);
        }
      } else {
        scan(
            e, [](int) {},
            [&](int i, int r) {
              slot[i] = place + r;
              row_index[place + r] = token(i);
            });
      }
    } else {
      // an id outside [0, E) is E itself, counted as this workgroup's own, or above, or negative
      each([&](int v, int i) {
        if (i < hi && (uint32_t)v >= (uint32_t)E) slot[i] = -1;
      });
      for (int64_t i = (int64_t)base + threadIdx.x; i < n; i += 64 * W) row_index[i] = -1;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Combine: out[t] = bf16(sum_j weight[t, j] y[slot[t, j]]), fp32, j ascending; a slot
// outside [0, R) adds nothing.  VEC columns per thread (8: one 16-byte load per
// row; 1 where rows are not 16-byte aligned).
// ---------------------------------------------------------------------------
template <int VEC>
__global__ __launch_bounds__(256) void k_expert_combine(const uint16_t* __restrict__ y, int64_t R, int64_t N,
                                                        const int* __restrict__ slot,
                                                        const float* __restrict__ weight, int64_t T, int topk,
                                                        uint16_t* __restrict__ out) {
  const int64_t nv = N / VEC;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < T * nv; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / nv, c = (i - t * nv) * VEC;
    const int* st = slot + t * topk;
    const float* wt = weight + t * topk;
    if constexpr (VEC == 8) {
      float a[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
      for (int j = 0; j < topk; ++j) {
        const int64_t s = st[j];
        if (s >= 0 && s < R) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(y + s * N + c);
          const float w = wt[j];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            a[2 * k] = __builtin_fmaf(w, bf16_lo(v[k]), a[2 * k]);
            a[2 * k + 1] = __builtin_fmaf(w, bf16_hi(v[k]), a[2 * k + 1]);
          }
        }
      }
      *reinterpret_cast<u32x4*>(out + t * N + c) =
          u32x4{pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7])};
    } else {
      float a = 0.0f;
      for (int j = 0; j < topk; ++j) {
        const int64_t s = st[j];
        if (s >= 0 && s < R) a = __builtin_fmaf(wt[j], __uint_as_float((uint32_t)y[s * N + c] << 16), a);
      }
      out[t * N + c] = (uint16_t)pack_bf16(a, 0.0f);
    }
  }
}

}  // namespace

hipError_t launch_expert_plan(const int32_t* ids, int64_t n, int64_t topk, int64_t E, int32_t* row_index,
                              int32_t* slot, int32_t* offsets, hipStream_t stream) {
  const dim3 grid((unsigned)(E + 1));
  Divider token;
  token.shift = 31;
  while ((int64_t{1} << (token.shift - 31)) < topk) ++token.shift;
  token.mul = ((uint64_t{1} << token.shift) + (uint64_t)topk - 1) / (uint64_t)topk;
  // 4 wavefronts per expert while each still has at most 1024 choices, else 16
  if (n <= 4096)
    hipLaunchKernelGGL((k_expert_plan<4, 8>), grid, dim3(256), 0, stream, ids, (int)n, token, (int)E, row_index, slot,
                       offsets);
  else
    hipLaunchKernelGGL((k_expert_plan<16, 16>), grid, dim3(1024), 0, stream, ids, (int)n, token, (int)E, row_index,
                       slot, offsets);
  return hipGetLastError();
}

hipError_t launch_expert_combine(const uint16_t* y, int64_t R, int64_t N, const int32_t* slot, const float* weights,
                                 int64_t T, int64_t topk, uint16_t* out, hipStream_t stream) {
  const int64_t threads = N % 8 == 0 ? T * (N / 8) : T * N;
  const int64_t blocks = (threads + 255) / 256;
  const dim3 grid((unsigned)(blocks < (int64_t(1) << 22) ? blocks : int64_t(1) << 22)), block(256);
  if (N % 8 == 0)
    hipLaunchKernelGGL(k_expert_combine<8>, grid, block, 0, stream, y, R, N, slot, weights, T, (int)topk, out);
  else
    hipLaunchKernelGGL(k_expert_combine<1>, grid, block, 0, stream, y, R, N, slot, weights, T, (int)topk, out);
  return hipGetLastError();
}

}  // namespace qpl
