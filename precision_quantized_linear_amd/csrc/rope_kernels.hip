// Norm of each head of the queries and keys and the rotation by their positions, in one pass, and its backward.
//
//   n = x r w,  r = 1 / sqrt(mean_c x_c^2 + eps)        (per head; w per channel)
//   pair i of the first `rotary` channels: (a, b) -> scale (a cos - b sin, a sin + b cos) of the angle
//   position * inv_freq[i]; pairs are (i, i + rotary / 2) or, interleaved, (2 i, 2 i + 1)
//
// Everything is fp32 up to the one rounding to bf16; the angle is formed in fp64, in turns, and reduced to half a turn
// before its fp32 sine and cosine, so that far positions keep theirs.
//
// Bound by HBM: x is read and y written once.  A lane holds two 16-byte vectors of a head that contain whole pairs
// (the vectors j and j + rotary / 16, or 2 j and 2 j + 1), so the rotation stays inside the lane; LP lanes make a head,
// and such a group walks heads of one token, because they share the angles.
#include <type_traits>

#include "qpl_device.h"
#include "qpl_internal.h"

namespace qpl {

namespace {

struct Side {
  const uint16_t* x;   // backward: the saved input
  const uint16_t* dy;  // backward
  uint16_t* y;         // backward: dx
  int64_t xh, xt, dh, dt, yh, yt;
  const uint16_t* w;
};

struct RopeKernelArgs {
  Side side[2];
  int heads0, heads;  // of the first side, of both
  int64_t tokens;
  int chunks;         // vectors of 8 channels per head
  int rot;            // lanes that rotate: rotary / 16
  int slots, lg_slots;  // groups that share a token in a workgroup
  float inv_dim, eps, scale;
  bool interleaved;
  const int* positions;
  const float* inv_freq;
  int axes, bound[3];
  float* partial;     // backward: [workgroups, 2, head_dim]
};

struct Pairs {
  float c[8], s[8];
};

__device__ __forceinline__ void unpack(const u32x4& v, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = bf16_lo(v[k]);
    f[2 * k + 1] = bf16_hi(v[k]);
  }
}

__device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
  return u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
}

// cos and sin, times the scale, of the token's angles of the pairs 8 j .. 8 j + 7.
__device__ __forceinline__ Pairs angles(const RopeKernelArgs& p, int64_t token, int j) {
  Pairs r;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = 8 * j + k;
    const int axis = (i >= p.bound[0]) + (i >= p.bound[1]) + (i >= p.bound[2]);
    const double turns = (double)p.positions[token * p.axes + axis] * ((double)p.inv_freq[i] * 0.15915494309189535);
    const float part = (float)(turns - __builtin_rint(turns));
    float s, c;
    sincospif(2.0f * part, &s, &c);
    r.c[k] = c * p.scale;
    r.s[k] = s * p.scale;
  }
  return r;
}

// The pairs of a lane's two vectors turned by the angles (BACK: by their opposites).
template <bool BACK>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const Pairs& t, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = a[2 * k], y = a[2 * k + 1], c = t.c[k], s = BACK ? -t.s[k] : t.s[k];
      a[2 * k] = __builtin_fmaf(x, c, -(y * s));
      a[2 * k + 1] = __builtin_fmaf(x, s, y * c);
      const float z = b[2 * k], w = b[2 * k + 1], d = t.c[k + 4], e = BACK ? -t.s[k + 4] : t.s[k + 4];
      b[2 * k] = __builtin_fmaf(z, d, -(w * e));
      b[2 * k + 1] = __builtin_fmaf(z, e, w * d);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = a[k], y = b[k], c = t.c[k], s = BACK ? -t.s[k] : t.s[k];
      a[k] = __builtin_fmaf(x, c, -(y * s));
      b[k] = __builtin_fmaf(x, s, y * c);
    }
  }
}

template <int LP>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = LP / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Where a thread stands: its lane of a head, vectors, token slot.
template <int LP>
struct Place {
  int j, va, vb, slot, token;
  bool in, rot;
  __device__ __forceinline__ Place(const RopeKernelArgs& p) {
    const int g = threadIdx.x / LP;
    j = threadIdx.x % LP;
    in = 2 * j < p.chunks;
    rot = j < p.rot;
    const bool half = rot && !p.interleaved;
    va = half ? j : 2 * j;
    vb = half ? j + p.rot : 2 * j + 1;
    slot = g & (p.slots - 1);
    token = g >> p.lg_slots;
  }
};

template <int LP, bool NORM>
__global__ __launch_bounds__(256) void k_qk_norm_rope(RopeKernelArgs p) {
  const Place<LP> at(p);
  const int64_t t = (int64_t)blockIdx.x * (256 / LP >> p.lg_slots) + at.token;
  if (t >= p.tokens) return;
  Pairs tr{};
  if (at.rot) tr = angles(p, t, at.j);
  for (int h = blockIdx.y * p.slots + at.slot; h < p.heads; h += gridDim.y * p.slots) {
    const bool second = h >= p.heads0;
    const Side& s = p.side[second];
    const int64_t hh = second ? h - p.heads0 : h;
    const u32x4 zero{0u, 0u, 0u, 0u};
    const u32x4* x = reinterpret_cast<const u32x4*>(s.x + hh * s.xh + t * s.xt);
    float a[8], b[8];
    unpack(at.in ? x[at.va] : zero, a);
    unpack(at.in ? x[at.vb] : zero, b);
    if constexpr (NORM) {
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = __builtin_fmaf(a[k], a[k], __builtin_fmaf(b[k], b[k], sum));
      const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(group_sum<LP>(sum), p.inv_dim, p.eps));
      if (s.w) {
        float wa[8], wb[8];
        unpack(at.in ? reinterpret_cast<const u32x4*>(s.w)[at.va] : zero, wa);
        unpack(at.in ? reinterpret_cast<const u32x4*>(s.w)[at.vb] : zero, wb);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          a[k] *= r * wa[k];
          b[k] *= r * wb[k];
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          a[k] *= r;
          b[k] *= r;
        }
      }
    }
    if (at.rot) turn<false>(a, b, tr, p.interleaved);
    if (at.in) {
      u32x4* y = reinterpret_cast<u32x4*>(s.y + hh * s.yh + t * s.yt);
      y[at.va] = pack(a);
      y[at.vb] = pack(b);
    }
  }
}

// Backward: d = the gradient of n = dy turned back, times the scale;
// dx = r (d w - x r^2 mean(d w x)),  dw = sum over tokens and heads of d x r.
// Workgroups stride over the tokens and leave one row of partial sums each, so the weights' gradients do not
// depend on their order.
template <int LP, bool NORM>
__global__ __launch_bounds__(256) void k_qk_norm_rope_backward(RopeKernelArgs p) {
  const Place<LP> at(p);
  const int per = 256 / LP >> p.lg_slots;  // tokens of a workgroup at a time
  float ga[2][8] = {}, gb[2][8] = {};
  for (int64_t t = (int64_t)blockIdx.x * per + at.token; t < p.tokens; t += (int64_t)gridDim.x * per) {
    Pairs tr{};
    if (at.rot) tr = angles(p, t, at.j);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const Side& s = p.side[which];
      const int n = which ? p.heads - p.heads0 : p.heads0;
      float wa[8], wb[8];
      const u32x4 zero{0u, 0u, 0u, 0u};
      if (NORM && s.w) {
        unpack(at.in ? reinterpret_cast<const u32x4*>(s.w)[at.va] : zero, wa);
        unpack(at.in ? reinterpret_cast<const u32x4*>(s.w)[at.vb] : zero, wb);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) wa[k] = wb[k] = 1.0f;
      }
      for (int h = at.slot; h < n; h += p.slots) {
        const u32x4* dy = reinterpret_cast<const u32x4*>(s.dy + h * s.dh + t * s.dt);
        float da[8], db[8];
        unpack(at.in ? dy[at.va] : zero, da);
        unpack(at.in ? dy[at.vb] : zero, db);
        if (at.rot) turn<true>(da, db, tr, p.interleaved);
        if constexpr (NORM) {
          const u32x4* x = reinterpret_cast<const u32x4*>(s.x + h * s.xh + t * s.xt);
          float a[8], b[8];
          unpack(at.in ? x[at.va] : zero, a);
          unpack(at.in ? x[at.vb] : zero, b);
          float sum = 0.0f, dot = 0.0f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            sum = __builtin_fmaf(a[k], a[k], __builtin_fmaf(b[k], b[k], sum));
            dot = __builtin_fmaf(da[k] * wa[k], a[k], __builtin_fmaf(db[k] * wb[k], b[k], dot));
          }
          const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(group_sum<LP>(sum), p.inv_dim, p.eps));
          const float m = group_sum<LP>(dot) * p.inv_dim * r * r;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            ga[which][k] = __builtin_fmaf(da[k], a[k] * r, ga[which][k]);
            gb[which][k] = __builtin_fmaf(db[k], b[k] * r, gb[which][k]);
            da[k] = r * __builtin_fmaf(-a[k], m, da[k] * wa[k]);
            db[k] = r * __builtin_fmaf(-b[k], m, db[k] * wb[k]);
          }
        }
        if (at.in) {
          u32x4* dx = reinterpret_cast<u32x4*>(s.y + h * s.yh + t * s.yt);
          dx[at.va] = pack(da);
          dx[at.vb] = pack(db);
        }
      }
    }
  }
  if (!NORM || !p.partial) return;
  // the groups' sums of a channel, group by group
  __shared__ float sums[256 / LP][16 * LP + 1];
  const int g = threadIdx.x / LP, dim = 8 * p.chunks;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    if (at.in) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        sums[g][8 * at.va + k] = ga[which][k];
        sums[g][8 * at.vb + k] = gb[which][k];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < dim; c += 256) {
      float v = 0.0f;
      for (int i = 0; i < 256 / LP; ++i) v += sums[i][c];
      p.partial[((int64_t)blockIdx.x * 2 + which) * dim + c] = v;
    }
  }
}

// The workgroups' partial sums [rows, 2, dim] added up: 16 threads per column, then those in order.
__global__ __launch_bounds__(256) void k_sum_partial(const float* __restrict__ partial, int rows, int dim,
                                                     float* __restrict__ dw0, float* __restrict__ dw1) {
  __shared__ float part[16][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;  // of 2 dim, dim a multiple of 16
  float v = 0.0f;
  for (int i = r; i < rows; i += 16) v += partial[(int64_t)i * 2 * dim + col];
  part[r][c] = v;
  __syncthreads();
  if (r == 0) {
    for (int i = 1; i < 16; ++i) v += part[i][c];
    float* dw = col < dim ? dw0 : dw1;
    if (dw) dw[col < dim ? col : col - dim] = v;
  }
}

int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

int lanes_of(int head_dim) { return 1 << log2_of(head_dim / 16); }

RopeKernelArgs kernel_args(const RopeSide (&side)[2], int64_t tokens, int head_dim, const RopeArgs& r) {
  RopeKernelArgs p{};
  for (int i = 0; i < 2; ++i) {
    const RopeSide& s = side[i];
    p.side[i] = Side{s.x.p,           s.y.p,          s.dx.p ? s.dx.p : s.y.p, s.x.head_stride, s.x.token_stride,
                     s.y.head_stride, s.y.token_stride, s.dx.p ? s.dx.head_stride : s.y.head_stride,
                     s.dx.p ? s.dx.token_stride : s.y.token_stride, s.weight};
  }
  p.heads0 = (int)side[0].heads;
  p.heads = (int)(side[0].heads + side[1].heads);
  p.tokens = tokens;
  p.chunks = head_dim / 8;
  p.rot = r.rotary / 16;
  p.inv_dim = 1.0f / (float)head_dim;
  p.eps = r.eps;
  p.scale = r.scale;
  p.interleaved = r.interleaved;
  p.positions = r.positions;
  p.inv_freq = r.inv_freq;
  p.axes = r.axes;
  for (int i = 0; i < 3; ++i) p.bound[i] = r.bound[i];
  return p;
}

// Groups that share a token: one for each head while the tokens are too few to fill the chip, else one for every
// four heads, because the angles are the same for all of a token's heads.
int token_slots(int heads, int64_t tokens, int lanes) {
  const int most = 256 / lanes;
  int want = 1;
  while (want < most && want < (tokens * lanes * heads < 256 * 1024 ? heads : (heads + 3) / 4)) want *= 2;
  return want;
}

constexpr int64_t kBackwardBlocks = 1024;

template <class F>
hipError_t by_lanes(int lanes, const F& f) {
  switch (lanes) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    default: return f(std::integral_constant<int, 32>{});
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeSide (&side)[2], int64_t tokens, int head_dim, const RopeArgs& r,
                               hipStream_t stream) {
  RopeKernelArgs p = kernel_args(side, tokens, head_dim, r);
  const int lanes = lanes_of(head_dim);
  p.slots = token_slots(p.heads, tokens, lanes);
  p.lg_slots = log2_of(p.slots);
  const int64_t per = 256 / lanes / p.slots;
  const bool few = tokens * lanes * p.heads < 256 * 1024;
  const dim3 grid((unsigned)((tokens + per - 1) / per), (unsigned)(few ? (p.heads + p.slots - 1) / p.slots : 1));
  return by_lanes(lanes, [&](auto lp) {
    if (r.norm) {
      hipLaunchKernelGGL((k_qk_norm_rope<decltype(lp)::value, true>), grid, dim3(256), 0, stream, p);
    } else {
      hipLaunchKernelGGL((k_qk_norm_rope<decltype(lp)::value, false>), grid, dim3(256), 0, stream, p);
    }
    return hipGetLastError();
  });
}

size_t qk_backward_bytes(int64_t tokens, int head_dim) {
  const int64_t n = tokens < kBackwardBlocks ? tokens : kBackwardBlocks;
  return (size_t)(8 * n * head_dim);
}

hipError_t launch_qk_norm_rope_backward(const RopeSide (&side)[2], int64_t tokens, int head_dim, const RopeArgs& r,
                                        float* ws, hipStream_t stream) {
  RopeKernelArgs p = kernel_args(side, tokens, head_dim, r);
  const int lanes = lanes_of(head_dim);
  p.slots = token_slots(p.heads, tokens, lanes);
  p.lg_slots = log2_of(p.slots);
  const bool sums = side[0].dweight || side[1].dweight;
  p.partial = sums ? ws : nullptr;
  const int64_t per = 256 / lanes / p.slots, n = (tokens + per - 1) / per;
  const dim3 grid((unsigned)(n < kBackwardBlocks ? n : kBackwardBlocks));
  const hipError_t e = by_lanes(lanes, [&](auto lp) {
    if (r.norm) {
      hipLaunchKernelGGL((k_qk_norm_rope_backward<decltype(lp)::value, true>), grid, dim3(256), 0, stream, p);
    } else {
      hipLaunchKernelGGL((k_qk_norm_rope_backward<decltype(lp)::value, false>), grid, dim3(256), 0, stream, p);
    }
    return hipGetLastError();
  });
  if (e != hipSuccess || !sums) return e;
  hipLaunchKernelGGL(k_sum_partial, dim3((unsigned)(head_dim / 8)), dim3(256), 0, stream, ws, (int)grid.x, head_dim,
                     side[0].dweight, side[1].dweight);
  return hipGetLastError();
}

}  // namespace qpl
