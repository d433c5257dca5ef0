// Norm of each head of the queries and keys and the rotation by their positions, in one pass, and its backward.
//
//   n = x r w,  r = 1 / sqrt(mean_c x_c^2 + eps)        (per head; w per channel)
//   pair i of the first `rotary` channels: (a, b) -> scale (a cos - b sin, a sin + b cos) of the angle
//   position * inv_freq[i]; pairs are (i, i + rotary / 2) or, interleaved, (2 i, 2 i + 1)
//
// Everything is fp32 up to the one rounding to bf16; the angle is formed in fp64, in turns, and reduced to half a turn
// before its fp32 sine and cosine, so that far positions keep theirs.
//
// Bound by HBM: x is read and y written once.  A lane holds two 16-byte vectors of a head, LP lanes make a head, and
// such a group walks heads of one token.  The vectors are chosen so that every pair lies inside a lane: j and j +
// rotary / 16 where pairs are half a rotary part apart, any two where they are neighbours.  A workgroup makes its
// tokens' cosines and sines once, in LDS, for all heads: made by each group for itself, 8192 tokens of 40 heads of 128
// channels took 88 us.  They take 28.6 us now (168 MB, 5.9 TB/s, part of it from caches; 36 us with inputs from HBM, 4.6
// TB/s), their backward 46 us (252 MB; 58 us with inputs from HBM, 4.3 TB/s, of which 4 are the sums' launch).
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
  int heads0, heads;    // of the first side, of both
  int64_t tokens;
  int chunks;           // vectors of 8 channels per head
  int rot;              // rotary / 16
  int lg_slots, lg_per; // groups that share a token in a workgroup, tokens of a workgroup at a time
  bool by_token;        // neighbouring groups take neighbouring tokens (else heads)
  float inv_dim, eps, scale;
  bool interleaved;
  const int* positions;
  const float* inv_freq;
  int axes, bound[3];
  int blocks0;          // backward: workgroups of the first side
  float* partial;       // backward: [workgroups, head_dim]
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

// cos and sin, times the scale, of the angles of `per` tokens from t0 on: cs [per, 8 rot pairs].  Zeros for tokens past
// the last: the groups without a token read them too, and the weights' gradients add up their products with zeros,
// which are NaNs where LDS is left as the kernel before left it.
__device__ __forceinline__ void make_angles(const RopeKernelArgs& p, int64_t t0, float2* cs) {
  const int pairs = 8 * p.rot, n = pairs << p.lg_per;
  for (int k = threadIdx.x; k < n; k += 256) {
    const int tt = k / pairs, i = k - tt * pairs;
    if (t0 + tt >= p.tokens) {
      cs[k] = float2{0.0f, 0.0f};
      continue;
    }
    const int axis = (i >= p.bound[0]) + (i >= p.bound[1]) + (i >= p.bound[2]);
    const double turns = (double)p.positions[(t0 + tt) * p.axes + axis] * ((double)p.inv_freq[i] * 0.15915494309189535);
    float s, c;
    sincospif(2.0f * (float)(turns - __builtin_rint(turns)), &s, &c);
    cs[k] = float2{c * p.scale, s * p.scale};
  }
}

// Rotation of a pair; BACK: by the opposite angle.
template <bool BACK>
__device__ __forceinline__ void turn(float& x, float& y, float c, float s0) {
  const float s = BACK ? -s0 : s0, a = x, b = y;
  x = __builtin_fmaf(a, c, -(b * s));
  y = __builtin_fmaf(a, s, b * c);
}

// Sum over the LP lanes of a group, in all of them (LP 16 and less inside a row of the data path).
template <int LP>
__device__ __forceinline__ float group_sum(float v) {
  auto add = [&](auto ctrl) {
    v += __uint_as_float(__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  if constexpr (LP >= 2) add(std::integral_constant<int, 0xB1>{});   // lane ^ 1
  if constexpr (LP >= 4) add(std::integral_constant<int, 0x4E>{});   // lane ^ 2
  if constexpr (LP >= 8) add(std::integral_constant<int, 0x141>{});  // 7 - lane of eight
  if constexpr (LP >= 16) add(std::integral_constant<int, 0x140>{}); // 15 - lane of sixteen
  if constexpr (LP >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// Where a thread stands: its vectors of a head, its slot among the groups of a token, its token.
template <int LP>
struct Place {
  int va, vb, pa, pb, slot, token;  // pa, pb: first pairs (interleaved: four in each vector, else eight)
  bool in, ra, rb;                  // has vectors; they turn
  __device__ __forceinline__ Place(const RopeKernelArgs& p) {
    const int g = threadIdx.x / LP, j = threadIdx.x % LP, half = p.chunks >> 1;
    in = j < half;
    if (p.interleaved) {
      va = j;
      vb = j + half;
      ra = in && va < 2 * p.rot;
      rb = in && vb < 2 * p.rot;
      pa = 4 * va;
      pb = 4 * vb;
    } else {
      ra = rb = in && j < p.rot;
      va = ra ? j : p.rot + j;  // behind the rotary part the vectors j - rot and half - rot + (j - rot)
      vb = ra ? j + p.rot : half + j;
      pa = pb = 8 * j;
    }
    slot = p.by_token ? g >> p.lg_per : g & ((1 << p.lg_slots) - 1);
    token = p.by_token ? g & ((1 << p.lg_per) - 1) : g >> p.lg_slots;
  }
  // the cosines and sines of this thread's pairs, from its token's
  __device__ __forceinline__ Pairs pairs(const RopeKernelArgs& p, const float2* cs) const {
    Pairs t{};
    const float2* row = cs + token * 8 * p.rot;
    if (ra) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        t.c[k] = row[pa + k].x;
        t.s[k] = row[pa + k].y;
      }
    }
    if (rb) {
#pragma unroll
      for (int k = 4; k < 8; ++k) {
        const int i = p.interleaved ? pb + k - 4 : pb + k;
        t.c[k] = row[i].x;
        t.s[k] = row[i].y;
      }
    }
    return t;
  }
  template <bool BACK>
  __device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const Pairs& t, bool interleaved) const {
    if (interleaved) {
      if (ra) {
#pragma unroll
        for (int k = 0; k < 4; ++k) turn<BACK>(a[2 * k], a[2 * k + 1], t.c[k], t.s[k]);
      }
      if (rb) {
#pragma unroll
        for (int k = 0; k < 4; ++k) turn<BACK>(b[2 * k], b[2 * k + 1], t.c[k + 4], t.s[k + 4]);
      }
    } else if (ra) {
#pragma unroll
      for (int k = 0; k < 8; ++k) turn<BACK>(a[k], b[k], t.c[k], t.s[k]);
    }
  }
};

template <int LP, bool NORM>
__global__ __launch_bounds__(256) void k_qk_norm_rope(RopeKernelArgs p) {
  extern __shared__ float2 cs[];
  const Place<LP> at(p);
  const int64_t t0 = (int64_t)blockIdx.x << p.lg_per, t = t0 + at.token;
  const int step = gridDim.y << p.lg_slots;
  const bool live = at.in && t < p.tokens;
  const u32x4 zero{0u, 0u, 0u, 0u};
  u32x4 va, vb;
  auto load = [&](int h) {
    const Side& s = p.side[h >= p.heads0];
    const u32x4* x = reinterpret_cast<const u32x4*>(s.x + (int64_t)(h >= p.heads0 ? h - p.heads0 : h) * s.xh + t * s.xt);
    va = x[at.va];
    vb = x[at.vb];
  };
  int h = (blockIdx.y << p.lg_slots) + at.slot;
  va = vb = zero;
  if (live && h < p.heads) load(h);
  u32x4 wa[2] = {zero, zero}, wb[2] = {zero, zero};
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4* w = reinterpret_cast<const u32x4*>(p.side[i].w);
      if (w && at.in) {
        wa[i] = w[at.va];
        wb[i] = w[at.vb];
      } else {
        wa[i] = wb[i] = u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};  // ones
      }
    }
  }
  make_angles(p, t0, cs);
  __syncthreads();
  const Pairs tr = at.pairs(p, cs);
  for (; h < p.heads; h += step) {
    float a[8], b[8];
    unpack(va, a);
    unpack(vb, b);
    // the next head's vectors are on their way while this one is turned
    if (live && h + step < p.heads) load(h + step);
    const bool second = h >= p.heads0;
    if constexpr (NORM) {
      float sum = 0.0f, w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = __builtin_fmaf(a[k], a[k], __builtin_fmaf(b[k], b[k], sum));
      const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(group_sum<LP>(sum), p.inv_dim, p.eps));
      unpack(second ? wa[1] : wa[0], w);
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] *= r * w[k];
      unpack(second ? wb[1] : wb[0], w);
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] *= r * w[k];
    }
    at.template rotate<false>(a, b, tr, p.interleaved);
    if (live) {
      const Side& s = p.side[second];
      u32x4* y = reinterpret_cast<u32x4*>(s.y + (int64_t)(second ? h - p.heads0 : h) * s.yh + t * s.yt);
      y[at.va] = pack(a);
      y[at.vb] = pack(b);
    }
  }
}

// Backward: d = the gradient of n = dy turned back, times the scale;
// dx = r (d w - x r^2 mean(d w x)),  dw = sum over tokens and heads of d x r.
// The first blocks0 workgroups take the first side, the others the second; they stride over the tokens and leave one
// row of partial sums each, so the weights' gradients do not depend on their order.
template <int LP, bool NORM>
__global__ __launch_bounds__(256) void k_qk_norm_rope_backward(RopeKernelArgs p) {
  extern __shared__ float2 cs[];
  const Place<LP> at(p);
  const bool second = (int)blockIdx.x >= p.blocks0;
  const Side& s = p.side[second];
  const int heads = second ? p.heads - p.heads0 : p.heads0;
  const int block = second ? blockIdx.x - p.blocks0 : blockIdx.x, blocks = second ? gridDim.x - p.blocks0 : p.blocks0;
  const int slots = 1 << p.lg_slots;
  const u32x4 zero{0u, 0u, 0u, 0u};
  float wa[8], wb[8], ga[8] = {}, gb[8] = {};
#pragma unroll
  for (int k = 0; k < 8; ++k) wa[k] = wb[k] = 1.0f;
  if (NORM && s.w && at.in) {
    unpack(reinterpret_cast<const u32x4*>(s.w)[at.va], wa);
    unpack(reinterpret_cast<const u32x4*>(s.w)[at.vb], wb);
  }
  for (int64_t t0 = (int64_t)block << p.lg_per; t0 < p.tokens; t0 += (int64_t)blocks << p.lg_per) {
    const int64_t t = t0 + at.token;
    const bool live = at.in && t < p.tokens;
    __syncthreads();  // the tokens before are done with cs
    make_angles(p, t0, cs);
    __syncthreads();
    const Pairs tr = at.pairs(p, cs);
    u32x4 v[4] = {zero, zero, zero, zero};
    auto load = [&](int h) {
      const u32x4* d = reinterpret_cast<const u32x4*>(s.dy + h * s.dh + t * s.dt);
      v[0] = d[at.va];
      v[1] = d[at.vb];
      if constexpr (NORM) {
        const u32x4* x = reinterpret_cast<const u32x4*>(s.x + h * s.xh + t * s.xt);
        v[2] = x[at.va];
        v[3] = x[at.vb];
      }
    };
    int h = at.slot;
    if (live && h < heads) load(h);
    for (; h < heads; h += slots) {
      float da[8], db[8], a[8], b[8];
      unpack(v[0], da);
      unpack(v[1], db);
      unpack(v[2], a);
      unpack(v[3], b);
      if (live && h + slots < heads) load(h + slots);
      at.template rotate<true>(da, db, tr, p.interleaved);
      if constexpr (NORM) {
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
          ga[k] = __builtin_fmaf(da[k], a[k] * r, ga[k]);
          gb[k] = __builtin_fmaf(db[k], b[k] * r, gb[k]);
          da[k] = r * __builtin_fmaf(-a[k], m, da[k] * wa[k]);
          db[k] = r * __builtin_fmaf(-b[k], m, db[k] * wb[k]);
        }
      }
      if (live) {
        u32x4* dx = reinterpret_cast<u32x4*>(s.y + h * s.yh + t * s.yt);
        dx[at.va] = pack(da);
        dx[at.vb] = pack(db);
      }
    }
  }
  if (!NORM || !p.partial) return;
  // the groups' sums of a channel, group by group
  __shared__ float sums[256 / LP][16 * LP + 1];
  const int dim = 8 * p.chunks;
  if (at.in) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      sums[threadIdx.x / LP][8 * at.va + k] = ga[k];
      sums[threadIdx.x / LP][8 * at.vb + k] = gb[k];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < dim; c += 256) {
    float v = 0.0f;
#pragma unroll 8
    for (int i = 0; i < 256 / LP; ++i) v += sums[i][c];
    p.partial[(int64_t)blockIdx.x * dim + c] = v;
  }
}

// The workgroups' partial sums [rows, dim] of a side added up: 64 threads for every four columns, then those in order.
// blockIdx.y: the side, rows [0, rows0) or [rows0, rows).
__global__ __launch_bounds__(256) void k_sum_partial(const float* __restrict__ partial, int rows0, int rows, int dim,
                                                     float* __restrict__ dw0, float* __restrict__ dw1) {
  __shared__ f32x4 part[64][4];
  float* dw = blockIdx.y ? dw1 : dw0;
  if (!dw) return;
  const int first = blockIdx.y ? rows0 : 0, last = blockIdx.y ? rows : rows0;
  const int c = threadIdx.x & 3, r = threadIdx.x >> 2;
  const f32x4* p = reinterpret_cast<const f32x4*>(partial) + blockIdx.x * 4 + c;  // dim is a multiple of 16
  f32x4 v{};
#pragma unroll 8
  for (int i = first + r; i < last; i += 64) v += p[(int64_t)i * (dim / 4)];
  part[r][c] = v;
  __syncthreads();
  if (threadIdx.x < 16) {
    const float* q = reinterpret_cast<const float*>(part) + threadIdx.x;
    float s = 0.0f;
#pragma unroll 16
    for (int i = 0; i < 64; ++i) s += q[16 * i];
    dw[blockIdx.x * 16 + threadIdx.x] = s;
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

// Workgroups of the backward, 768 of which the chip holds at once.  8192 tokens of 32 and 8 heads of 128, inputs from
// HBM: 62 us at 2048 and at 4096, 74 at 1024, where a third of the workgroups of the first side made three turns and
// the rest two; with every workgroup of a side making the same number of turns 60 at 2048, 63 at 4096, 65 at 768.
constexpr int64_t kBackwardBlocks = 2048;

// Workgroups for n turns: at most `most`, the fewest that make as many turns each as those would.
int64_t even_blocks(int64_t n, int64_t most) {
  const int64_t each = (n + most - 1) / most;
  return (n + each - 1) / each;
}

// Workgroups that fill the chip: below them heads are spread further.  32 and 8 heads of 128, head-major, us at 256, 768
// and 1024: forward of 1024 tokens 8.3, 6.7 and 6.6, of 1536 9.4, 8.8 and 9.2, of 2048 13.9, 11.3 and 11.3 (never
// spread: 12.2, 12.8 and 13.8); backward, where each workgroup ends with its sums, of 512 tokens 9.1, 10.2 and 10.2, of
// 1024 11.2, 16.8 and 16.8, of 2048 17.9, 23.4 and 23.5 (never spread: 12.0, 13.8 and 18.2).  Single tokens of 40
// heads take 3.4 us spread, 10.3 not.
constexpr int64_t kFill = 768, kFillBackward = 256;

// Groups that share a token, a power of two: so many that they walk four heads or more (the next head's loads run
// under the work on this one) and the fewest stand idle at the end.  Head-major tensors are contiguous along the
// tokens, so there neighbouring groups take tokens, at least eight of them.  With few tokens more groups share one,
// until the workgroups fill the chip or every head has a group.
void place_groups(RopeKernelArgs& p, int heads, int lanes, int64_t fill) {
  const int groups = 256 / lanes;
  int best = 1, least = heads;
  for (int s = 1; s <= groups && (s == 1 || 4 * s <= heads); s *= 2) {
    const int padded = (heads + s - 1) / s * s;
    if (padded <= least) {
      least = padded;
      best = s;
    }
  }
  p.by_token = p.side[0].xt < p.side[0].xh;
  while (p.by_token && best > 1 && groups / best < 8) best /= 2;
  while (best < groups && best < heads && p.tokens * best < fill * groups) best *= 2;
  p.lg_slots = log2_of(best);
  p.lg_per = log2_of(groups / best);
}

// Bytes of LDS that the angles of a workgroup's tokens take: 8 pairs at most for each lane of a head, 16 KB in all.
size_t angle_bytes(const RopeKernelArgs& p) { return (sizeof(float2) * 8 * (size_t)p.rot) << p.lg_per; }

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

constexpr int64_t kMostBlocks = int64_t(1) << 23;

hipError_t launch_qk_norm_rope(const RopeSide (&side)[2], int64_t tokens, int head_dim, const RopeArgs& r,
                               hipStream_t stream) {
  RopeKernelArgs p = kernel_args(side, tokens, head_dim, r);
  const int lanes = lanes_of(head_dim);
  place_groups(p, p.heads, lanes, kFill);
  // where that does not fill the chip, a token's heads go to several workgroups
  const int64_t per = int64_t(1) << p.lg_per, slots = int64_t(1) << p.lg_slots;
  const int64_t n = (tokens + per - 1) / per, turns = (p.heads + slots - 1) / slots, parts = (kFill + n - 1) / n;
  const size_t lds = angle_bytes(p);
  // A grid's threads are counted in 32 bits, and the runtime launches what is left of more without an error: so many
  // tokens go in slices.
  const int64_t each = kMostBlocks << p.lg_per;
  return by_lanes(lanes, [&](auto lp) {
    for (int64_t t0 = 0; t0 < tokens; t0 += each) {
      if (t0 > 0) {
        for (Side& s : p.side) {
          s.x += each * s.xt;
          s.y += each * s.yt;
        }
        p.positions += each * p.axes;
      }
      p.tokens = tokens - t0 < each ? tokens - t0 : each;
      const dim3 grid((unsigned)((p.tokens + per - 1) / per), (unsigned)(parts < turns ? parts : turns));
      if (r.norm) {
        hipLaunchKernelGGL((k_qk_norm_rope<decltype(lp)::value, true>), grid, dim3(256), lds, stream, p);
      } else {
        hipLaunchKernelGGL((k_qk_norm_rope<decltype(lp)::value, false>), grid, dim3(256), lds, stream, p);
      }
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
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
  place_groups(p, p.heads0, lanes, kFillBackward);
  const bool sums = side[0].dweight || side[1].dweight;
  p.partial = sums ? ws : nullptr;
  // the sides' shares of the workgroups are as their heads; one of a side takes at least one token
  const int64_t per = int64_t(1) << p.lg_per, n = (tokens + per - 1) / per, heads1 = p.heads - p.heads0;
  int64_t b0 = heads1 == 0 ? kBackwardBlocks : kBackwardBlocks * p.heads0 / p.heads;
  int64_t b1 = heads1 == 0 ? 0 : kBackwardBlocks - b0;
  b0 = even_blocks(n, b0 < 1 ? 1 : b0);
  if (heads1 > 0) b1 = even_blocks(n, b1 < 1 ? 1 : b1);
  p.blocks0 = (int)b0;
  const dim3 grid((unsigned)(b0 + b1));
  const size_t lds = angle_bytes(p);
  const hipError_t e = by_lanes(lanes, [&](auto lp) {
    if (r.norm) {
      hipLaunchKernelGGL((k_qk_norm_rope_backward<decltype(lp)::value, true>), grid, dim3(256), lds, stream, p);
    } else {
      hipLaunchKernelGGL((k_qk_norm_rope_backward<decltype(lp)::value, false>), grid, dim3(256), lds, stream, p);
    }
    return hipGetLastError();
  });
  if (e != hipSuccess || !sums) return e;
  hipLaunchKernelGGL(k_sum_partial, dim3((unsigned)(head_dim / 16), 2), dim3(256), 0, stream, ws, (int)b0, (int)(b0 + b1),
                     head_dim, side[0].dweight, side[1].dweight);
  return hipGetLastError();
}

}  // namespace qpl
