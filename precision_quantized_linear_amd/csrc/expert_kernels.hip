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
// Plan of many choices, in two launches over chunks of them: every workgroup of the second
// would have to read all choices to know the counts before its chunk, so the first writes
// counts[chunk][expert] (order-free integer atomics in LDS).  The second sums the columns
// of that matrix (an expert's first place, and what earlier chunks take of it) and hands out
// its chunk's places: each wavefront owns a contiguous run of the chunk, and of 64 choices
// those of one expert find each other by ballots over the id's bits.  131072 choices of 256
// experts: the form above reads them 257 times (19 us).
// SLICED, for more than PLAN_E experts: workgroup (c, s) serves the choices of chunk c for the
// PLAN_E experts from s PLAN_E, so the choices are read three times for each slice, not once for
// each expert.  The slices' sums for each chunk, which follow counts in the workspace, give the
// places before a slice.
// ---------------------------------------------------------------------------
constexpr int PLAN_E = 1024, PLAN_W = 16;

// LDS accesses of a wavefront's lanes stay on their side of this point.  A wavefront's LDS
// operations complete in order, so it costs no instruction.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ int wave_total(int v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

template <bool SLICED>
__global__ __launch_bounds__(64 * PLAN_W) void k_expert_count(const int* __restrict__ ids, int n, int chunk, int E,
                                                              int* __restrict__ counts) {
  constexpr int THREADS = 64 * PLAN_W;
  __shared__ int own[PLAN_E];
  __shared__ int sum;
  const int slice = SLICED ? blockIdx.y : 0, base = slice * PLAN_E;
  const int mine = SLICED ? min(E - base, PLAN_E) : E;  // experts of this workgroup
  for (int e = threadIdx.x; e < mine; e += THREADS) own[e] = 0;
  if (threadIdx.x == 0) sum = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * chunk;
  const int64_t hi = lo + chunk < n ? lo + chunk : n;
  for (int64_t i = lo + threadIdx.x; i < hi; i += THREADS) {
    const uint32_t v = (uint32_t)ids[i] - (uint32_t)base;
    if (v < (uint32_t)mine) atomicAdd(&own[v], 1);
  }
  __syncthreads();
  int part = 0;
  for (int e = threadIdx.x; e < mine; e += THREADS) {
    counts[(int64_t)blockIdx.x * E + base + e] = own[e];
    part += own[e];
  }
  if constexpr (SLICED) {
    part = wave_total(part);
    if ((threadIdx.x & 63) == 0) atomicAdd(&sum, part);
    __syncthreads();
    if (threadIdx.x == 0) counts[(int64_t)gridDim.x * E + (int64_t)blockIdx.x * gridDim.y + slice] = sum;
  }
}

// bits: 2^bits >= experts of a slice
template <bool SLICED>
__global__ __launch_bounds__(64 * PLAN_W) void k_expert_place(const int* __restrict__ ids, int n, int chunk,
                                                              Divider token, int E, int bits,
                                                              const int* __restrict__ counts,
                                                              int* __restrict__ row_index, int* __restrict__ slot,
                                                              int* __restrict__ offsets) {
  constexpr int THREADS = 64 * PLAN_W;
  __shared__ int next[PLAN_W][PLAN_E];  // a wavefront's next place of each expert
  __shared__ int before[PLAN_E], total[PLAN_E], wave_sum[PLAN_W];
  __shared__ int slices_before, slices_all;  // choices of the experts before the slice, and of all
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, c = blockIdx.x;
  const int slice = SLICED ? blockIdx.y : 0, base = slice * PLAN_E;
  const int experts = SLICED ? min(E - base, PLAN_E) : E;
  for (int e = threadIdx.x; e < experts; e += THREADS) before[e] = total[e] = 0;
  for (int i = threadIdx.x; i < PLAN_W * PLAN_E; i += THREADS) next[0][i] = 0;
  if (threadIdx.x == 0) slices_before = slices_all = 0;
  __syncthreads();
  // counts of this wavefront's run
  const int64_t lo = (int64_t)c * chunk + (int64_t)wv * (chunk / PLAN_W);
  const int64_t end = lo + chunk / PLAN_W;
  const int64_t hi = end < n ? end : n;
  for (int64_t i = lo + lane; i < hi; i += 64) {
    const uint32_t v = (uint32_t)ids[i] - (uint32_t)base;
    if (v < (uint32_t)experts) atomicAdd(&next[wv][v], 1);
  }
  // column sums, THREADS / 2^bits rows of the matrix at a time
  const int e0 = threadIdx.x & ((1 << bits) - 1), step = THREADS >> bits;
  if (e0 < experts) {
    int b = 0, t = 0;
#pragma unroll 16
    for (int r = threadIdx.x >> bits; r < (int)gridDim.x; r += step) {
      const int k = counts[(int64_t)r * E + base + e0];
      t += k;
      b += r < c ? k : 0;
    }
    atomicAdd(&total[e0], t);
    atomicAdd(&before[e0], b);
  }
  if constexpr (SLICED) {
    const int* sums = counts + (int64_t)gridDim.x * E;
    const int slices = gridDim.y, cells = (int)gridDim.x * slices;
    int b = 0, t = 0;
    for (int i = threadIdx.x; i < cells; i += THREADS) {
      t += sums[i];
      b += i % slices < slice ? sums[i] : 0;
    }
    t = wave_total(t);
    b = wave_total(b);
    if (lane == 0) {
      atomicAdd(&slices_all, t);
      atomicAdd(&slices_before, b);
    }
  }
  __syncthreads();
  // exclusive sum of the totals: thread e for expert e of the slice (at most THREADS)
  const int e = threadIdx.x;
  const int mine = e < experts ? total[e] : 0;
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(sum, d, 64);
    if (lane >= d) sum += o;
  }
  if (lane == 63) wave_sum[wv] = sum;
  __syncthreads();
  int first = sum - mine, all = 0;
#pragma unroll
  for (int w = 0; w < PLAN_W; ++w) {
    if (w < wv) first += wave_sum[w];
    all += wave_sum[w];
  }
  if constexpr (SLICED) {
    first += slices_before;
    all = slices_all;
  }
  if (e < experts) {
    if (c == 0) offsets[base + e] = first;
    int place = first + before[e];
#pragma unroll
    for (int w = 0; w < PLAN_W; ++w) {
      const int k = next[w][e];
      next[w][e] = place;
      place += k;
    }
  }
  if (c == 0 && slice == 0 && threadIdx.x == 0) offsets[E] = all;
  __syncthreads();
  const uint64_t earlier = (1ull << lane) - 1ull;
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    const uint32_t id = i < hi ? (uint32_t)ids[i] : 0xFFFFFFFFu;  // outside [0, E)
    const uint32_t v = id - (uint32_t)base;
    const bool valid = v < (uint32_t)experts;
    uint64_t peers = __ballot(valid);
    if (SLICED && peers == 0 && slice > 0) continue;
    for (int k = 0; k < bits; ++k) {
      const bool set = (v >> k) & 1;
      const uint64_t b = __ballot(set);
      peers &= set ? b : ~b;
    }
    int place = 0;
    if (valid) place = next[wv][v] + __popcll(peers & earlier);
    wave_order();  // the peers' reads before the first one's sum
    if (valid) {
      slot[i] = place;
      row_index[place] = token((int)i);
      if ((peers & earlier) == 0) next[wv][v] = place + __popcll(peers);
    } else if (i < hi && slice == 0 && id >= (uint32_t)E) {
      slot[i] = -1;
    }
    wave_order();  // and that before the reads of the next 64
  }
  if (slice == 0)
    for (int64_t i = (int64_t)all + (int64_t)c * THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * THREADS)
      row_index[i] = -1;
}

// Choices of a chunk: 2048, or what makes at most 256 chunks.
int plan_chunk(int64_t n) {
  const int64_t c = (n + 255) / 256;
  return c <= 2048 ? 2048 : (int)((c + 1023) / 1024 * 1024);
}

int plan_slices(int64_t E) { return (int)((E + PLAN_E - 1) / PLAN_E); }

// Which form.  One launch reads all choices once per expert, chunks cost a second launch.  In the one
// launch an expert's workgroup has 4 wavefronts, or 16, of which not all workgroups are on the chip
// at once past some hundred experts.  Measured, us in a graph (4 wavefronts / 16 / chunks):
//   choices  64 experts      256            512             1024            2048            8192           65536
//   1024     3.6/3.5/6.5     3.6/3.6/6.8    3.7/4.7/6.9     3.9/6.5/7.3     4.9/9.9/8.4     9.6/31/9.0     55/-/8.8
//   4096     4.2/4.2/7.0     4.2/4.4/7.6    4.3/6.1/7.9     4.7/8.4/8.6     6.2/13/9.8      12.2/39/10.2   69/-/10.0
//   8192     5.8/5.5/7.5     5.8/6.2/8.0    5.9/8.9/8.6     6.6/12.3/9.4    8.6/19/10.5     17.3/54/10.6   -/407/11.8
//   12288    7.2/6.7/7.6     7.5/7.6/8.2    7.5/10.8/8.8    8.2/14.5/10.1   11.1/22/11.2    22/66/11.6
//   16384    8.7/5.0/7.6     8.8/5.9/8.4    9.0/7.8/9.1     9.7/10.7/10.8   13.4/16.1/12.0  28/47/12.2     -/333/21.9
//   24576    11.6/7.2/7.7    11.9/8.8/8.7   12.1/11.6/9.7   13.2/16.0/11.6  17.9/23/12.9    38/70/13.6
//   32768    14.7/6.4/7.8    14.9/7.9/9.0   15.3/10.3/10.2  16.5/14.0/9.7   22/20/10.9      48/61/11.5     -/438/35.5
//   65536    -/13.1/8.2      -/13.8/10.1                    -/22/10.9       -/33/12.4                      -/659/74.0
bool plan_in_chunks(int64_t n, int64_t E) {
  return E <= 256 ? n >= 32768 : E > 8192 || n > 12288 || n * E > int64_t(1) << 24;
}

// Plans that needed no workspace while one launch was the rule for them still run without one, as far as
// their n E reads end in some milliseconds (2^32 of them take 0.7).
bool plan_in_one(int64_t n, int64_t E) {
  return !plan_in_chunks(n, E) || ((n < 32768 || E > PLAN_E) && n * E <= int64_t(1) << 35);
}

bool plan_by_four(int64_t n, int64_t E) { return n <= 4096 || E > 256; }

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

size_t expert_plan_bytes(int64_t n, int64_t E) {
  if (!plan_in_chunks(n, E)) return 0;
  const int64_t chunks = (n + plan_chunk(n) - 1) / plan_chunk(n);
  return (size_t)(4 * chunks * (E + (E > PLAN_E ? plan_slices(E) : 0)));
}

bool expert_plan_needs_none(int64_t n, int64_t E) { return plan_in_one(n, E); }

hipError_t launch_expert_plan(const int32_t* ids, int64_t n, int64_t topk, int64_t E, int32_t* row_index,
                              int32_t* slot, int32_t* offsets, int32_t* counts, hipStream_t stream) {
  const dim3 grid((unsigned)(E + 1));
  Divider token;
  token.shift = 31;
  while ((int64_t{1} << (token.shift - 31)) < topk) ++token.shift;
  token.mul = ((uint64_t{1} << token.shift) + (uint64_t)topk - 1) / (uint64_t)topk;
  if (counts && plan_in_chunks(n, E)) {
    const int chunk = plan_chunk(n);
    const dim3 chunks((unsigned)((n + chunk - 1) / chunk), (unsigned)plan_slices(E)), block(64 * PLAN_W);
    int bits = 0;
    while ((int64_t{1} << bits) < (E < PLAN_E ? E : PLAN_E)) ++bits;
    if (E <= PLAN_E)
      hipLaunchKernelGGL(k_expert_count<false>, chunks, block, 0, stream, ids, (int)n, chunk, (int)E, counts);
    else
      hipLaunchKernelGGL(k_expert_count<true>, chunks, block, 0, stream, ids, (int)n, chunk, (int)E, counts);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (E <= PLAN_E)
      hipLaunchKernelGGL(k_expert_place<false>, chunks, block, 0, stream, ids, (int)n, chunk, token, (int)E, bits,
                         counts, row_index, slot, offsets);
    else
      hipLaunchKernelGGL(k_expert_place<true>, chunks, block, 0, stream, ids, (int)n, chunk, token, (int)E, bits,
                         counts, row_index, slot, offsets);
    return hipGetLastError();
  }
  if (plan_by_four(n, E))
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
