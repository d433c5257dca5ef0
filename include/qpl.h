/*
 * qpl.h - C ABI of the MI355X (gfx950) quantized linear library (libqpl.so).
 *
 * The operations are those of the two checkpoint schemes in the Diffusers guide
 * "BFL (fp8r / nvfp4)" (intro bullets and the "Kernels" section), plus the
 * low-rank branch of SVDQuant ("Bringing Nunchaku 4-bit Diffusion Inference to
 * Diffusers", section "Background: SVDQuant and Nunchaku").
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Tensors are dense, row-major, in device memory owned by the caller.  The
 *   library allocates nothing and keeps no pointer after a call returns.
 * - bf16 values travel as their 16-bit patterns (uint16_t).
 * - E4M3 is the OCP FP8 E4M3 encoding (bias 7, largest finite 448, NaN only at
 *   S.1111.111, no infinity).  E2M1 is the OCP MX FP4 element type (magnitudes
 *   0, 0.5, 1, 1.5, 2, 3, 4, 6).  Encoders round to nearest even, saturate at the
 *   largest finite magnitude and keep the sign of zero.
 * - A linear is y[M,N] = x[M,K] * W[N,K]^T (the nn.Linear layout).
 * - Packed E2M1: byte j of a row holds element 2j in its low nibble and element
 *   2j+1 in its high nibble.  Block scales are row-major [rows, K/16].
 * - `stream` is a hipStream_t (NULL = the default stream).  Work is queued on it
 *   and the call returns without waiting; no entry point synchronizes the host.
 * - Arguments are checked on the host before anything is queued; a bad argument
 *   returns a non-zero status and touches no memory.  Checks: non-NULL pointers,
 *   16-byte aligned pointers, M, N >= 1, K >= 16 and K % 16 == 0, scalars finite
 *   and > 0, workspace large enough, and a current HIP device that is gfx950.
 * - Size limits of the linears (QPL_ERR_SHAPE beyond them): the GEMMs address a
 *   256-row tile of an operand with 32-bit offsets below 2^30, so K < 2^22 for
 *   fp8r and INT4 (K-byte rows) and K < 2^23 for nvfp4 (K/2-byte rows); INT8 has
 *   K <= 2^17, which keeps its int32 sums exact, FP8B K < 2^22; with a
 *   low-rank branch (R > 0) K <= 2^21 and the activation's scales (8 M ceil(K/128)
 *   bytes for nvfp4, 4 M K/64 for INT4) below 2^31 bytes.
 * - Inputs must be finite: NaN or infinity in x or W is outside the contract.
 * - Faults inside a kernel surface at the caller's next synchronization.
 */
#ifndef QPL_H
#define QPL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QPL_OK = 0,
  QPL_ERR_NULL = 1,      /* a required pointer is NULL */
  QPL_ERR_SHAPE = 2,     /* M or N < 1, K < 16, K % 16 != 0, R outside [0, 128], or a size overflows */
  QPL_ERR_ALIGN = 3,     /* a pointer is not 16-byte aligned (4-byte for the arrays that say so) */
  QPL_ERR_ARG = 4,       /* a scale is not finite and > 0, unknown scheme, or low-rank pointers inconsistent with R */
  QPL_ERR_WORKSPACE = 5, /* ws_bytes < qlinear_workspace_bytes(...) */
  QPL_ERR_DEVICE = 6,    /* no HIP device, or the current device is not gfx950 */
  QPL_ERR_LAUNCH = 7     /* the HIP runtime rejected a kernel launch */
} qpl_status;

typedef enum { QPL_FP8R = 0, QPL_NVFP4 = 1, QPL_INT4 = 2, QPL_INT8 = 3, QPL_FP8B = 4 } qpl_scheme;

/*
 * Row-wise FP8 quantization (guide "BFL (fp8r / nvfp4)", intro bullet on fp8r:
 * activations are quantized per row to E4M3 at run time).  The same routine
 * quantizes a weight [N,K] into `weight` / `weight_scale`.
 *   x        bf16 [M,K]            input
 *   x_q      uint8 E4M3 [M,K]      out: codes, E4M3(x / s[m]) with a correctly
 *                                  rounded fp32 division
 *   x_scale  float [M]             out: s[m] = max_k |x[m,k]| / 448 (fp32); an
 *                                  all-zero row gives s = 0 and signed-zero codes
 */
qpl_status quant_act_fp8_row(const uint16_t* x, int64_t M, int64_t K,
                             uint8_t* x_q, float* x_scale, void* stream);

/*
 * NVFP4 quantization under a global scale g (guide, intro bullet on nvfp4: packed
 * E2M1 values with an E4M3 scale per 16 elements and a calibrated fp32
 * `input_scale`).  With g = weight_scale_2 the same routine quantizes a weight.
 * Per 16-element block: sf = E4M3(bmax / (6 g)), d = dec(sf) * g (fp32),
 * codes E2M1(x / d) (signed zeros when d == 0).
 *   x              bf16 [M,K]                  input
 *   input_scale    g, finite and > 0, with 6 g finite in fp32 (else QPL_ERR_ARG)
 *   smooth         float [K] or NULL: SVDQuant smoothing factors (Nunchaku post,
 *                  "Background: SVDQuant and Nunchaku": activation outliers move
 *                  into the weights, whose column k carries smooth[k]).  When
 *                  given, the quantized activation is x_hat[m,k] =
 *                  bf16_rne(x[m,k] / smooth[k]) (correctly rounded fp32
 *                  division).  The factors are device data the call does not
 *                  check: they must be positive and finite and every x / smooth
 *                  finite in bf16; otherwise the codes are unspecified.
 *   x_q            uint8 [M,K/2]               out: packed E2M1 codes
 *   x_block_scale  uint8 E4M3 [M,K/16]         out: block scales
 * All pointers 16-byte aligned (smooth too when not NULL).
 */
qpl_status quant_act_nvfp4(const uint16_t* x, int64_t M, int64_t K, float input_scale,
                           const float* smooth, uint8_t* x_q, uint8_t* x_block_scale, void* stream);

/*
 * fp8r linear (guide, "Kernels" table, fp8r row: a row-wise scaled FP8 GEMM):
 *   y[m,n] = bf16_rne( sum_k dec(xq[m,k]) dec(w[n,k]) * s_x[m] * weight_scale[n] )
 * with xq, s_x from quant_act_fp8_row(x), fp32 accumulation.
 *   weight        uint8 E4M3 [N,K]
 *   weight_scale  float [N]
 *   y             bf16 [M,N]          out
 *   ws, ws_bytes  scratch of at least qlinear_workspace_bytes(QPL_FP8R, M, K, N, 0)
 */
qpl_status qlinear_fp8r(const uint16_t* x, int64_t M, int64_t K, int64_t N,
                        const uint8_t* weight, const float* weight_scale,
                        uint16_t* y, void* ws, size_t ws_bytes, void* stream);

/*
 * qlinear_fp8r without a workspace argument and without any allocation, for callers
 * that cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc).  Same arguments, checks, kernels and
 * results as qlinear_fp8r; the workspace is instead a static device array of
 * QPL_NOALLOC_SCRATCH_BYTES inside the library, one per GPU, held from the first call
 * on that GPU (which looks up its address) until the process ends.
 *   Limit: the fp8r workspace, 256 ceil(M K / 256) + 256 ceil(4 M / 256) bytes, must
 *   fit in QPL_NOALLOC_SCRATCH_BYTES (32 MiB: M K up to about 33.5 M, e.g. 9216 x 3072),
 *   else QPL_ERR_WORKSPACE and nothing is queued.
 *   Sharing: every call on one GPU uses that GPU's one array, so calls that overlap on
 *   one GPU (different streams, or different threads without ordering) race and give
 *   undefined results; calls in one stream are ordered and safe.  Nothing in the array
 *   needs to start at zero; it keeps the last call's quantized activation.
 * No hipMalloc, hipFree, event or other allocating call is made; kernel timing
 * (qpl_timing_enable) does not cover this entry point.
 */
#define QPL_NOALLOC_SCRATCH_BYTES (32u << 20)
qpl_status qlinear_fp8r_noalloc(const uint16_t* x, int64_t M, int64_t K, int64_t N,
                                const uint8_t* weight, const float* weight_scale,
                                uint16_t* y, void* stream);

/*
 * nvfp4 linear (guide, "Kernels" table, nvfp4 row: an activation quantize followed
 * by a block-scaled FP4 GEMM), optionally with the SVDQuant low-rank branch:
 *   y = bf16_rne( input_scale * weight_scale_2 *
 *                 sum_b sx[m,b] sw[n,b] sum_{k in b} e2m1(xq) e2m1(w)  +  (x L1) L2 )
 * where xq, sx come from quant_act_nvfp4(x, input_scale, smooth) and the low-rank
 * term is accumulated in fp32 before the single rounding to bf16.  With smooth,
 * x in both terms is the smoothed x_hat that quant_act_nvfp4 defines (the
 * weight and L1 of such a layer were built for x_hat).
 *   weight          uint8 [N,K/2]        packed E2M1
 *   weight_scale    uint8 E4M3 [N,K/16]
 *   weight_scale_2  global weight scale, finite and > 0
 *   input_scale     calibrated activation scale, finite and > 0, 6 * input_scale finite;
 *                   the product input_scale * weight_scale_2 must be a normal fp32
 *                   number (else QPL_ERR_ARG); it scales the fp32 4-bit product
 *   smooth          float [K] smoothing factors or NULL (as in quant_act_nvfp4)
 *   lora_down       bf16 [K,R] (L1) or NULL when R == 0
 *   lora_up         bf16 [R,N] (L2) or NULL when R == 0
 *   R               rank, 0..128
 *   y               bf16 [M,N]          out
 *   ws, ws_bytes    scratch of at least qlinear_workspace_bytes(QPL_NVFP4, M, K, N, R);
 *                   after the call it holds the quantized activation the GEMM read:
 *                   its first M K/2 bytes are the packed codes (identical to
 *                   quant_act_nvfp4's x_q), and the 8 M S bytes from offset
 *                   256 ceil(M K/2 / 256) its block scales in the GEMM's slab-major
 *                   layout [S, M, 8], S = ceil(K/128): byte (s M + m) 8 + i is block
 *                   8 s + i of row m (quant_act_nvfp4's x_block_scale[m, 8 s + i]),
 *                   zero for 8 s + i >= K/16.
 * The GEMM multiplies the packed operands as they are: E2M1 codes and E4M3 block
 * scales are expanded in registers to exact f16 values and summed in fp32 on the
 * MFMA units.  With R > 0 the 4-bit product is scaled by input_scale *
 * weight_scale_2 before the low-rank term is added.
 */
qpl_status qlinear_nvfp4(const uint16_t* x, int64_t M, int64_t K, int64_t N,
                         const uint8_t* weight, const uint8_t* weight_scale,
                         float weight_scale_2, float input_scale, const float* smooth,
                         const uint16_t* lora_down, const uint16_t* lora_up, int64_t R,
                         uint16_t* y, void* ws, size_t ws_bytes, void* stream);

/*
 * INT4 variant of the SVDQuant W4A4 linear (Nunchaku post, "Introducing Nunchaku
 * Lite": svdq_w4a4 comes in INT4 and NVFP4 variants; the post gives no INT4
 * format, this library's):
 *   codes          signed 4-bit two's complement, channel 2j in the low nibble of
 *                  byte j: uint8 [rows, K/2]
 *   scales         float [rows, K/64], one per group of 64 channels
 *   rule           s = amax / 7 (fp32), q = clamp(rint(x / s), -8, 7) with a
 *                  correctly rounded division, ties to even; an all-zero group
 *                  has s = 0 and codes 0.  The same rule quantizes a weight.
 * quant_act_int4: x bf16 [M,K] (K % 64 == 0) -> x_q, x_scale; with smooth
 *   (float [K] or NULL, as in quant_act_nvfp4) the quantized activation is
 *   bf16_rne(x / smooth).
 * qlinear_int4:
 *   y = bf16_rne( sum_g sx[m,g] sw[n,g] sum_{k in g} qx qw  +  (x L1) L2 )
 *   with qx, sx from quant_act_int4(x, smooth), fp32 accumulation, and the
 *   low-rank term (x replaced by the smoothed x when smooth is given) added
 *   before the single rounding.  weight uint8 [N,K/2], weight_scale float
 *   [N,K/64], lora_down / lora_up / R as in qlinear_nvfp4; ws of at least
 *   qlinear_workspace_bytes(QPL_INT4, M, K, N, R).
 * All pointers 16-byte aligned.
 */
qpl_status quant_act_int4(const uint16_t* x, int64_t M, int64_t K, const float* smooth,
                          uint8_t* x_q, float* x_scale, void* stream);
qpl_status qlinear_int4(const uint16_t* x, int64_t M, int64_t K, int64_t N,
                        const uint8_t* weight, const float* weight_scale, const float* smooth,
                        const uint16_t* lora_down, const uint16_t* lora_up, int64_t R,
                        uint16_t* y, void* ws, size_t ws_bytes, void* stream);

/*
 * Weight-only 4-bit linear with bf16 activations (Nunchaku post, "Introducing
 * Nunchaku Lite": the awq_w4a16 layer, 4-bit weights and 16-bit activations for
 * the memory-bound adaptive-normalization and modulation projections).  The post
 * gives no format; this library's:
 *   weight        uint8 [N,K/2]     codes q in 0..15, channel 2j in the low nibble of byte j
 *   weight_scale  bf16 [N,K/group]  one scale s per group of `group` input channels
 *   weight_zero   uint8 [N,K/group] one zero point z in 0..15 per group
 *   group         32, 64 or 128; K % group == 0 (else QPL_ERR_ARG / QPL_ERR_SHAPE)
 * The weight value is (q - z) * s, exact in fp32.
 *
 * quant_weight_awq: quantize a bf16 weight w [N,K] into that format.  Per group:
 *   hi = max(max w, 0), lo = min(min w, 0), s = bf16_rne(fp32((hi - lo) / 15)),
 *   z = clamp(rint(-lo / s), 0, 15), q = clamp(rint(w / s) + z, 0, 15)
 *   (fp32, correctly rounded divisions, ties to even); s == 0 gives q = z = 0.
 *   Activation-aware channel scaling, if any, is applied to w beforehand.
 *   The group spans (hi - lo) must be finite in fp32.
 *
 * qlinear_awq_w4a16: y[m,n] = bf16_rne( sum_k x[m,k] (q[n,k] - z[n,g]) s[n,g] ),
 *   g = k / group, fp32 accumulation.  x bf16 [M,K], y bf16 [M,N].  Built for
 *   small M (one row per image): the weight is streamed once per two rows of x.
 * All pointers 16-byte aligned.  No workspace.
 */
qpl_status quant_weight_awq(const uint16_t* w, int64_t N, int64_t K, int64_t group,
                            uint8_t* w_q, uint16_t* w_scale, uint8_t* w_zero, void* stream);
qpl_status qlinear_awq_w4a16(const uint16_t* x, int64_t M, int64_t K, int64_t N,
                             const uint8_t* weight, const uint16_t* weight_scale,
                             const uint8_t* weight_zero, int64_t group, uint16_t* y, void* stream);

/*
 * Model-specific epilogues (Nunchaku post, "Introducing Nunchaku Lite", first
 * paragraph: the original engine's fused QKV projections and fused GELU/MLP
 * kernels).  The *_ex calls are qlinear_fp8r / qlinear_nvfp4 / qlinear_int4 with an
 * epilogue descriptor `epi` (NULL: the plain call); everything else about them is
 * as documented above.
 *   act       QPL_ACT_GELU_TANH: y = bf16(gelu(v)) with v the layer's fp32 result
 *             and gelu(v) = v / 2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))), the tanh
 *             form used by DiT feed-forward blocks, evaluated in fp32 as
 *             v / (1 + exp(-2u)) through exp2 and a reciprocal (a few fp32 ulps)
 *   q, k, v   fused QKV projection (all three set, or all NULL): the weight is
 *             [W_q; W_k; W_v] (N = 3 heads head_dim rows) and row m of the result
 *             goes to q, k and v instead of y:
 *               part[(h tokens + token_offset + m) head_dim + e] = y[m, p d + h head_dim + e]
 *             for part p = 0, 1, 2 (q, k, v), head h, d = heads head_dim; each of
 *             q, k, v is bf16 [heads, tokens, head_dim] (the layout attention reads;
 *             token_offset places the rows, e.g. image tokens after text tokens).
 *             Requires head_dim a power of two in [8, 1024], 0 <= token_offset and
 *             token_offset + M <= tokens, 16-byte aligned q, k, v, and act NONE;
 *             y may then be NULL.  Rows of q, k, v outside the M written are left
 *             untouched.
 * Errors beyond the plain call's: QPL_ERR_ARG for an unknown act or act with QKV,
 * QPL_ERR_NULL for one or two of q, k, v, or for y NULL without them,
 * QPL_ERR_SHAPE for the QKV shape conditions above.
 */
typedef enum { QPL_ACT_NONE = 0, QPL_ACT_GELU_TANH = 1, QPL_ACT_SILU = 2 /* gated blocks only */ } qpl_act;

typedef struct {
  qpl_act act;
  uint16_t* q;
  uint16_t* k;
  uint16_t* v;
  int64_t heads, head_dim, tokens, token_offset;
} qpl_epilogue;

qpl_status qlinear_fp8r_ex(const uint16_t* x, int64_t M, int64_t K, int64_t N,
                           const uint8_t* weight, const float* weight_scale, const qpl_epilogue* epi,
                           uint16_t* y, void* ws, size_t ws_bytes, void* stream);
qpl_status qlinear_nvfp4_ex(const uint16_t* x, int64_t M, int64_t K, int64_t N,
                            const uint8_t* weight, const uint8_t* weight_scale,
                            float weight_scale_2, float input_scale, const float* smooth,
                            const uint16_t* lora_down, const uint16_t* lora_up, int64_t R,
                            const qpl_epilogue* epi, uint16_t* y, void* ws, size_t ws_bytes, void* stream);
qpl_status qlinear_int4_ex(const uint16_t* x, int64_t M, int64_t K, int64_t N,
                           const uint8_t* weight, const float* weight_scale, const float* smooth,
                           const uint16_t* lora_down, const uint16_t* lora_up, int64_t R,
                           const qpl_epilogue* epi, uint16_t* y, void* ws, size_t ws_bytes, void* stream);

/*
 * GELU MLP of nvfp4 layers (same post and paragraph: fused GELU/MLP kernels):
 *   h = bf16(gelu(fc1(x)))      fc1 as qlinear_nvfp4 with act GELU, [M,K] -> [M,H]
 *   y = fc2(h)                  fc2 as qlinear_nvfp4, [M,H] -> [M,N]
 * GELU runs in fc1's GEMM epilogue; fc2 quantizes h with its own smoothing, input
 * scale and (fused with the quantize) low-rank down-projection, then runs its GEMM.
 * The result equals the two layers called one after the other.  Either layer may
 * carry smoothing and a low-rank branch; each layer's tensors are as in
 * qlinear_nvfp4 (weight [rows, cols/2], weight_scale [rows, cols/16], ...).
 * Workspace: qlinear_mlp_nvfp4_workspace_bytes(M, K, H, N, fc1->R, fc2->R) bytes (0
 * for invalid sizes); it starts with fc2's qlinear_nvfp4 workspace, so after the
 * call it holds fc2's quantized input as described there (codes, then slab-major
 * block scales), and the 2 M H bytes at offset qlinear_workspace_bytes(QPL_NVFP4,
 * M, H, N, fc2->R) hold h.  Errors: as qlinear_nvfp4 for either layer.
 */
typedef struct {
  const uint8_t* weight;        /* uint8 [rows, cols/2], two E2M1 codes per byte */
  const uint8_t* weight_scale;  /* E4M3 [rows, cols/16] */
  float weight_scale_2;
  float input_scale;
  const float* smooth;          /* float [cols] or NULL */
  const uint16_t* lora_down;    /* bf16 [cols, R] or NULL */
  const uint16_t* lora_up;      /* bf16 [R, rows] or NULL */
  int64_t R;
} qpl_nvfp4_layer;

size_t qlinear_mlp_nvfp4_workspace_bytes(int64_t M, int64_t K, int64_t H, int64_t N, int64_t R1, int64_t R2);
qpl_status qlinear_mlp_nvfp4(const uint16_t* x, int64_t M, int64_t K, int64_t H, int64_t N,
                             const qpl_nvfp4_layer* fc1, const qpl_nvfp4_layer* fc2,
                             uint16_t* y, void* ws, size_t ws_bytes, void* stream);

/*
 * 8-bit integer linear (W8A8): int8 codes with one fp32 scale per row of x (token)
 * and one per row of W (output channel).
 *   rule   a = max_k |x[m,k]|, s[m] = a / 127 (fp32, correctly rounded),
 *          q[m,k] = rint(127 x[m,k] / a) of the exact quotient, ties to even (so a code
 *          does not depend on how s was rounded); an all-zero row has s = 0 and
 *          codes 0.  The same rule quantizes a weight [N,K].
 * quant_act_int8: x bf16 [M,K] -> x_q int8 [M,K], x_scale float [M]; with smooth
 *   (float [K] or NULL, as in quant_act_nvfp4) the quantized activation is
 *   bf16_rne(x / smooth).
 * qlinear_int8: y[m,n] = bf16_rne((sum_k q_x q_w) s_x[m] weight_scale[n]), the sum
 *   exact in int32, with q_x, s_x from quant_act_int8(x, smooth).
 *   weight int8 [N,K], any codes in [-128, 127]; weight_scale float [N]; ws of at
 *   least qlinear_workspace_bytes(QPL_INT8, M, K, N, 0) bytes, which is 0 for a few rows
 *   (they are quantized inside the product's kernel; ws may then be NULL).
 * qlinear_int8_ex: the same with an epilogue (see qlinear_fp8r_ex).
 * All pointers 16-byte aligned.  K <= 2^17 for the linears (QPL_ERR_SHAPE beyond).
 */
qpl_status quant_act_int8(const uint16_t* x, int64_t M, int64_t K, const float* smooth,
                          int8_t* x_q, float* x_scale, void* stream);
qpl_status qlinear_int8(const uint16_t* x, int64_t M, int64_t K, int64_t N,
                        const int8_t* weight, const float* weight_scale, const float* smooth,
                        uint16_t* y, void* ws, size_t ws_bytes, void* stream);
qpl_status qlinear_int8_ex(const uint16_t* x, int64_t M, int64_t K, int64_t N,
                           const int8_t* weight, const float* weight_scale, const float* smooth,
                           const qpl_epilogue* epi, uint16_t* y, void* ws, size_t ws_bytes, void* stream);

/*
 * Mixture-of-experts linears on the 8-bit integer scheme.  E experts (1..65536), each
 * with its own weight; every token goes to topk of them (1..256).  Sizes: M, R, T topk
 * below 2^31 - 2^16.  Index and offset arrays are device data that the calls do not check:
 * whatever they hold, no call reads or writes outside the arrays it was given.
 *
 * expert_plan: sorts the router's choices by expert.
 *   expert_ids  int32 [T, topk]  expert of each choice; an id outside [0, E) (say -1)
 *                                means no expert
 *   row_index   int32 [T topk]   out: the token of each place in expert order; -1 behind the last
 *   slot        int32 [T, topk]  out: the place of each choice, -1 for no expert
 *   offsets     int32 [E + 1]    out: expert e has the places offsets[e] .. offsets[e+1] - 1
 *   Places of one expert are in order of (token, choice).
 *   ws          at least expert_plan_workspace_bytes(T, topk, E) bytes (0 for few choices of not
 *               too many experts: ws may then be NULL).  It may also be NULL with T topk < 32768 or
 *               E > 1024 if T topk E <= 2^35: the plan then reads all choices once per expert
 *
 * qlinear_grouped_int8: product row i of R, offsets[e] <= i < offsets[e+1], is
 *   y[i] = bf16_rne(act((sum_k q_x q_w[e]) s_x weight_scale[e]))
 *   with q_x, s_x the quantized row x[row_index[i]] (x[i] when row_index is NULL; then
 *   R <= M).  Experts may have any number of rows, none included.
 *   x             bf16 [M, K]
 *   row_index     int32 [R] or NULL; an index outside [0, M) stands for a row of zeros
 *   offsets       int32 [E + 1], nondecreasing, within [0, R] (else the rows' values are
 *                 unspecified); rows of y in no expert's range are left untouched
 *   weight        int8 [E, N, K], weight_scale float [E, N]
 *   act           QPL_ACT_NONE or QPL_ACT_GELU_TANH
 *   y             bf16 [R, N]
 *   ws            at least qlinear_grouped_int8_workspace_bytes(R, K, N, E) bytes
 *
 * expert_combine: out[t] = bf16_rne(sum_j weights[t,j] y[slot[t,j]]), fp32, j ascending;
 *   a slot outside [0, R) adds nothing (a token without experts gets zeros).
 *   y bf16 [R, N], slot int32 [T, topk], weights float [T, topk], out bf16 [T, N].
 *
 * qlinear_moe_int8: a GELU MLP of experts, all of the above in one call:
 *   plan of expert_ids; h = gelu(grouped(x, fc1)) with fc1 [E, H, K]; grouped(h, fc2) with
 *   fc2 [E, N, H]; y [T, N] = combine with expert_weights float [T, topk].  h and
 *   the experts' outputs are bf16.  ws of at least
 *   qlinear_moe_int8_workspace_bytes(T, topk, K, H, N, E).
 *
 * expert_ids, row_index, slot, offsets and the choices' weights need 4-byte alignment
 * (QPL_ERR_ALIGN), the other pointers 16-byte as usual.  Errors as for the linears:
 * QPL_ERR_SHAPE for E, topk or a size out of range, QPL_ERR_ARG for an unknown act.
 */
qpl_status expert_plan(const int32_t* expert_ids, int64_t T, int64_t topk, int64_t E,
                       int32_t* row_index, int32_t* slot, int32_t* offsets,
                       void* ws, size_t ws_bytes, void* stream);
size_t expert_plan_workspace_bytes(int64_t T, int64_t topk, int64_t E);
size_t qlinear_grouped_int8_workspace_bytes(int64_t R, int64_t K, int64_t N, int64_t E);
qpl_status qlinear_grouped_int8(const uint16_t* x, int64_t M, int64_t K, int64_t N, int64_t E,
                                const int8_t* weight, const float* weight_scale,
                                const int32_t* row_index, int64_t R, const int32_t* offsets, qpl_act act,
                                uint16_t* y, void* ws, size_t ws_bytes, void* stream);
qpl_status expert_combine(const uint16_t* y, int64_t R, int64_t N, const int32_t* slot,
                          const float* weights, int64_t T, int64_t topk, uint16_t* out, void* stream);
size_t qlinear_moe_int8_workspace_bytes(int64_t T, int64_t topk, int64_t K, int64_t H, int64_t N, int64_t E);
qpl_status qlinear_moe_int8(const uint16_t* x, int64_t T, int64_t K, int64_t H, int64_t N, int64_t E, int64_t topk,
                            const int32_t* expert_ids, const float* expert_weights,
                            const int8_t* fc1_weight, const float* fc1_scale,
                            const int8_t* fc2_weight, const float* fc2_scale,
                            uint16_t* y, void* ws, size_t ws_bytes, void* stream);

/*
 * Block-scaled fp8 (FP8B): E4M3 codes with an fp32 scale for every 128 channels of a row of x and for every
 * 128 x 128 block of a weight, the form that block-scaled checkpoints carry.
 *   rule   a = max |v| over the block, s = a * fp32(1 / 448) in fp32 (as torch evaluates a / 448 on the GPU; the
 *          row-wise rule above divides), codes E4M3(v / s) with a correctly rounded division; an all-zero block has
 *          s = 0 and signed-zero codes.  A last block holds what is left of K (or N).
 * quant_act_fp8b:    x bf16 [M,K] -> x_q uint8 [M,K], x_scale float [M, ceil(K/128)].
 * quant_weight_fp8b: w bf16 [N,K] -> w_q uint8 [N,K], w_scale float [ceil(N/128), ceil(K/128)]; K <= 2^31 - 128.
 * transpose_fp8b:    a quantized weight turned over: weight_t [K,N], weight_t_scale [ceil(K/128), ceil(N/128)]
 *                    (N % 16 == 0, K <= 2^31 - 128), the same values.  With it the gradient of a linear's input is a linear:
 *                    dx = qlinear_fp8b(dy, weight_t).
 * qlinear_fp8b:      y[m,n] = bf16_rne(sum_b x_scale[m,b] weight_scale[n/128,b] sum_{k in b} q_x q_w), with q_x and
 *                    x_scale from quant_act_fp8b(x).  A block's sum comes from the FP8 matrix instructions (which
 *                    cut each product below 2^-13 of the largest of its group of eight) and is folded into fp32
 *                    accumulators.  The product of two scales must not overflow fp32; below 2^-126 it
 *                    loses bits.
 * qlinear_fp8b_ex:   the same with an epilogue (see qlinear_fp8r_ex).
 *   ws   at least qlinear_workspace_bytes(QPL_FP8B, M, K, N, 0) bytes, which is 0 for a few rows (they are quantized
 *        inside the product's kernel; ws may then be NULL).
 * qlinear_gated_fp8b: a gated feed-forward block's first half in one product,
 *     g = x Wg^T, u = x Wu^T (as qlinear_fp8b, before their rounding),  h = bf16_rne(act(g) u)
 *   gate, up  weights [H,K] with scales [ceil(H/128), ceil(K/128)];  H % 16 == 0
 *   act       QPL_ACT_SILU or QPL_ACT_GELU_TANH, on fp32 values
 *   h         bf16 [M,H] out
 *   g, u      bf16 [M,H] out, what the backward pass needs, or both NULL
 *   ws        at least qlinear_gated_fp8b_workspace_bytes(M, K, H) bytes (0 for a few rows, as above)
 * qlinear_gated_fp8b_backward: from dh and the saved bf16 g, u (all [M,H]),
 *     dg = bf16_rne(dh u act'(g)),  du = bf16_rne(dh act(g)),
 *     dx = bf16_rne(Q(dg) Wg + Q(du) Wu),  Q the rule above over blocks of 128 of H (the rounding of x to its codes
 *     passes gradients through unchanged)
 *   gate_t, up_t  the weights turned over (transpose_fp8b): [K,H], scales [ceil(K/128), ceil(H/128)]
 *   dx            bf16 [M,K] out;  dg, du  bf16 [M,H] out (for qlinear_weight_grad), or both NULL; either may be dh, g
 *                 or u itself
 *   ws            at least qlinear_gated_fp8b_backward_workspace_bytes(M, K, H) bytes
 * qlinear_weight_grad: dw[n,k] = sum_m dy[m,n] x[m,k] of bf16 dy [M,N] and x [M,K], fp32 [N,K], summed in fp32: the
 *   gradient of any linear's weight.  N % 16 == 0 and K % 16 == 0, both at most 2^23.
 *
 * Codes, activations and workspaces need 16-byte alignment, arrays of scales 4-byte.  K < 2^22 (in the backward H
 * rounded up to 128 below 2^21).
 */
typedef struct {
  const uint8_t* weight;
  const float* weight_scale;
} qpl_fp8b_weight;

qpl_status quant_act_fp8b(const uint16_t* x, int64_t M, int64_t K, uint8_t* x_q, float* x_scale, void* stream);
qpl_status quant_weight_fp8b(const uint16_t* w, int64_t N, int64_t K, uint8_t* w_q, float* w_scale, void* stream);
qpl_status transpose_fp8b(const uint8_t* weight, const float* weight_scale, int64_t N, int64_t K, uint8_t* weight_t,
                          float* weight_t_scale, void* stream);
qpl_status qlinear_fp8b(const uint16_t* x, int64_t M, int64_t K, int64_t N, const uint8_t* weight,
                        const float* weight_scale, uint16_t* y, void* ws, size_t ws_bytes, void* stream);
qpl_status qlinear_fp8b_ex(const uint16_t* x, int64_t M, int64_t K, int64_t N, const uint8_t* weight,
                           const float* weight_scale, const qpl_epilogue* epi, uint16_t* y, void* ws, size_t ws_bytes,
                           void* stream);
size_t qlinear_gated_fp8b_workspace_bytes(int64_t M, int64_t K, int64_t H);
qpl_status qlinear_gated_fp8b(const uint16_t* x, int64_t M, int64_t K, int64_t H, const qpl_fp8b_weight* gate,
                              const qpl_fp8b_weight* up, qpl_act act, uint16_t* h, uint16_t* g, uint16_t* u, void* ws,
                              size_t ws_bytes, void* stream);
size_t qlinear_gated_fp8b_backward_workspace_bytes(int64_t M, int64_t K, int64_t H);
qpl_status qlinear_gated_fp8b_backward(const uint16_t* dh, const uint16_t* g, const uint16_t* u, int64_t M, int64_t K,
                                       int64_t H, const qpl_fp8b_weight* gate_t, const qpl_fp8b_weight* up_t,
                                       qpl_act act, uint16_t* dx, uint16_t* dg, uint16_t* du, void* ws,
                                       size_t ws_bytes, void* stream);
qpl_status qlinear_weight_grad(const uint16_t* dy, const uint16_t* x, int64_t M, int64_t N, int64_t K, float* dw,
                               void* stream);

/*
 * Norm of each head of the queries and keys, and the rotation by their positions, in one pass over what a fused QKV
 * projection wrote:
 *     n = x w / sqrt(mean over the head of x^2 + eps)      (norm != 0; w bf16 [head_dim], or NULL for ones)
 *     (a, b) -> scale (a cos t - b sin t, a sin t + b cos t),  t = position * inv_freq[i]
 *   for pair i of the first rotary_dim channels: channels (i, i + rotary_dim / 2), or (2 i, 2 i + 1) with
 *   interleaved.  The other channels are not rotated.  All in fp32 up to the one rounding of the result (the sum of a
 *   head's squares too: it overflows where values pass 2^59); angles in fp64, so that far positions keep theirs.
 * A tensor's element (head, token, channel) lies at head * head_stride + token * token_stride + channel; strides are
 * multiples of 8 elements.  heads up to 65536, head_dim a multiple of 16 up to 512.  The output may be the input
 * itself (same pointer and strides); other overlaps are not allowed, and a written view may not hold two elements in
 * one place (QPL_ERR_SHAPE).  q and k may have different numbers of heads; k may be NULL.
 *   rope  NULL (or rotary_dim 0): norm only.  positions int32 [tokens, axes]: with more than one axis (up to 4), the
 *         first sections[0] pairs turn by the first position of a token, the next sections[1] by the second, ... (they
 *         add up to rotary_dim / 2).  inv_freq float [rotary_dim / 2].  rotary_dim a multiple of 16 up to head_dim.
 *         scale, finite and > 0, multiplies the rotated channels.
 * qk_norm_rope_backward: per tensor x the saved input, y its output's gradient, dx (out) the input's gradient,
 *   dweight (out, float [head_dim], or NULL) the weight's, summed over heads and tokens in a fixed order.  dx may be x
 *   or y itself.  ws at least qk_norm_rope_backward_workspace_bytes(tokens, head_dim) bytes (may be NULL without any
 *   dweight).
 * Errors: QPL_ERR_ARG for eps or scale not finite and > 0, eps below 2^-126 (subnormal), a weight without norm, a
 * dweight without weight, neither norm nor rotation.
 * qpl_rope_frequencies (host): base^(-2 i / rotary_dim), scaled for contexts longer than the trained ones:
 *   LINEAR  divided by factor;   NTK  with base * factor^(rotary_dim / (rotary_dim - 2));
 *   YARN    channels that turn at most low_turns times over trained_tokens are divided by factor, those that turn at
 *           least high_turns times are kept, in between both are mixed, linearly in the number of turns (a ramp that
 *           is linear in the channel's index instead gives other frequencies), and *scale = 0.1 ln(factor) + 1 (else
 *           1).
 */
typedef struct {
  const uint16_t* x;
  uint16_t* y;
  int64_t heads;
  int64_t x_head_stride, x_token_stride, y_head_stride, y_token_stride;
  const uint16_t* weight;
  uint16_t* dx; /* backward only, like the rest */
  int64_t dx_head_stride, dx_token_stride;
  float* dweight;
} qpl_heads;

typedef struct {
  const int32_t* positions;
  const float* inv_freq;
  int64_t rotary_dim, axes;
  int64_t sections[4];
  int interleaved;
  float scale;
} qpl_rope;

typedef enum { QPL_ROPE_PLAIN = 0, QPL_ROPE_LINEAR = 1, QPL_ROPE_NTK = 2, QPL_ROPE_YARN = 3 } qpl_rope_kind;
typedef struct {
  qpl_rope_kind kind;
  double factor, trained_tokens, low_turns, high_turns;
} qpl_rope_scaling;

qpl_status qk_norm_rope(const qpl_heads* q, const qpl_heads* k, int64_t tokens, int64_t head_dim, int norm, float eps,
                        const qpl_rope* rope, void* stream);
size_t qk_norm_rope_backward_workspace_bytes(int64_t tokens, int64_t head_dim);
qpl_status qk_norm_rope_backward(const qpl_heads* q, const qpl_heads* k, int64_t tokens, int64_t head_dim, int norm,
                                 float eps, const qpl_rope* rope, void* ws, size_t ws_bytes, void* stream);
qpl_status qpl_rope_frequencies(int64_t rotary_dim, double base, const qpl_rope_scaling* scaling, float* inv_freq,
                                float* scale);

/*
 * Dequantize a weight to bf16 (guide, "Kernels" section, last paragraph: on other
 * devices the weight is dequantized to compute_dtype on every forward and the
 * layer runs as a regular linear; that linear is the caller's).
 *   QPL_FP8R:  weight uint8 E4M3 [N,K], weight_scale float [N];
 *              w[n,k] = bf16_rne(dec(w) * s[n])
 *   QPL_NVFP4: weight uint8 [N,K/2] packed E2M1, weight_scale uint8 E4M3 [N,K/16];
 *              w[n,k] = bf16_rne((e2m1(w) * dec(sf)) * weight_scale_2)
 *   weight_scale_2 is ignored for QPL_FP8R.
 *   w_bf16  bf16 [N,K]  out
 */
qpl_status dequant_weight(qpl_scheme scheme, const uint8_t* weight, const void* weight_scale,
                          float weight_scale_2, int64_t N, int64_t K,
                          uint16_t* w_bf16, void* stream);

/* Bytes of scratch that the scheme's linear needs for these sizes
 * (0 if the sizes are invalid, and for INT8 and FP8B also where none is needed).  The scratch may be reused between calls that
 * are ordered on one stream. */
size_t qlinear_workspace_bytes(qpl_scheme scheme, int64_t M, int64_t K, int64_t N, int64_t R);

/*
 * Calibration helper for the nvfp4 global scales (guide, intro bullet on nvfp4:
 * `weight_scale_2` and the calibrated `input_scale`).
 *   qpl_amax_bf16: *amax (device float) = max(*amax, max_i |x[i]|) over n >= 1
 *                  bf16 values; the caller sets *amax to 0 before the first batch.
 *                  x needs 16-byte alignment; amax needs 4-byte alignment.
 *   qpl_nvfp4_global_scale: amax / (448 * 6) in fp32 (host function).
 */
qpl_status qpl_amax_bf16(const uint16_t* x, int64_t n, float* amax, void* stream);
float qpl_nvfp4_global_scale(float amax);

/*
 * Per-kernel timing (a profiling aid, off by default).  While enabled, every kernel
 * launch of the library is bracketed by two HIP events recorded on the launch's
 * stream.  qpl_timing_collect_n waits for all recorded events, writes for each of the
 * first `count` kernel kinds the number of launches and their summed duration in
 * milliseconds since the previous collect (arrays of `count` entries, caller-owned
 * host memory; entries past QPL_KERNEL_COUNT become 0), and clears the records of all
 * kinds.  Events are created by the library on first use and reused.  Not
 * thread-safe with respect to concurrent collect calls.
 *   qpl_timing_collect: in source, the same with count = QPL_KERNEL_COUNT.  The exported
 *   function of that name has no count, so it writes the QPL_TIMING_COLLECT_KINDS kinds
 *   that it began with: programs built when there were no more have arrays of that size.
 * Errors: QPL_ERR_NULL, and QPL_ERR_ARG for a negative count.
 */
typedef enum {
  QPL_KERNEL_QUANT_FP8_ROW = 0,     /* fp8r activation / weight quantize */
  QPL_KERNEL_QUANT_NVFP4 = 1,       /* nvfp4 quantize to packed codes */
  QPL_KERNEL_QUANT_NVFP4_LINEAR = 2, /* nvfp4 quantize inside qlinear_nvfp4 (R = 0; slab-major scales),
                                        with the weight's block scales into the GEMM's layout */
  QPL_KERNEL_GEMM_FP8R = 3,
  QPL_KERNEL_GEMM_NVFP4 = 4,
  QPL_KERNEL_GEMM_NVFP4_LOWRANK = 5, /* nvfp4 GEMM with the low-rank epilogue */
  QPL_KERNEL_LOWRANK_PREP = 6,      /* low-rank factor transposes (qlinear_int4) */
  QPL_KERNEL_DEQUANT = 7,
  QPL_KERNEL_AMAX = 8,
  QPL_KERNEL_NVFP4_PREP = 9,        /* qlinear_nvfp4's preparation when R > 0: the weight's block scales
                                       into the GEMM's layout and the low-rank factor layouts */
  QPL_KERNEL_QUANT_NVFP4_LOWRANK = 10, /* nvfp4 quantize fused with x L1 (qlinear_nvfp4, R > 0) */
  QPL_KERNEL_QUANT_W4G = 11,        /* quant_weight_awq */
  QPL_KERNEL_GEMV_W4A16 = 12,       /* qlinear_awq_w4a16 */
  QPL_KERNEL_QUANT_INT4 = 13,       /* quant_act_int4, and the INT4 quantize inside qlinear_int4 (R = 0) */
  QPL_KERNEL_INT4_EXPAND = 14,      /* INT4 weight codes -> E4M3 bytes inside qlinear_int4 */
  QPL_KERNEL_GEMM_INT4 = 15,
  QPL_KERNEL_QUANT_INT4_LOWRANK = 16, /* INT4 quantize fused with x L1 (qlinear_int4, R > 0) */
  QPL_KERNEL_GEMM_EPILOGUE = 17,    /* any GEMM with a GELU or QKV epilogue (the *_ex calls, fc1 of
                                       qlinear_mlp_nvfp4) */
  QPL_KERNEL_QUANT_INT8 = 18,       /* quant_act_int8, and the quantize inside the 8-bit integer linears */
  QPL_KERNEL_GEMM_INT8 = 19,
  QPL_KERNEL_GEMM_INT8_GROUPED = 20,
  QPL_KERNEL_EXPERT_PLAN = 21,       /* expert_plan; in qlinear_moe_int8 with few choices also fc1's quantize */
  QPL_KERNEL_EXPERT_COMBINE = 22,
  QPL_KERNEL_QUANT_FP8B = 23,        /* quant_act_fp8b, quant_weight_fp8b, and the quantize inside the FP8B linears */
  QPL_KERNEL_GEMM_FP8B = 24,         /* also the product of the gated backward */
  QPL_KERNEL_GATED_FP8B = 25,
  QPL_KERNEL_GATED_BACKWARD = 26,    /* the gradients of both projections and their codes */
  QPL_KERNEL_TRANSPOSE_FP8B = 27,
  QPL_KERNEL_WEIGHT_GRAD = 28,
  QPL_KERNEL_QK_NORM_ROPE = 29,      /* both directions */
  QPL_KERNEL_COUNT = 30
} qpl_kernel;

void qpl_timing_enable(int on);
/* Time only the kernel kinds whose bit (1 << kind) is set in `kinds` (0 = off);
 * an event pair costs a few microseconds of stream time per timed launch. */
void qpl_timing_select(uint32_t kinds);
qpl_status qpl_timing_collect_n(int64_t* launches, double* total_ms, int count);
#define QPL_TIMING_COLLECT_KINDS 18
qpl_status qpl_timing_collect(int64_t* launches, double* total_ms);
#define qpl_timing_collect(launches, total_ms) qpl_timing_collect_n((launches), (total_ms), QPL_KERNEL_COUNT)

/* Static description of a status code. */
const char* qpl_status_str(qpl_status status);

#ifdef __cplusplus
}
#endif

#endif /* QPL_H */
