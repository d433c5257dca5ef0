"""Block-scaled fp8 linears, the gated feed-forward block on them with its backward, and the gradient of a weight
(oracle; test infrastructure only).

The format and rules are this library's (each listed, with its reason, in the design notes):

* a block is 128 channels of a row of x, or 128 x 128 of a weight; what is left at the end is a block too;
* s = max |v| times fp32(1 / 448), in fp32 (how torch divides a tensor by 448 on the GPU), codes E4M3(v / s) with a
  correctly rounded fp32 division; a zero block has s = 0 and signed-zero codes;
* y = bf16(sum of the products of the codes' values), defined as dequantize-then-multiply in float64;
* gated: h = act(g) u of two such linears; its backward takes g and u in bf16, rounds dg and du to bf16, and
  multiplies their codes by the weights.
"""
import math

import numpy as np

from .formats import bf16_bits_to_f32, e4m3_decode, e4m3_encode, f32_to_bf16_bits
from .reference import gemm_gamma_fp8_dot

F32 = np.float32
B = 128
HALF_BF16 = 2.0 ** -8  # half a bf16 step, relative


def _codes(v, s):
    """E4M3 codes of float32 v under a scale s (float32, broadcast)."""
    with np.errstate(divide="ignore", invalid="ignore"):
        q = (v / s).astype(F32)
    zero = np.where(np.signbit(v), F32(-0.0), F32(0.0))
    return e4m3_encode(np.where(s > 0, q, zero).astype(F32))


def quant_act(x_bits):
    """bf16 [M, K] -> (codes uint8 [M, K], scales float32 [M, ceil(K / 128)])."""
    x = bf16_bits_to_f32(x_bits)
    M, K = x.shape
    s = np.stack([np.max(np.abs(x[:, k:k + B]), axis=1) for k in range(0, K, B)], 1)
    s = (s * (F32(1.0) / F32(448.0))).astype(F32)
    return _codes(x, np.repeat(s, B, axis=1)[:, :K]), s


def quant_weight(w_bits):
    """bf16 [N, K] -> (codes uint8 [N, K], scales float32 [ceil(N / 128), ceil(K / 128)])."""
    w = bf16_bits_to_f32(w_bits)
    N, K = w.shape
    s = np.array([[np.max(np.abs(w[n:n + B, k:k + B])) for k in range(0, K, B)] for n in range(0, N, B)], F32)
    s = (s * (F32(1.0) / F32(448.0))).astype(F32)
    return _codes(w, spread(s, N, K)), s


def spread(s, N, K):
    """Block scales of a weight, one for each element."""
    return np.repeat(np.repeat(s, B, axis=0)[:N], B, axis=1)[:, :K]


def dequant_act(q, s):
    return e4m3_decode(q) * np.repeat(np.asarray(s, np.float64), B, axis=1)[:, :q.shape[1]]


def dequant_weight(q, s):
    return e4m3_decode(q) * spread(np.asarray(s, np.float64), *q.shape)


def gamma(K):
    """Floor of the sums, in units of sum |products|: a block's 128 products by the fp8 dot unit, one rounding of
    the product of two scales, one fma a block, and at most 16 partial sums added up (fp32 roundings)."""
    return gemm_gamma_fp8_dot(B) + (math.ceil(K / B) + 18) * 2.0 ** -24


def linear(a, b):
    """(float64 a b^T, bound on an fp32 result's error) of dequantized operands."""
    return a @ b.T, gamma(a.shape[1]) * (np.abs(a) @ np.abs(b).T)


def rounded(err, ref):
    """The bound of a value rounded to bf16: half a step of what it can have been."""
    return err + HALF_BF16 * (np.abs(ref) + err)


# ---- activations -----------------------------------------------------------------------------------
def _sigma(v):
    return np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


C0 = math.sqrt(2.0 / math.pi)


def _exponent(v, act):
    """act(v) = v sigma(exponent)."""
    return v if act == "silu" else 2.0 * C0 * (v + 0.044715 * v ** 3)


def act_ref(v, act):
    return v * _sigma(_exponent(v, act))


def slope_ref(v, act):
    e = _exponent(v, act)
    d = 1.0 if act == "silu" else 2.0 * C0 * (1.0 + 3.0 * 0.044715 * v * v)
    s = _sigma(e)
    with np.errstate(over="ignore", invalid="ignore"):
        return s + np.where(np.abs(e) < 700, v * d, 0.0) * s * _sigma(-e)


def sigma_error(v, act):
    """Relative error of an fp32 sigma(exponent): the exponent is off by up to four roundings of itself (2^-24
    each, two of them its constants'), exp2, the sum and the reciprocal by one unit in the last place (2^-23)."""
    return 2.0 ** -23 * (3.0 + 2.0 * np.abs(_exponent(v, act)))


# exp2 overflows or flushes past these exponents; what is lost there is below 1e-36
FLUSHED = 1e-36


def act_error(v, act):
    """Bound on the error of an fp32 act(v)."""
    e = np.minimum(sigma_error(v, act), 1.0)
    return np.abs(act_ref(v, act)) * (e + 2.0 ** -23) + FLUSHED


def slope_error(v, act):
    """Bound on the error of an fp32 act'(v): both terms off by their sigmas and four roundings."""
    x = np.clip(v, -12.0, 12.0) if act != "silu" else v
    e = np.minimum(sigma_error(x, act), 1.0)
    s, o = _sigma(_exponent(x, act)), _sigma(-_exponent(x, act))
    d = 1.0 if act == "silu" else 2.0 * C0 * (1.0 + 3.0 * 0.044715 * x * x)
    return (e + 2.0 ** -22) * (s + 2.0 * np.abs(x * d) * s * o) + FLUSHED


MAX_SLOPE = 1.13  # of either activation


# ---- gated block -----------------------------------------------------------------------------------
def gated(x, wg, wu, act):
    """((h, bound), (g, bound), (u, bound)) of dequantized operands; bounds hold for the bf16 results."""
    g, eg = linear(x, wg)
    u, eu = linear(x, wu)
    a = act_ref(g, act)
    ea = act_error(g, act) + MAX_SLOPE * eg + 2.0 ** -22 * eg * (1 + np.abs(g))
    err = ea * (np.abs(u) + eu) + np.abs(a) * eu
    h = a * u
    err = err + 2.0 ** -24 * (np.abs(h) + err)
    return (h, rounded(err, h)), (g, rounded(eg, g)), (u, rounded(eu, u))


def gate_gradients(dh, g, u, act):
    """((dg, bound), (du, bound)) of float64 dh, g, u; bounds hold for the bf16 results."""
    dg, du = dh * u * slope_ref(g, act), dh * act_ref(g, act)
    eg = np.abs(dh * u) * slope_error(g, act) + 3 * 2.0 ** -24 * np.abs(dg)
    eu = np.abs(dh) * act_error(g, act) + 2.0 ** -24 * np.abs(du)
    return (dg, rounded(eg, dg)), (du, rounded(eu, du))


def gated_input_grad(dg_bits, du_bits, wg, wu):
    """(dx, bound) from the bf16 gradients of the projections and dequantized weights [H, K]."""
    d = [dequant_act(*quant_act(b)) for b in (dg_bits, du_bits)]
    dx = d[0] @ wg + d[1] @ wu
    err = 2 * gamma(2 * wg.shape[0]) * (np.abs(d[0]) @ np.abs(wg) + np.abs(d[1]) @ np.abs(wu))
    return dx, rounded(err, dx)


def code_error(x_bits):
    """Bound on |x - its quantized value|: half a step of a normal code (2^-4 of the value), or of the
    subnormal grid (2^-10 scales), and the quotient's rounding."""
    x = np.abs(bf16_bits_to_f32(x_bits).astype(np.float64))
    s = np.repeat(quant_act(x_bits)[1].astype(np.float64), B, axis=1)[:, :x.shape[1]]
    return np.maximum(x * 2.0 ** -4, s * 2.0 ** -10) + x * 2.0 ** -23


def weight_grad(dy_bits, x_bits):
    """(float64 dy^T x, bound on an fp32 sum of M exact products in any order)."""
    dy, x = bf16_bits_to_f32(dy_bits).astype(np.float64), bf16_bits_to_f32(x_bits).astype(np.float64)
    return dy.T @ x, dy.shape[0] * 2.0 ** -24 * (np.abs(dy).T @ np.abs(x))


def exact_operands(rng, M, K, N):
    """x (bf16 bits), codes and scales of a weight whose linear is exact in fp32 in any order, with the result's
    bits: x is 0 or +-448 2^p with a p of its own for each block, so its codes are 0 or +-448 under the scale 2^p,
    and the weight's codes are 0, +-1, +-2 under power-of-two scales.  Sums are multiples of 448 / 4 below 2^24 of
    that unit for K <= 2^14."""
    kb, nb = -(-K // B), -(-N // B)
    p = rng.integers(-1, 2, (M, kb))
    x = 448.0 * np.repeat(2.0 ** p, B, axis=1)[:, :K] * rng.integers(-1, 2, (M, K))
    for b in range(kb):  # every block has its largest value
        x[:, b * B] = 448.0 * 2.0 ** p[:, b]
    w = rng.integers(-2, 3, (N, K)).astype(F32)
    s = (2.0 ** rng.integers(-1, 2, (nb, kb))).astype(F32)
    y = x @ (w.astype(np.float64) * spread(s.astype(np.float64), N, K)).T
    return f32_to_bf16_bits(x.astype(F32)), e4m3_encode(w), s, y
