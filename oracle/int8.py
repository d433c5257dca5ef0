"""8-bit integer linears and the routing of tokens to experts (oracle; test
infrastructure only).

The format and rules are this library's (each listed, with its reason, in the
design notes):

* per row: a = max |x|, s = a / 127 (fp32, correctly rounded), q = rint(127 x / a) of
  the exact quotient, ties to even; a zero row has s = 0 and codes 0.  127 x is exact
  in float64 and a float64 quotient of it is a tie exactly when the real one is (a
  quotient of 8-bit significands is a tie or at least 1.5e-5 of itself away from one);
* the layer: y = bf16(act((sum_k q_x q_w) s_x s_w)), the sum exact;
* the plan: places in order of (expert, token, choice), ids outside the experts left out;
* the combination: sum over a token's choices of weight times row.
"""
import numpy as np

from .epilogue import gelu_interval
from .formats import bf16_bits_to_f32, f32_to_bf16_bits

F32 = np.float32


def quant_int8(x_bits):
    """Row-wise symmetric 8-bit quantization of a bf16 [R, K] tensor -> (int8 [R, K], float32 [R])."""
    x = bf16_bits_to_f32(x_bits)
    a = np.max(np.abs(x), axis=1)
    s = (a / F32(127.0)).astype(F32)
    q = np.zeros(x.shape, dtype=np.int8)
    live = a > 0
    q[live] = np.rint(127.0 * x[live].astype(np.float64) / a[live].astype(np.float64)[:, None]).astype(np.int8)
    return q, s


def sums(xq, wq):
    """Exact int64 [M, N] sums of products of the codes (float64 products and sums are exact below 2^53)."""
    return np.rint(np.asarray(xq, np.float64) @ np.asarray(wq, np.float64).T).astype(np.int64)


def qlinear_int8_bits(xq, xs, wq, ws):
    """bf16 bits of the layer without an activation: the int32 sum rounded to fp32, two fp32
    products, one rounding to bf16, which leaves one possible value for each element."""
    acc = sums(xq, wq).astype(F32)
    with np.errstate(over="ignore", under="ignore"):
        v = ((acc * np.asarray(xs, F32)[:, None]).astype(F32) * np.asarray(ws, F32)[None, :]).astype(F32)
    return f32_to_bf16_bits(v)


def qlinear_int8_ref(xq, xs, wq, ws):
    """float64 [M, N] of the layer without an activation."""
    return sums(xq, wq) * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)[None, :]


def gelu_bounds(ref):
    """[lo, hi] (float64) of gelu of the layer: three fp32 roundings (2^-24 of the value
    each) before it, its fp32 evaluation, and half a bf16 step (2^-8 of the value) after it."""
    lo, hi = gelu_interval(ref, 3 * 2.0 ** -24 * np.abs(ref))
    return lo - 2.0 ** -8 * np.abs(lo), hi + 2.0 ** -8 * np.abs(hi)


def plan_ref(ids, E):
    """(row_index [T k], slot [T, k], offsets [E + 1]) of router choices ids [T, k], one choice at a time."""
    T, k = ids.shape
    lists = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                lists[ids[t, j]].append((t, j))
    row_index = np.full(T * k, -1, np.int32)
    slot = np.full((T, k), -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    place = 0
    for e in range(E):
        offsets[e] = place
        for t, j in lists[e]:
            row_index[place] = t
            slot[t, j] = place
            place += 1
    offsets[E] = place
    return row_index, slot, offsets


def combine_ref(y_bits, slot, weights):
    """(float64 [T, N] sums, float64 [T, N] bound on the error of a bf16 result: the fp32 sum
    of k products loses at most k 2^-24 of the magnitudes, the result half a bf16 step)."""
    y = bf16_bits_to_f32(y_bits).astype(np.float64)
    T, k = slot.shape
    out = np.zeros((T, y.shape[1]))
    mag = np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= slot[t, j] < y.shape[0]:
                p = np.float64(weights[t, j]) * y[slot[t, j]]
                out[t] += p
                mag[t] += np.abs(p)
    return out, 2.0 ** -8 * np.abs(out) + k * 2.0 ** -24 * (1.0 + 2.0 ** -8) * mag
