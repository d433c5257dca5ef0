"""Norm of each head and rotation by position, with their gradients, in float64 (oracle; test infrastructure only).

Heads are [heads, tokens, head_dim]; `turn` holds scale e^{i angle} for [tokens, pairs].
"""
import numpy as np

EPS = 2.0 ** -24


def turns(positions, inv_freq, sections=None, scale=1.0):
    """scale e^{i position inv_freq} [tokens, pairs]; positions [tokens] or [tokens, axes]."""
    p = np.asarray(positions, np.float64)
    f = np.asarray(inv_freq, np.float64)
    if p.ndim == 1:
        p = p[:, None]
        axis = np.zeros(len(f), int)
    else:
        axis = np.repeat(np.arange(len(sections)), sections)
    return scale * np.exp(1j * (p[:, axis] * f[None, :]))


def rotate(v, turn, interleaved):
    """The pairs of the first 2 turn.shape[1] channels, as complex numbers, times turn."""
    n = turn.shape[1]
    out = np.array(v, np.float64)
    a, b = (v[..., 0:2 * n:2], v[..., 1:2 * n:2]) if interleaved else (v[..., :n], v[..., n:2 * n])
    z = (a + 1j * b) * turn
    if interleaved:
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = z.real, z.imag
    else:
        out[..., :n], out[..., n:2 * n] = z.real, z.imag
    return out


def pair_sum(v, n, scale, interleaved):
    """scale (|a| + |b|) at both channels of a pair, |v| elsewhere: what errors of a rotation are measured by."""
    out = np.abs(v)
    a, b = (out[..., 0:2 * n:2], out[..., 1:2 * n:2]) if interleaved else (out[..., :n], out[..., n:2 * n])
    s = scale * (a + b)
    if interleaved:
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = s, s
    else:
        out[..., :n], out[..., n:2 * n] = s, s
    return out


def forward(x, weight, turn, interleaved, eps, norm=True):
    """(y, bound for a bf16 result).  In fp32 the mean of D squares is off by (D + 2) 2^-24 of itself, its square root
    by half of that, the reciprocal root, two products, the angle's cosine and sine (2^-22 of 1) and the rotation's
    two products by one rounding each."""
    x = np.asarray(x, np.float64)
    D, n = x.shape[-1], turn.shape[1]
    scale = np.abs(turn).max() if n else 1.0
    v = x
    if norm:
        w = 1.0 if weight is None else np.asarray(weight, np.float64)
        v = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    y = rotate(v, turn, interleaved)
    err = ((D / 2 + 5 if norm else 0) + 8) * EPS * pair_sum(v, n, scale, interleaved)
    return y, err + 2.0 ** -8 * (np.abs(y) + err)


def backward(dy, x, weight, turn, interleaved, eps, norm=True):
    """((dx, bound for a bf16 result), (dweight, bound for an fp32 one)).  The sums over D and the factors are off by
    the roundings that forward counts; a sum over heads and tokens by at most their number of roundings."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    D, n = x.shape[-1], turn.shape[1]
    scale = np.abs(turn).max() if n else 1.0
    d = rotate(dy, np.conj(turn), interleaved)
    size = pair_sum(dy, n, scale, interleaved)
    if not norm:
        err = 8 * EPS * size
        return (d, err + 2.0 ** -8 * (np.abs(d) + err)), None
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (d * x * r).sum((0, 1))
    terms = x.shape[0] * x.shape[1]
    dw_err = (terms + D / 2 + 16) * EPS * (size * np.abs(x) * r).sum((0, 1))
    g = d * w
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdims=True))
    mag = size * np.abs(w)
    err = (2 * D + 24) * EPS * r * (mag + np.abs(x) * r * r * (mag * np.abs(x)).mean(-1, keepdims=True))
    return (dx, err + 2.0 ** -8 * (np.abs(dx) + err)), (dw, dw_err)
