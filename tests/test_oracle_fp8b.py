"""Pins of the block-scaled fp8 oracle, its gated block and gradients."""
from fractions import Fraction

import numpy as np
import pytest

from helpers import adversarial_rows
from oracle import fp8b
from oracle.formats import bf16_bits_to_f32, e4m3_decode, e4m3_encode, f32_to_bf16_bits
from oracle.quant import quant_fp8_row


def bits(a):
    return f32_to_bf16_bits(np.asarray(a, np.float32))


@pytest.mark.parametrize("K", [16, 128, 144, 400])
def test_row_blocks_against_the_row_scheme(K):
    # each block by itself is a row of the fp8 row scheme, which has pins of its own, but for how the scale is rounded:
    # one step up at most, and codes move where the quotient lies next to a border between two
    x = adversarial_rows(K, seed=K)
    q, s = fp8b.quant_act(x)
    for b in range(0, K, 128):
        wq, ws = quant_fp8_row(x[:, b:b + 128])
        up = s[:, b // 128].view(np.int32).astype(np.int64) - ws.view(np.int32)
        assert ((up >= 0) & (up <= 1)).all()
        same, moved = q[:, b:b + 128][up == 0], np.abs(q[:, b:b + 128].astype(int) - wq)[up == 1]
        assert np.array_equal(same, wq[up == 0]) and (moved <= 1).all()


def test_scale_against_rationals():
    # every significand of bf16: the product with the fp32 number next to 1 / 448, rounded to nearest
    c = Fraction(float(np.float32(1) / np.float32(448)))
    assert abs(c - Fraction(1, 448)) * 448 < Fraction(1, 2 ** 24)
    x = np.zeros((128, 128), np.uint16)
    x[:, 3] = 0x3F80 + np.arange(128)
    s = fp8b.quant_act(x)[1][:, 0]
    for m, got in zip(range(128, 256), s):
        want = Fraction(m, 128) * c
        step = Fraction(float(np.spacing(got)))
        assert abs(Fraction(float(got)) - want) * 2 <= step


@pytest.mark.parametrize("p", [-120, -8, 0, 30, 119])
def test_scale_of_a_largest_code_is_exact(p):
    x = np.zeros((1, 128), np.uint16)
    x[0, 0] = bits(448.0 * 2.0 ** p)
    assert fp8b.quant_act(x)[1][0, 0] == np.float32(2.0 ** p)


def test_weight_blocks_share_one_scale():
    rng = np.random.default_rng(0)
    w = bits(rng.standard_normal((300, 272)) * 0.02)
    q, s = fp8b.quant_weight(w)
    assert s.shape == (3, 3)
    for i in range(3):
        for j in range(3):
            blk = w[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            top = np.abs(bf16_bits_to_f32(blk)).max()
            assert s[i, j] == top * (np.float32(1) / np.float32(448))
            want = e4m3_encode((bf16_bits_to_f32(blk) / s[i, j]).astype(np.float32))
            assert np.array_equal(q[128 * i:128 * i + 128, 128 * j:128 * j + 128], want)


def test_zero_block_and_largest_code():
    x = np.zeros((2, 256), np.uint16)
    x[0, :128:3] = 0x8000
    x[1, 5] = bits(-3.0)
    q, s = fp8b.quant_act(x)
    assert s[0].tolist() == [0, 0] and set(q[0, :128].tolist()) == {0, 0x80} and not q[0, 128:].any()
    assert s[1, 0] == np.float32(3) * (np.float32(1) / np.float32(448)) and q[1, 5] == 0xFE and s[1, 1] == 0


def test_linear_against_rationals():
    rng = np.random.default_rng(1)
    M, K, N = 2, 144, 3
    xq, xs = fp8b.quant_act(bits(rng.standard_normal((M, K))))
    wq, ws = fp8b.quant_weight(bits(rng.standard_normal((N, K))))
    y, _ = fp8b.linear(fp8b.dequant_act(xq, xs), fp8b.dequant_weight(wq, ws))
    xv, wv = e4m3_decode(xq), e4m3_decode(wq)
    for m in range(M):
        for n in range(N):
            t = sum(Fraction(float(xv[m, k])) * Fraction(float(wv[n, k])) * Fraction(float(xs[m, k // 128])) *
                    Fraction(float(ws[0, k // 128])) for k in range(K))
            assert abs(float(t) - y[m, n]) <= 1e-13 * (1 + abs(float(t)))


def test_exact_operands_are_exact():
    rng = np.random.default_rng(2)
    x, w, s, y = fp8b.exact_operands(rng, 5, 1040, 140)
    q, xs = fp8b.quant_act(x)
    assert np.array_equal(fp8b.dequant_act(q, xs), bf16_bits_to_f32(x).astype(np.float64))
    assert set(np.unique(np.abs(e4m3_decode(q)))) <= {0.0, 448.0}
    unit = np.abs(y) / 112.0
    assert np.array_equal(unit, np.rint(unit)) and unit.max() < 2 ** 24


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_slopes_against_differences(act):
    v = np.linspace(-9, 9, 181)
    h = 1e-5
    d = (fp8b.act_ref(v + h, act) - fp8b.act_ref(v - h, act)) / (2 * h)
    assert np.abs(d - fp8b.slope_ref(v, act)).max() < 1e-8
    assert np.abs(fp8b.slope_ref(np.linspace(-20, 20, 4001), act)).max() < fp8b.MAX_SLOPE
    big = np.array([-1e6, -80.0, 80.0, 1e6])
    assert np.allclose(fp8b.slope_ref(big, act), [0, 0, 1, 1], atol=1e-30)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_gradients_against_differences(act):
    rng = np.random.default_rng(3)
    M, K, H = 3, 6, 5
    x, wg, wu = rng.standard_normal((M, K)), rng.standard_normal((H, K)), rng.standard_normal((H, K))
    dh = rng.standard_normal((M, H))

    def loss(x, wg, wu):
        return (fp8b.act_ref(x @ wg.T, act) * (x @ wu.T) * dh).sum()

    (dg, _), (du, _) = fp8b.gate_gradients(dh, x @ wg.T, x @ wu.T, act)
    want = [dg @ wg + du @ wu, dg.T @ x, du.T @ x]
    for i, got in enumerate(want):
        args = [x, wg, wu]
        num = np.zeros_like(got)
        for j in np.ndindex(got.shape):
            at = [a.copy() for a in args]
            at[i][j] += 1e-6
            up = loss(*at)
            at[i][j] -= 2e-6
            num[j] = (up - loss(*at)) / 2e-6
        assert np.abs(num - got).max() < 1e-7


def test_code_error_bounds_the_codes():
    x = adversarial_rows(272, seed=9)[:9]
    v = fp8b.dequant_act(*fp8b.quant_act(x))
    # below the normal fp32 range a scale is not accurate to 2^-23
    top = np.abs(bf16_bits_to_f32(x)).max(1) > 1e-30
    assert (np.abs(v - bf16_bits_to_f32(x))[top] <= fp8b.code_error(x)[top]).all()


def test_bounds_catch_planted_errors():
    # a block's scale taken from its neighbour, a missing block, a transposed pair of channels: each outside the bound
    rng = np.random.default_rng(4)
    a = fp8b.dequant_act(*fp8b.quant_act(bits(rng.standard_normal((4, 512)))))
    b = fp8b.dequant_weight(*fp8b.quant_weight(bits(rng.standard_normal((64, 512)))))
    y, err = fp8b.linear(a, b)
    lim = fp8b.rounded(err, y)
    for wrong in (np.concatenate([a[:, :128] * 1.05, a[:, 128:]], 1), np.concatenate([a[:, :384], 0 * a[:, 384:]], 1),
                  np.concatenate([a[:, 1:2], a[:, :1], a[:, 2:]], 1)):
        assert (np.abs(wrong @ b.T - y) > lim).any()
