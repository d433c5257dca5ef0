"""Pins for oracle.int8: the row max maps to +-127, grid values round-trip, every
quotient of bf16 significands against rationals (ties included), zero rows, a rational
brute force of the layer, and the plan and the combination from their definitions."""
from fractions import Fraction

import numpy as np

from oracle.formats import bf16_bits_to_f32, f32_to_bf16_bits
from oracle.int8 import (combine_ref, gelu_bounds, plan_ref, qlinear_int8_bits, qlinear_int8_ref, quant_int8, sums)
from synthetic import bf16_round, make

F32 = np.float32


def bits(v):
    return bf16_round(np.asarray(v, dtype=F32))


def round_half_even(f):
    n = f.numerator // f.denominator
    d = f - n
    return n + (d > Fraction(1, 2) or (d == Fraction(1, 2) and n % 2 == 1))


def test_row_max_and_scale():
    x = make("fp8r_tiny")["x"]
    q, s = quant_int8(x)
    v = bf16_bits_to_f32(x)
    a = np.abs(v).max(axis=1)
    assert np.array_equal(s, (a / F32(127)).astype(F32))
    assert np.all(np.abs(q.astype(int)).max(axis=1) == 127)
    assert np.all(np.abs(v - q * s[:, None].astype(np.float64)) <= s[:, None] * (0.5 + 1e-5))


def test_grid_values_round_trip():
    rng = np.random.default_rng(1)
    q = rng.integers(-127, 128, size=(5, 64))
    q[:, 7] = 127
    e = rng.integers(-60, 60, size=(5, 1))
    got, s = quant_int8(bits(q * np.ldexp(1.0, e)))
    assert np.array_equal(got, q) and np.array_equal(s, np.ldexp(1.0, e)[:, 0].astype(F32))


def test_codes_against_rationals():
    # every pair of significands, the smaller value scaled by 1, 1/2 .. 1/512
    for j in range(128, 256):
        i = np.arange(128, 256)
        x = np.concatenate([i * 2.0 ** -p for p in range(10)] + [-i * 2.0 ** -p for p in range(10)])
        x = np.concatenate([[float(j)], x[np.abs(x) <= j]])
        q, _ = quant_int8(bits(x[None]))
        # the sign is symmetric under ties to even, so rationals of one half are enough
        want = [round_half_even(Fraction(abs(float(v))) * 127 / j) * (1 if v > 0 else -1) for v in x]
        assert np.array_equal(q[0], want), j


def test_ties_exist_and_go_to_even():
    q, _ = quant_int8(bits([[254.0, 1.0, 3.0, 5.0, -1.0, -3.0], [200.0, 100.0, -100.0, 0.0, 0.0, 0.0]]))
    assert q.tolist() == [[127, 0, 2, 2, 0, -2], [127, 64, -64, 0, 0, 0]]   # 0.5, 1.5, 2.5; 63.5


def test_zero_rows_and_signed_zeros():
    q, s = quant_int8(np.array([[0, 0x8000, 0, 0x8000]], np.uint16))
    assert not q.any() and s[0] == 0.0


def test_layer_against_rationals():
    rng = np.random.default_rng(3)
    xb, wb = bits(rng.standard_normal((4, 32))), bits(rng.standard_normal((5, 32)))
    xq, xs = quant_int8(xb)
    wq, ws = quant_int8(wb)
    ref = qlinear_int8_ref(xq, xs, wq, ws)
    got = bf16_bits_to_f32(qlinear_int8_bits(xq, xs, wq, ws)).astype(np.float64)
    for m in range(4):
        for n in range(5):
            acc = sum(int(a) * int(b) for a, b in zip(xq[m], wq[n]))
            assert sums(xq, wq)[m, n] == acc
            exact = Fraction(acc) * Fraction(float(xs[m])) * Fraction(float(ws[n]))
            assert abs(Fraction(ref[m, n]) - exact) <= abs(exact) * Fraction(1, 2 ** 50)
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -20))


def test_gelu_bounds_hold_the_rounded_value():
    v = np.linspace(-8, 8, 4001)
    g = v / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))
    y = bf16_bits_to_f32(f32_to_bf16_bits(g.astype(F32)))
    lo, hi = gelu_bounds(v)
    assert np.all((y >= lo) & (y <= hi)) and np.all(hi - lo <= 0.02 * np.abs(g) + 1e-5)


def test_plan():
    ids = np.array([[2, 0], [0, 3], [-1, 2], [9, 0]])
    row_index, slot, offsets = plan_ref(ids, 4)
    assert offsets.tolist() == [0, 3, 3, 5, 6]
    assert slot.tolist() == [[3, 0], [1, 5], [-1, 4], [-1, 2]]
    assert row_index.tolist() == [0, 1, 3, 0, 2, 1, -1, -1]


def test_combination():
    y = bits([[1.0, 2.0], [4.0, -8.0], [3.0, 5.0]])
    out, tol = combine_ref(y, np.array([[0, 1], [2, -1], [-1, 3]]), np.array([[0.5, 0.25], [2.0, 9.0], [1.0, 1.0]], F32))
    assert out.tolist() == [[1.5, -1.0], [6.0, 10.0], [0.0, 0.0]]
    assert np.all(tol >= 2.0 ** -8 * np.abs(out)) and tol[2].tolist() == [0.0, 0.0]
