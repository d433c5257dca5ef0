"""Pins of the norm and rotation oracle."""
import numpy as np
import pytest

from oracle import rope


def case(interleaved, D=16, n=4, H=2, T=3, seed=0):
    rng = np.random.default_rng(seed)
    x, dy, w = rng.standard_normal((H, T, D)), rng.standard_normal((H, T, D)), rng.standard_normal(D)
    return x, dy, w, rope.turns(np.array([0, 5, 100000]), 10000.0 ** (-np.arange(n) / n), scale=1.2)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_by_its_formula(interleaved):
    x, _, _, _ = case(interleaved)
    f = np.array([1.0, 0.25, 0.5, 0.125])
    pos = np.array([3, -7, 0])
    y = rope.rotate(x, rope.turns(pos, f, scale=2.0), interleaved)
    for i in range(4):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 4)
        for t in range(3):
            c, s = 2 * np.cos(pos[t] * f[i]), 2 * np.sin(pos[t] * f[i])
            assert np.allclose(y[:, t, a], x[:, t, a] * c - x[:, t, b] * s)
            assert np.allclose(y[:, t, b], x[:, t, a] * s + x[:, t, b] * c)
    assert np.array_equal(y[..., 8:], x[..., 8:])


def test_sections_take_their_axis():
    f = np.array([1.0, 0.5, 0.25, 0.125])
    pos = np.array([[1, 2, 3], [4, 5, 6]])
    t = rope.turns(pos, f, sections=(1, 2, 1))
    want = np.stack([pos[:, 0] * f[0], pos[:, 1] * f[1], pos[:, 1] * f[2], pos[:, 2] * f[3]], 1)
    assert np.allclose(t, np.exp(1j * want))


def test_relative_positions():
    # the product of a rotated query and key depends on the distance alone
    x, y, _, _ = case(False)
    f = np.array([1.0, 0.5, 0.25, 0.125])
    dots = []
    for base in (0, 1000):
        a = rope.rotate(x, rope.turns(np.full(3, base + 9), f), False)[..., :8]
        b = rope.rotate(y, rope.turns(np.full(3, base + 2), f), False)[..., :8]
        dots.append((a * b).sum(-1))
    assert np.allclose(*dots)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_gradients_against_differences(interleaved, norm):
    x, dy, w, turn = case(interleaved)
    eps = 1e-3
    (dx, _), more = rope.backward(dy, x, w, turn, interleaved, eps, norm)

    def loss(x, w):
        return (rope.forward(x, w, turn, interleaved, eps, norm)[0] * dy).sum()

    num = np.zeros_like(x)
    for j in np.ndindex(x.shape):
        up, dn = x.copy(), x.copy()
        up[j] += 1e-6
        dn[j] -= 1e-6
        num[j] = (loss(up, w) - loss(dn, w)) / 2e-6
    assert np.abs(num - dx).max() < 1e-7
    if norm:
        dw = [(loss(x, w + 1e-6 * e) - loss(x, w - 1e-6 * e)) / 2e-6 for e in np.eye(w.size)]
        assert np.abs(np.array(dw) - more[0]).max() < 1e-7
    else:
        assert more is None


def test_unit_norm():
    x, _, _, turn = case(False)
    y, _ = rope.forward(x, None, np.ones((3, 0)), False, 1e-12)
    assert np.allclose((y * y).mean(-1), 1)
