"""Every kernel of the dense 8-bit integer product against the oracle, bit for bit: each entry
names the kernel that its size takes, and a host test holds the library's rule to that.  Row counts
leave whole, half and quarter last tiles, column counts leave edges and segments off 16 bytes,
and K leaves one, two, three and more pieces of 128 bytes, so that every ring wraps."""
import numpy as np
import pytest
import torch

import int8_instances
import precision_quantized_linear_amd as qpl
from helpers import bf16_bits, host, to_dev, to_dev_bf16
from oracle.formats import bf16_bits_to_f32
from oracle.int8 import gelu_bounds, qlinear_int8_bits, qlinear_int8_ref, quant_int8
from synthetic import bf16_round

S4, S2 = "128x128 four stages", "128x128 two stages"
SHAPES = [("token", 3, 400, 70),
          ("16x16", 40, 2064, 50), ("16x32", 33, 528, 1540), ("32x32", 33, 528, 3001), ("32x32", 1300, 16, 100),
          ("64x64", 33, 144, 4100), ("64x64", 515, 16, 3600), ("64x64", 1025, 16, 4100), ("64x64", 8200, 656, 9),
          ("64x128", 65, 528, 8200), ("64x128", 1300, 656, 6000), ("64x128", 4500, 16, 2050),
          (S4, 1025, 144, 3001), (S4, 515, 528, 3600), (S4, 577, 16, 5003), (S4, 129, 1040, 12000),
          (S2, 4097, 144, 2050), (S2, 4097, 528, 2050), (S2, 833, 16, 12000), (S2, 4097, 16, 4100),
          (S2, 6000, 656, 2570),
          ("128x256", 577, 400, 8200), ("128x256", 1025, 16, 6000), ("128x256", 833, 528, 5003),
          ("128x256", 4097, 528, 5003), ("128x256", 1300, 528, 12000), ("128x256", 8200, 16, 4100),
          ("256x256", 4097, 144, 3001), ("256x256", 4190, 272, 3001), ("256x256", 4300, 400, 3001),
          ("256x256", 8200, 272, 5003), ("256x256", 4500, 2064, 3600), ("256x256", 4097, 528, 8200),
          ("256x256", 4500, 528, 12000)]
EPILOGUES = [("token", 5, 256, 3, 64), ("16x16", 40, 528, 2, 64), ("16x32", 33, 528, 8, 64), ("32x32", 33, 528, 17, 64),
             ("64x64", 33, 144, 30, 64), ("64x128", 65, 528, 43, 64), (S4, 1025, 144, 17, 64), (S2, 4097, 144, 10, 64),
             ("128x256", 833, 528, 26, 64), ("256x256", 4190, 272, 18, 64), ("256x256", 4500, 400, 9, 128)]


def test_sizes_reach_every_kernel():
    assert [(int8_instances.dense(M, K, N), M, K, N) for _, M, K, N in SHAPES] == SHAPES
    assert [(int8_instances.dense(M, K, 3 * h * d), M, K, h, d) for _, M, K, h, d in EPILOGUES] == EPILOGUES
    for cases in (SHAPES, EPILOGUES):
        assert {c[0] for c in cases} == set(int8_instances.NAMES) | {int8_instances.TOKEN}


def operands(M, K, N):
    rng = np.random.default_rng(M + 3 * K + N)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.integers(0, K, max(K // 100, 1))] *= 10
    return bf16_round(x), rng.integers(-128, 128, (N, K)).astype(np.int8), rng.uniform(1e-4, 2e-3, N).astype(np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,M,K,N", SHAPES)
def test_every_kernel(kernel, M, K, N):
    x, w, ws = operands(M, K, N)
    whole = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    # behind one row, so y starts at any element: 16-byte aligned by a multiple of 8 columns only
    start = 1 if N % 8 == 0 else 0
    y = qpl.qlinear_int8(to_dev_bf16(x), to_dev(w), to_dev(ws), y=whole[start:start + M])
    got = bf16_bits(whole)
    assert np.all(got[:start] == 0x40E0) and np.all(got[start + M:] == 0x40E0) and y.shape == (M, N)
    # of the largest outputs every third row, and the first and last tile
    rows = np.arange(M) if M * N < 2 ** 24 else np.unique(np.r_[:256, np.arange(0, M, 3), M - 300:M])
    xq, xs = quant_int8(x[rows])
    bad = np.argwhere(got[start + rows] != qlinear_int8_bits(xq, xs, w, ws))
    assert bad.size == 0, (len(bad), rows[bad[:5, 0]].tolist(), bad[:5].tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,M,K,heads,head_dim", EPILOGUES)
def test_every_epilogue(kernel, M, K, heads, head_dim):
    d, off = heads * head_dim, 5
    x, w, ws = operands(M, K, 3 * d)
    xd, wd, sd = to_dev_bf16(x), to_dev(w), to_dev(ws)
    rows = np.arange(M) if M < 1100 else np.unique(np.r_[:256, np.arange(0, M, 7), M - 300:M])
    xq, xs = quant_int8(x[rows])
    want = qlinear_int8_bits(xq, xs, w, ws)
    parts = [torch.full((heads, M + off + 3, head_dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    qpl.qlinear_int8(xd, wd, sd, qkv=(*parts, off))
    for p, t in enumerate(parts):
        got = bf16_bits(t)
        assert np.all(got[:, :off] == 0x40E0) and np.all(got[:, off + M:] == 0x40E0)
        part = want[:, p * d:(p + 1) * d].reshape(len(rows), heads, head_dim).swapaxes(0, 1)
        assert np.array_equal(got[:, off + rows], part), "qkv"[p]
    g = bf16_bits_to_f32(bf16_bits(qpl.qlinear_int8(xd, wd, sd, act="gelu_tanh"))[rows]).astype(np.float64)
    lo, hi = gelu_bounds(qlinear_int8_ref(xq, xs, w, ws))
    assert np.all((g >= lo) & (g <= hi))
