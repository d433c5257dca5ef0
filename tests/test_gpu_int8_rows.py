"""Both forms of the 8-bit integer row quantizer (a wavefront or a workgroup per row) at the borders of
the rule between them, against the oracle, bit for bit."""
import numpy as np
import pytest
import torch

import int8_instances
import precision_quantized_linear_amd as qpl
from helpers import bf16_bits, host, to_dev
from oracle.int8 import qlinear_int8_bits, quant_int8
from oracle.quant import smooth_bf16
from synthetic import smooth_factors

# a workgroup per row?  rows, K
PLAIN = [(False, 3, 512), (True, 3, 528), (True, 264, 528), (False, 265, 528), (True, 1024, 2048), (False, 1025, 2048),
         (True, 2100, 8208), (False, 4200, 8208), (True, 1, 12288), (False, 6145, 12288), (True, 6145, 12304),
         (True, 9000, 16384), (True, 5, 16400), (True, 40, 70000)]
GATHERED = [(False, 5, 512), (True, 66, 528), (False, 67, 528), (True, 1026, 8208), (False, 1027, 8208),
            (True, 3000, 12304), (True, 30, 16400)]


def test_sizes_stand_at_the_borders():
    assert [(int8_instances.split(r, K, False), r, K) for _, r, K in PLAIN] == PLAIN
    assert [(int8_instances.split(r, K, True), r, K) for _, r, K in GATHERED] == GATHERED


@pytest.mark.parametrize("K", [513 * 16, 12288, 12304, 20000, 1 << 17])
def test_long_rows_are_never_read_twice_by_a_wavefront(K):
    for rows in (1, 100, 2048, 2049, 10 ** 6):
        assert K <= 12288 or (int8_instances.split(rows, K, False) and int8_instances.split(rows, K, True))


def rows_of(M, K):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn((M, K), generator=g, device="cuda")
    x *= torch.logspace(-30, 30, M, device="cuda")[:, None]
    x[M // 2] = 0
    return x.to(torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("split,M,K", PLAIN)
def test_quantizer(split, M, K):
    x = rows_of(M, K)
    pick = np.unique(np.r_[:min(M, 40), M // 2, np.random.default_rng(M).integers(0, M, 60), M - 1])
    at = torch.from_numpy(pick).cuda()
    for smooth in (False, True):
        lam = smooth_factors("svdq_w4a4", K=K) if smooth else None
        xq = torch.full((M + 2, K), 9, dtype=torch.int8, device="cuda")
        xs = torch.full((M + 4,), 9.0, device="cuda")
        qpl.quant_act_int8(x, smooth=to_dev(lam) if smooth else None, x_q=xq[1:M + 1], x_scale=xs[:M])
        bits = bf16_bits(x[at])
        wq, ws = quant_int8(smooth_bf16(bits, lam) if smooth else bits)
        assert np.array_equal(host(xq[1:M + 1][at]), wq) and np.array_equal(host(xs[:M][at]), ws)
        assert bool((xq[0] == 9).all()) and bool((xq[M + 1] == 9).all()) and bool((xs[M:] == 9).all())


@pytest.mark.gpu
@pytest.mark.parametrize("split,R,K", GATHERED)
def test_gathered(split, R, K):
    N, E, M = 40, 3, R // 4 + 2
    rng = np.random.default_rng(R)
    x = rows_of(M, K)
    idx = rng.integers(-1, M + 1, R).astype(np.int32)
    w, ws = rng.integers(-128, 128, (E, N, K), dtype=np.int8), rng.uniform(1e-4, 2e-3, (E, N)).astype(np.float32)
    offsets = np.array([0, R // 5, R // 5, R], np.int32)
    y = bf16_bits(qpl.qlinear_grouped_int8(x, to_dev(w), to_dev(ws), to_dev(offsets), row_index=to_dev(idx)))
    rows = np.where(((idx >= 0) & (idx < M))[:, None], bf16_bits(x)[np.clip(idx, 0, M - 1)], 0).astype(np.uint16)
    xq, xs = quant_int8(rows)
    for e in range(E):
        at = slice(offsets[e], offsets[e + 1])
        assert np.array_equal(y[at], qlinear_int8_bits(xq[at], xs[at], w[e], ws[e])), e
