"""Long rows through the staged 8-bit integer products: hundreds of pieces of 128 bytes around each
ring, byte offsets up to a tile of rows of 2^17, and int32 sums next to -2^31 in every kernel."""
import numpy as np
import pytest
import torch

import int8_instances
import precision_quantized_linear_amd as qpl
from helpers import bf16_bits, host
from oracle.int8 import qlinear_int8_bits, quant_int8

S4, S2 = "128x128 four stages", "128x128 two stages"
DENSE = [("64x64", 65, 20000, 3001), ("64x128", 65, 20000, 8200), (S4, 515, 20000, 3600), (S2, 3001, 20000, 2570),
         ("128x256", 833, 20000, 5003), ("256x256", 4097, 20000, 2050), ("64x64", 40, 131072, 4100),
         ("64x128", 129, 131072, 6000), (S4, 515, 131072, 3600), (S2, 3001, 131072, 2570),
         ("128x256", 833, 131072, 5003), ("256x256", 4097, 131072, 2050)]
GROUPED = [("64x64", 100, 131072, 3001, 3), (S4, 1300, 131056, 1540, 3), ("128x256", 4097, 131072, 2050, 2),
           ("256x256", 6000, 131072, 2050, 2)]


def test_sizes_reach_the_staged_kernels():
    assert [(int8_instances.dense(M, K, N), M, K, N) for _, M, K, N in DENSE] == DENSE
    assert [(int8_instances.grouped(R, K, N, E), R, K, N, E) for _, R, K, N, E in GROUPED] == GROUPED
    assert {c[0] for c in DENSE} == set(int8_instances.NAMES) - {"16x16", "16x32", "32x32"}


def operands(M, K, N, E=1):
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-128, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    # codes of 127 throughout, against weights of -128 and 127: with K = 2^17 sums of -2130706432 and 2114060288
    x[[0, M // 2, M - 1]] = 1.0
    w[:, [0, N // 2, N - 1]] = -128
    w[:, [1, N // 3, N - 2]] = 127
    ws = torch.rand((E, N), generator=g, device="cuda") * 1e-5 + 1e-6
    rows = np.unique(np.r_[0:3, M // 2, np.random.default_rng(1).integers(0, M, 24), M - 2, M - 1])
    cols = np.unique(np.r_[0:20, N // 3, N // 2, np.random.default_rng(2).integers(0, N, 80), N - 20:N])
    return x, w, ws, rows, cols


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,M,K,N", DENSE)
def test_long_rows(kernel, M, K, N):
    x, w, ws, rows, cols = operands(M, K, N)
    y = qpl.qlinear_int8(x, w[0], ws[0])
    r, c = torch.from_numpy(rows).cuda(), torch.from_numpy(cols).cuda()
    xq, xs = quant_int8(bf16_bits(x[r].contiguous()))
    want = qlinear_int8_bits(xq, xs, host(w[0, c]), host(ws[0, c]))
    assert np.array_equal(bf16_bits(y[r][:, c].contiguous()), want)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,R,K,N,E", GROUPED)
def test_long_rows_by_expert(kernel, R, K, N, E):
    x, w, ws, rows, cols = operands(R, K, N, E)
    offsets = np.array([0] + [R * (e + 1) // E - (7 if e + 1 < E else 0) for e in range(E)], np.int32)
    y = qpl.qlinear_grouped_int8(x, w, ws, torch.from_numpy(offsets).cuda())
    c = torch.from_numpy(cols).cuda()
    for e in range(E):
        at = rows[(rows >= offsets[e]) & (rows < offsets[e + 1])]
        r = torch.from_numpy(at).cuda()
        xq, xs = quant_int8(bf16_bits(x[r].contiguous()))
        want = qlinear_int8_bits(xq, xs, host(w[e, c]), host(ws[e, c]))
        assert len(at) and np.array_equal(bf16_bits(y[r][:, c].contiguous()), want), e
