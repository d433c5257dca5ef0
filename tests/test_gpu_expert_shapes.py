"""Every kernel of the grouped 8-bit integer product against the oracle, bit for bit: each entry
names the kernel that its size takes, and a host test holds the library's rule to that.  The experts
have uneven rows, some none and some one, so that tiles end at every row count next to another
expert's rows, whose outputs they must not touch."""
import numpy as np
import pytest
import torch

import int8_instances
import precision_quantized_linear_amd as qpl
from helpers import bf16_bits, to_dev, to_dev_bf16
from oracle.formats import bf16_bits_to_f32
from oracle.int8 import gelu_bounds, qlinear_int8_bits, qlinear_int8_ref, quant_int8
from synthetic import bf16_round

S4, S2 = "128x128 four stages", "128x128 two stages"
SHAPES = [("16x16", 17, 528, 40, 5), ("16x16", 300, 144, 33, 7), ("16x32", 40, 528, 3001, 8), ("16x32", 300, 2064, 257, 5),
          ("32x32", 130, 16, 513, 8), ("32x32", 1500, 528, 40, 64), ("64x64", 17, 16, 1027, 16),
          ("64x64", 1500, 528, 100, 33), ("64x64", 4097, 528, 40, 1), ("64x128", 40, 16, 4100, 64),
          ("64x128", 130, 528, 1540, 33), (S4, 4097, 1040, 513, 8), (S4, 700, 528, 4100, 2), (S2, 6000, 528, 513, 16),
          (S2, 4097, 16, 2050, 3), (S2, 2050, 16, 4100, 1), ("128x256", 2050, 528, 3001, 16),
          ("128x256", 4097, 16, 4100, 5), ("128x256", 8000, 144, 2050, 33), ("256x256", 8000, 1040, 4100, 5),
          ("256x256", 8000, 2064, 3001, 8), ("256x256", 8000, 1040, 3001, 1)]
ONE_OF_EACH = [("16x16", 17, 528, 40, 5), ("16x32", 300, 2064, 257, 5), ("32x32", 1500, 528, 40, 64),
               ("64x64", 1500, 528, 100, 33), ("64x128", 130, 528, 1540, 33), (S4, 4097, 1040, 513, 8),
               (S2, 6000, 528, 513, 16), ("128x256", 2050, 528, 3001, 16), ("256x256", 8000, 2064, 3001, 8)]


def test_sizes_reach_every_kernel():
    for cases in (SHAPES, ONE_OF_EACH):
        assert [(int8_instances.grouped(R, K, N, E), R, K, N, E) for _, R, K, N, E in cases] == cases
        assert {c[0] for c in cases} == set(int8_instances.NAMES)


def split(R, E, rng):
    """Rows of each expert, R together: an empty one and one with a single row among them where E allows."""
    cuts = np.sort(rng.integers(0, R + 1, E - 1))
    rows = np.diff(np.concatenate([[0], cuts, [R]]))
    if E > 3:
        rows[1] += rows[2]
        rows[2] = 0
        if rows[3] > 1:
            rows[1] += rows[3] - 1
            rows[3] = 1
    assert rows.sum() == R
    return rows


def weights(R, K, N, E, rng):
    x = bf16_round(rng.standard_normal((R, K)).astype(np.float32))
    return x, rng.integers(-128, 128, (E, N, K), dtype=np.int8), rng.uniform(1e-4, 2e-3, (E, N)).astype(np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,R,K,N,E", SHAPES)
def test_every_kernel(kernel, R, K, N, E):
    rng = np.random.default_rng(R + K + N + E)
    x, w, ws = weights(R, K, N, E, rng)
    idx = rng.integers(0, R // 3 + 1, R).astype(np.int32)
    idx[R // 2], idx[R // 3] = -1, R // 3 + 1
    xd, wd, sd, ri = to_dev_bf16(x), to_dev(w), to_dev(ws), to_dev(idx)
    M = R // 3 + 1                                            # rows of x that the gathered form has
    xg = np.where(((idx >= 0) & (idx < M))[:, None], x[np.clip(idx, 0, M - 1)], 0).astype(np.uint16)
    # the last rows, and a few in front, belong to nobody
    first, behind = min(3, R // 8), min(5, R // 8)
    offsets = first + np.concatenate([[0], np.cumsum(split(R - first - behind, E, rng))]).astype(np.int32)
    od = to_dev(offsets.astype(np.int32))
    sample = np.arange(R) if R * N < 2 ** 23 else np.unique(np.r_[np.arange(0, R, 5), (offsets[:, None] + np.arange(-3, 3)).ravel().clip(0, R - 1)])
    for rows, kw in ((x, dict(x=xd)), (xg, dict(x=xd[:M], row_index=ri))):
        xq, xs = quant_int8(rows[sample])
        y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
        qpl.qlinear_grouped_int8(weight=wd, weight_scale=sd, offsets=od, y=y, **kw)
        got = bf16_bits(y)
        assert np.all(got[:first] == 0x40E0) and np.all(got[R - behind:] == 0x40E0)
        act = qpl.qlinear_grouped_int8(weight=wd, weight_scale=sd, offsets=od, act="gelu_tanh", **kw)
        act = bf16_bits_to_f32(bf16_bits(act))
        for e in range(E):
            at = np.flatnonzero((sample >= offsets[e]) & (sample < offsets[e + 1]))
            bad = np.argwhere(got[sample[at]] != qlinear_int8_bits(xq[at], xs[at], w[e], ws[e]))
            assert bad.size == 0, (e, len(bad), sample[at][bad[:5, 0]].tolist(), bad[:5].tolist())
            lo, hi = gelu_bounds(qlinear_int8_ref(xq[at], xs[at], w[e], ws[e]))
            g = act[sample[at]].astype(np.float64)
            assert np.all((g >= lo) & (g <= hi)), e


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,R,K,N,E", ONE_OF_EACH)
def test_offsets_that_lie(kernel, R, K, N, E):
    # values are unspecified; no row outside the R and no byte outside the workspace is written, and the call ends
    rng = np.random.default_rng(R + E)
    x, w, ws = weights(R, K, N, E, rng)
    whole = torch.full((R + 40, N), 7.0, dtype=torch.bfloat16, device="cuda")
    start = 16
    need = qpl.qlinear_grouped_int8_workspace_bytes(R, K, N, E)
    work = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    xd, wd, sd = to_dev_bf16(x), to_dev(w), to_dev(ws)
    wild = rng.integers(-2 ** 31, 2 ** 31, E + 1)
    for offsets in (wild, np.where(np.arange(E + 1) % 2, R, 0), np.arange(E + 1)[::-1] * (R // E), R + np.arange(E + 1),
                    rng.integers(-9, R + 9, E + 1)):
        qpl.qlinear_grouped_int8(xd, wd, sd, to_dev(offsets.astype(np.int32)), y=whole[start:start + R], workspace=work[:need])
        torch.cuda.synchronize()
        assert bool((whole[:start] == 7).all()) and bool((whole[start + R:] == 7).all())
        assert bool((work[need:] == 0x5A).all())


# few choices (plan and first quantizer in one launch) and many, with tall tiles in both products
MLPS = [(S2, S4, 500, 2, 2, 528, 4112, 2056), ("128x256", "128x256", 1025, 2, 16, 528, 3008, 3001),
        ("256x256", S2, 4000, 2, 5, 1040, 4112, 513)]


def test_mlps_reach_tall_tiles():
    assert [(int8_instances.grouped(T * k, K, H, E), int8_instances.grouped(T * k, H, N, E), T, k, E, K, H, N)
            for _, _, T, k, E, K, H, N in MLPS] == MLPS


@pytest.mark.gpu
@pytest.mark.parametrize("first,second,T,topk,E,K,H,N", MLPS)
def test_mlp_is_its_parts(first, second, T, topk, E, K, H, N):
    from test_gpu_experts import composed, moe_inputs
    args = moe_inputs(T, topk, E, K, H, N, "invalid")
    y = qpl.qlinear_moe_int8(*args)
    assert torch.equal(y, composed(*args)) and bool(y.any())
