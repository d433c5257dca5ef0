"""Routing and the grouped 8-bit integer linear on the GPU against the CPU oracle: the plan
and the grouped outputs exactly, the combination within its fp32 bound, and the MLP
of experts bit for bit against the calls that it is made of."""
import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as qpl
from helpers import bf16_bits, host, to_dev, to_dev_bf16
from oracle.formats import bf16_bits_to_f32
from oracle.int8 import combine_ref, gelu_bounds, plan_ref, qlinear_int8_bits, qlinear_int8_ref, quant_int8
from synthetic import bf16_round

pytestmark = pytest.mark.gpu


def choices(T, topk, E, seed=0, kind="random"):
    rng = np.random.default_rng(seed)
    if kind == "random":
        return rng.integers(0, E, (T, topk)).astype(np.int32)
    if kind == "one":                                # every choice the same expert
        return np.full((T, topk), E - 1, np.int32)
    if kind == "skewed":
        return np.minimum((rng.exponential(0.15, (T, topk)) * E), E - 1).astype(np.int32)
    if kind == "none":                               # no expert at all
        return np.full((T, topk), -1, np.int32)
    ids = rng.integers(-2, E + 3, (T, topk)).astype(np.int32)   # "invalid": some outside the experts
    ids[0, 0] = np.iinfo(np.int32).min
    ids[-1, -1] = np.iinfo(np.int32).max
    return ids


PLANS = [(1, 1, 1, "random"), (1, 8, 64, "random"), (3, 1, 5, "none"), (7, 3, 4, "invalid"), (63, 2, 9, "skewed"),
         (64, 4, 16, "one"), (85, 3, 300, "random"), (257, 4, 8, "invalid"), (1024, 4, 64, "random"),
         (1025, 4, 64, "skewed"), (4097, 1, 3, "random"), (5000, 7, 33, "invalid"), (16384, 8, 256, "skewed"),
         (40, 256, 65536, "random"), (20000, 2, 2, "none"), (8192, 4, 1, "random"), (33000, 1, 1000, "invalid"),
         (20011, 5, 1024, "skewed"), (32768, 1, 64, "one"), (70001, 3, 1025, "random"), (300000, 2, 100, "invalid"),
         (600000, 1, 7, "skewed")]


@pytest.mark.parametrize("T,topk,E,kind", PLANS)
def test_plan(T, topk, E, kind):
    ids = choices(T, topk, E, seed=T, kind=kind)
    got = [host(t) for t in qpl.expert_plan(to_dev(ids), E)]
    for name, a, b in zip(("row_index", "slot", "offsets"), got, plan_ref(ids, E)):
        assert np.array_equal(a, b), name


COMBINES = [(1, 1, 1, 1), (1, 8, 8, 8), (5, 2, 10, 24), (33, 3, 50, 7), (64, 4, 256, 2048), (9, 256, 20, 40), (700, 6, 4200, 1160)]


@pytest.mark.parametrize("T,topk,R,N", COMBINES)
def test_combine(T, topk, R, N):
    rng = np.random.default_rng(T)
    y = bf16_round(rng.standard_normal((R, N)).astype(np.float32))
    slot = rng.integers(-2, R + 2, (T, topk)).astype(np.int32)
    wt = rng.standard_normal((T, topk)).astype(np.float32)
    if T > 1:
        slot[1] = -1
    out = bf16_bits_to_f32(bf16_bits(qpl.expert_combine(to_dev_bf16(y), to_dev(slot), to_dev(wt)))).astype(np.float64)
    ref, tol = combine_ref(y, slot, wt)
    assert np.all(np.abs(out - ref) <= tol)
    if T > 1:
        assert not out[1].any()


def test_combine_skips_what_it_does_not_sum():
    # rows that no slot names may hold NaN
    y = torch.full((6, 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    y[2] = 3.0
    out = qpl.expert_combine(y, to_dev(np.array([[2, -1, 6]], np.int32)), to_dev(np.array([[0.5, 1, 1]], np.float32)))
    assert bool((out == 1.5).all())


def weights(E, N, K, seed=0):
    rng = np.random.default_rng(seed + 77)
    return rng.integers(-128, 128, (E, N, K)).astype(np.int8), rng.uniform(1e-4, 2e-3, (E, N)).astype(np.float32)


def grouped_want(xq, xs, w, ws, offsets, f):
    return np.concatenate([f(xq[lo:hi], xs[lo:hi], w[e], ws[e]) for e, (lo, hi) in enumerate(zip(offsets, offsets[1:]))]
                          or [np.zeros((0, w.shape[1]))])


# rows of each expert; K; N
GROUPS = [([1], 16, 1), ([0, 0, 5], 48, 9), ([3, 0, 16, 17, 1], 80, 40), ([1] * 40, 64, 33), ([0, 200, 0], 144, 100),
          ([100, 3, 64, 65, 0, 1], 272, 130), ([300, 700, 20, 0, 513], 400, 264), ([5] * 300, 128, 16),
          ([0] * 3000 + [2] + [0] * 2000 + [1], 32, 16), ([2000, 0, 0, 0, 0, 0, 0, 1], 128, 72), ([1500, 900, 1300], 336, 513), ([256] * 16, 512, 512)]


@pytest.mark.parametrize("rows,K,N", GROUPS)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(rows, K, N, gather):
    rng = np.random.default_rng(K + N)
    E, R = len(rows), sum(rows)
    M = max(R // 3, 1) if gather else R
    x = bf16_round(rng.standard_normal((M, K)).astype(np.float32))
    w, ws = weights(E, N, K)
    offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    idx = rng.integers(0, M, R).astype(np.int32)
    idx[R // 2] = -1 if R > 4 else idx[R // 2]
    idx[R // 3] = M if R > 4 else idx[R // 3]
    xd, wd, sd, od = to_dev_bf16(x), to_dev(w), to_dev(ws), to_dev(offsets)
    ri = to_dev(idx) if gather else None
    xr = np.where(((idx >= 0) & (idx < M))[:, None], x[np.clip(idx, 0, M - 1)], 0) if gather else x
    xq, xs = quant_int8(xr.astype(np.uint16))
    y = qpl.qlinear_grouped_int8(xd, wd, sd, od, row_index=ri)
    assert np.array_equal(bf16_bits(y), grouped_want(xq, xs, w, ws, offsets, qlinear_int8_bits))
    g = bf16_bits_to_f32(bf16_bits(qpl.qlinear_grouped_int8(xd, wd, sd, od, row_index=ri, act="gelu_tanh")))
    lo, hi = gelu_bounds(grouped_want(xq, xs, w, ws, offsets, qlinear_int8_ref))
    assert np.all((g >= lo) & (g <= hi))


@pytest.mark.parametrize("rows,first,R", [([4, 0, 9], 0, 40), ([100, 150], 7, 400), ([30, 2, 1], 3, 36), ([0, 0], 0, 5)])
def test_rows_outside_the_experts_stay(rows, first, R):
    K, N = 64, 48
    x = bf16_round(np.random.default_rng(0).standard_normal((R, K)).astype(np.float32))
    w, ws = weights(len(rows), N, K)
    offsets = (first + np.concatenate([[0], np.cumsum(rows)])).astype(np.int32)
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    qpl.qlinear_grouped_int8(to_dev_bf16(x), to_dev(w), to_dev(ws), to_dev(offsets), y=y)
    xq, xs = quant_int8(x)
    want = np.full((R, N), 0x40E0, np.uint16)                                   # 7.0
    want[offsets[0]:offsets[-1]] = grouped_want(xq, xs, w, ws, offsets, qlinear_int8_bits)
    assert np.array_equal(bf16_bits(y), want)


@pytest.mark.parametrize("offsets", [[-5, 10, 500, 30], [60, 40, 20, 0], [0, 2 ** 31 - 1, -2 ** 31, 50], [0, 50, 0, 50]])
def test_bad_offsets_stay_inside_the_rows(offsets):
    # values are unspecified; nothing outside the 50 rows is written and the call ends
    K, N, R = 64, 48, 50
    x = bf16_round(np.random.default_rng(0).standard_normal((R, K)).astype(np.float32))
    w, ws = weights(3, N, K)
    whole = torch.full((R + 20, N), 7.0, dtype=torch.bfloat16, device="cuda")
    qpl.qlinear_grouped_int8(to_dev_bf16(x), to_dev(w), to_dev(ws), to_dev(np.array(offsets, np.int32)),
                             y=whole[10:10 + R])
    torch.cuda.synchronize()
    assert bool((whole[:10] == 7).all()) and bool((whole[10 + R:] == 7).all())


def test_many_lying_offsets_stay_inside_the_tile_list():
    # every other expert claims all 2^24 rows: 2^33 and more tiles, the list holds a few hundred thousand
    E, R = 65536, 1 << 24
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = R
    x = torch.ones((R, 16), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((E, 1, 16), dtype=torch.int8, device="cuda")
    y = torch.full((R + 64, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    need = qpl.qlinear_grouped_int8_workspace_bytes(R, 16, 1, E)
    work = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    qpl.qlinear_grouped_int8(x, w, torch.ones((E, 1), device="cuda"), offsets, y=y[:R], workspace=work[:need])
    torch.cuda.synchronize()
    assert bool((y[R:] == 7).all()) and bool((work[need:] == 0x5A).all())


def moe_inputs(T, topk, E, K, H, N, kind="random"):
    rng = np.random.default_rng(T + E)
    x = bf16_round(rng.standard_normal((T, K)).astype(np.float32))
    wt = rng.uniform(0, 1, (T, topk)).astype(np.float32)
    f1, f2 = (dict(weight=to_dev(a), weight_scale=to_dev(b)) for a, b in (weights(E, H, K, 1), weights(E, N, H, 2)))
    return to_dev_bf16(x), to_dev(choices(T, topk, E, seed=T, kind=kind)), to_dev(wt), f1, f2


def composed(x, ids, wt, f1, f2):
    row_index, slot, offsets = qpl.expert_plan(ids, f1["weight"].shape[0])
    h = qpl.qlinear_grouped_int8(x, f1["weight"], f1["weight_scale"], offsets, row_index=row_index, act="gelu_tanh")
    y = qpl.qlinear_grouped_int8(h, f2["weight"], f2["weight_scale"], offsets)
    return qpl.expert_combine(y, slot, wt)


MOES = [(1, 1, 1, 16, 16, 1, "random"), (1, 2, 8, 128, 64, 40, "random"), (7, 4, 16, 256, 96, 136, "random"),
        (50, 2, 4, 144, 80, 33, "invalid"), (33, 3, 6, 64, 48, 24, "none"), (300, 4, 8, 256, 176, 264, "skewed"),
        (900, 2, 3, 128, 512, 96, "one"), (128, 8, 1024, 64, 48, 16, "invalid"), (1024, 1, 7, 528, 32, 20, "skewed"),
        (17000, 2, 5, 32, 16, 8, "invalid"), (64, 16, 1000, 2064, 16, 8, "random"), (205, 5, 4, 96, 32, 24, "skewed")]


@pytest.mark.parametrize("T,topk,E,K,H,N,kind", MOES)
def test_moe_is_its_parts(T, topk, E, K, H, N, kind):
    args = moe_inputs(T, topk, E, K, H, N, kind)
    y = qpl.qlinear_moe_int8(*args)
    assert torch.equal(y, composed(*args))
    if kind == "none":
        assert not bool(y.any())


def test_slices_of_the_choices():
    """A part of a batch: choices, weights and slots that start at any element."""
    x, ids, wt, f1, f2 = moe_inputs(23, 3, 5, 64, 32, 40)
    whole = qpl.qlinear_moe_int8(x, ids, wt, f1, f2)
    part = qpl.qlinear_moe_int8(x[7:20], ids[7:20], wt[7:20], f1, f2)
    assert torch.equal(part, whole[7:20])
    row_index, slot, offsets = qpl.expert_plan(ids[7:20], 5)
    assert np.array_equal(host(slot), plan_ref(host(ids)[7:20], 5)[1])
    y = torch.randn((69, 40), device="cuda").to(torch.bfloat16)
    out = qpl.expert_combine(y, ids[7:20], wt[7:20])
    assert torch.equal(out, qpl.expert_combine(y, ids[7:20].clone(), wt[7:20].clone()))


def test_moe_against_the_oracle():
    """One token at a time in 64 bits from the GPU's own h, so that no code of h is open."""
    T, topk, E, K, H, N = 20, 3, 5, 96, 64, 56
    x, ids, wt, f1, f2 = moe_inputs(T, topk, E, K, H, N)
    row_index, slot, offsets = qpl.expert_plan(ids, E)
    h = qpl.qlinear_grouped_int8(x, f1["weight"], f1["weight_scale"], offsets, row_index=row_index, act="gelu_tanh")
    hq, hs = quant_int8(bf16_bits(h))
    i, s, w = host(ids), host(slot), host(wt).astype(np.float64)
    xq, xs = quant_int8(bf16_bits(x))
    ref, tol = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(topk):
            e, p = i[t, j], s[t, j]
            lo, hi = gelu_bounds(qlinear_int8_ref(xq[t:t + 1], xs[t:t + 1], host(f1["weight"])[e], host(f1["weight_scale"])[e]))
            hv = bf16_bits_to_f32(bf16_bits(h[p:p + 1]))
            assert np.all((hv >= lo) & (hv <= hi))
            v = qlinear_int8_ref(hq[p:p + 1], hs[p:p + 1], host(f2["weight"])[e], host(f2["weight_scale"])[e])[0]
            ref[t] += w[t, j] * v
            # each row is rounded to bf16 (half a step, 2^-8), after three fp32 roundings
            tol[t] += (2.0 ** -8 + (3 + topk) * 2.0 ** -24) * 1.01 * np.abs(w[t, j] * v)
    y = bf16_bits_to_f32(bf16_bits(qpl.qlinear_moe_int8(x, ids, wt, f1, f2))).astype(np.float64)
    assert np.all(np.abs(y - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))


def test_moe_streams_graphs_and_two_at_once():
    a, b = moe_inputs(40, 2, 6, 128, 96, 72), moe_inputs(500, 2, 6, 128, 96, 72)
    want = [composed(*a), composed(*b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(qpl.qlinear_moe_int8(*a, stream=s1), qpl.qlinear_moe_int8(*b, stream=s2)) for _ in range(4)]
    torch.cuda.synchronize()
    for ya, yb in outs:
        assert torch.equal(ya, want[0]) and torch.equal(yb, want[1])
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        y1 = qpl.qlinear_moe_int8(*a)
    with torch.cuda.graph(g2):
        y2 = qpl.qlinear_moe_int8(*b)
    ids = a[1].clone()
    for i in range(4):
        a[1].copy_(torch.roll(ids, i, 0))          # another plan in each replay
        y1.zero_()
        y2.zero_()
        g1.replay()
        g2.replay()
        eager = composed(*a)
        torch.cuda.synchronize()
        assert torch.equal(y1, eager) and torch.equal(y2, want[1]), i


def test_refusals_of_the_binding():
    x, ids, wt, f1, f2 = moe_inputs(8, 2, 4, 64, 32, 24)
    row_index, slot, offsets = qpl.expert_plan(ids, 4)
    with pytest.raises(ValueError, match="^offsets:"):
        qpl.qlinear_grouped_int8(x, f1["weight"], f1["weight_scale"], offsets[:4])
    with pytest.raises(ValueError, match="^row_index:"):
        qpl.qlinear_grouped_int8(x, f1["weight"], f1["weight_scale"], offsets, row_index=row_index.long())
    with pytest.raises(ValueError, match="^act:"):
        qpl.qlinear_grouped_int8(x, f1["weight"], f1["weight_scale"], offsets, act="relu")
    with pytest.raises(ValueError, match="^expert_ids:"):
        qpl.expert_plan(ids.long(), 4)
    with pytest.raises(ValueError, match="^expert_ids:"):
        qpl.expert_plan(ids.t(), 4)                          # not contiguous
    with pytest.raises(ValueError, match="^num_experts:"):
        qpl.expert_plan(ids, 0)
    with pytest.raises(qpl.QPLError):
        qpl.expert_plan(ids, 65537)
    with pytest.raises(ValueError, match="^weights:"):
        qpl.expert_combine(x, slot, wt.double())
    with pytest.raises(ValueError, match="^fc2.weight:"):
        qpl.qlinear_moe_int8(x, ids, wt, f1, dict(f2, weight=f2["weight"][:, :, :16].contiguous()))
