"""Block-scaled fp8 linear, gated block, its backward and the gradient of a weight on the GPU, against the CPU oracle:
codes and scales bit for bit, products that are exact in fp32 bit for bit, the others within the bounds that the
oracle derives from their roundings."""
import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as qpl
from helpers import adversarial_rows, bf16_bits, host, to_dev, to_dev_bf16
from oracle import fp8b
from oracle.epilogue import gelu_interval, qkv_split_ref
from oracle.formats import bf16_bits_to_f32, f32_to_bf16_bits
from synthetic import bf16_round
from test_fp8b_abi import GATED, LINEAR, PAIR

pytestmark = pytest.mark.gpu


def f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def back(t):
    return f64(bf16_bits(t))


def activation(rng, M, K):
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.integers(0, K, max(K // 100, 1))] *= 10
    return bf16_round(x)


def weight(rng, N, K):
    """(codes, scales) of a weight whose blocks differ in size."""
    w = rng.standard_normal((N, K)) * fp8b.spread(np.exp(rng.standard_normal((-(-N // 128), -(-K // 128)))), N, K)
    return fp8b.quant_weight(bf16_round((w / np.sqrt(K)).astype(np.float32)))


def layer(w):
    return dict(weight=to_dev(w[0]), weight_scale=to_dev(w[1]))


def within(got, ref, bound):
    bad = np.argwhere(~(np.abs(got - ref) <= bound))
    assert bad.size == 0, (len(bad), bad[:5].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])], bound[tuple(bad[0])])


# ---- quantizers ----------------------------------------------------------------------
@pytest.mark.parametrize("K", [16, 128, 144, 1040, 2048, 2064, 12288])
def test_quantizer_adversarial(K):
    x = adversarial_rows(K, seed=K)
    q, s = qpl.quant_act_fp8b(to_dev_bf16(x))
    wq, ws = fp8b.quant_act(x)
    assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)


@pytest.mark.parametrize("M", [1, 5, 1030])
def test_quantizer_rows(M):
    x = activation(np.random.default_rng(M), M, 4112)
    q, s = qpl.quant_act_fp8b(to_dev_bf16(x))
    wq, ws = fp8b.quant_act(x)
    assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)


def test_quantizer_gives_the_codes_of_torch_on_the_gpu():
    # the rule written down in torch, its division by 448 on the GPU: many quotients lie on a border between two codes
    x = to_dev_bf16(activation(np.random.default_rng(11), 200, 2048))
    q, s = qpl.quant_act_fp8b(x)
    b = x.float().reshape(200, 16, 128)
    want_s = b.abs().amax(2, keepdim=True) / 448.0
    want = (b.double() / want_s.double()).float().to(torch.float8_e4m3fn)
    assert torch.equal(s, want_s[..., 0]) and torch.equal(q.reshape(200, 16, 128), want.view(torch.uint8))


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (130, 272), (10, 2048), (1000, 400)])
def test_weight_quantizer(N, K):
    w = adversarial_rows(K, seed=N)
    w = np.concatenate([w] * (N // len(w) + 1))[:N]
    q, s = qpl.quant_weight_fp8b(to_dev_bf16(w))
    wq, ws = fp8b.quant_weight(w)
    assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)


@pytest.mark.parametrize("N,K", [(16, 16), (128, 256), (144, 400), (1040, 272), (2064, 4112)])
def test_transpose(N, K):
    rng = np.random.default_rng(N)
    q = rng.integers(0, 256, (N, K)).astype(np.uint8)
    s = rng.random((-(-N // 128), -(-K // 128))).astype(np.float32)
    t, ts = qpl.transpose_fp8b(to_dev(q), to_dev(s))
    assert np.array_equal(host(t), q.T) and np.array_equal(host(ts), s.T)


# ---- linear ----------------------------------------------------------------------------
@pytest.mark.parametrize("M,K,N", LINEAR)
def test_linear_exact(M, K, N):
    x, w, s, y = fp8b.exact_operands(np.random.default_rng(M + K + N), M, min(K, 16384), N)
    got = qpl.qlinear_fp8b(to_dev_bf16(x), to_dev(w), to_dev(s))
    bad = np.argwhere(bf16_bits(got) != f32_to_bf16_bits(y.astype(np.float32)))
    assert bad.size == 0, (len(bad), bad[:5].tolist())


@pytest.mark.parametrize("M,K,N", [s for s in LINEAR if s[0] * s[1] * s[2] < 1 << 31])
def test_linear(M, K, N):
    rng = np.random.default_rng(M + K + N)
    x, w = activation(rng, M, K), weight(rng, N, K)
    got = back(qpl.qlinear_fp8b(to_dev_bf16(x), *map(to_dev, w)))
    y, err = fp8b.linear(fp8b.dequant_act(*fp8b.quant_act(x)), fp8b.dequant_weight(*w))
    within(got, y, fp8b.rounded(err, y))


@pytest.mark.parametrize("M", [1, 12, 40, 300, 1100])
def test_linear_gelu(M):
    rng = np.random.default_rng(M)
    K, N = 1040, 1030
    x, w = activation(rng, M, K), weight(rng, N, K)
    got = back(qpl.qlinear_fp8b(to_dev_bf16(x), *map(to_dev, w), act="gelu_tanh"))
    lo, hi = gelu_interval(*fp8b.linear(fp8b.dequant_act(*fp8b.quant_act(x)), fp8b.dequant_weight(*w)))
    assert np.all((got >= lo - fp8b.HALF_BF16 * np.abs(lo)) & (got <= hi + fp8b.HALF_BF16 * np.abs(hi)))


@pytest.mark.parametrize("M,heads,dim", [(1, 2, 16), (7, 3, 64), (65, 5, 128), (300, 8, 128), (1100, 6, 256)])
def test_linear_qkv_scatter(M, heads, dim):
    K, N, off = 272, 3 * heads * dim, 3
    x, w, s, y = fp8b.exact_operands(np.random.default_rng(M), M, K, N)
    tokens = M + off + 2
    parts = [torch.full((heads, tokens, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    qpl.qlinear_fp8b(to_dev_bf16(x), to_dev(w), to_dev(s), qkv=(*parts, off))
    bits = f32_to_bf16_bits(y.astype(np.float32))
    for i, p in enumerate(parts):
        want = bits[:, i * heads * dim:(i + 1) * heads * dim].reshape(M, heads, dim).transpose(1, 0, 2)
        got = bf16_bits(p)
        assert np.array_equal(got[:, off:off + M], want)
        rest = np.delete(got, np.s_[off:off + M], axis=1)
        assert (rest == f32_to_bf16_bits(np.array([7.0], np.float32))[0]).all()     # tokens around it untouched


def test_input_grad_is_a_linear_with_the_weight_turned_over():
    rng = np.random.default_rng(5)
    M, K, N = 70, 272, 400
    dy, w = activation(rng, M, N), weight(rng, N, K)
    t = qpl.transpose_fp8b(*map(to_dev, w))
    got = back(qpl.qlinear_fp8b(to_dev_bf16(dy), *t))
    dx, err = fp8b.linear(fp8b.dequant_act(*fp8b.quant_act(dy)), fp8b.dequant_weight(*w).T)
    within(got, dx, fp8b.rounded(err, dx))


@pytest.mark.parametrize("M", [4, 64, 600])
def test_zero_rows_and_blocks(M):
    rng = np.random.default_rng(M)
    K, N = 400, 272
    x, w, s, _ = fp8b.exact_operands(rng, M, K, N)
    x[::3] = 0
    x[1, 128:256] = 0x8000
    s[1:] = 0.0
    y = f64(x) @ fp8b.dequant_weight(w, s).T
    got = back(qpl.qlinear_fp8b(to_dev_bf16(x), to_dev(w), to_dev(s)))
    assert np.array_equal(got, f64(f32_to_bf16_bits(y.astype(np.float32))))


def test_strided_operands_are_refused_and_views_of_rows_are_not():
    x, w, s, y = fp8b.exact_operands(np.random.default_rng(0), 70, 256, 130)
    dx, dw, ds = to_dev_bf16(x), to_dev(w), to_dev(s)
    assert np.array_equal(back(qpl.qlinear_fp8b(dx[3:60], dw, ds)), f64(f32_to_bf16_bits(y[3:60].astype(np.float32))))
    with pytest.raises(ValueError, match="^x:"):
        qpl.qlinear_fp8b(dx[:, :128], dw[:, :128].contiguous(), ds[:, :1].contiguous())
    with pytest.raises(ValueError, match="^weight_scale:"):
        qpl.qlinear_fp8b(dx, dw, ds[:1].contiguous())
    with pytest.raises(ValueError, match="^y:"):
        qpl.qlinear_fp8b(dx, dw, ds, y=torch.empty((70, 131), dtype=torch.bfloat16, device="cuda"))


def test_scales_at_four_byte_alignment():
    x, w, s, y = fp8b.exact_operands(np.random.default_rng(0), 70, 256, 130)
    flat = torch.empty(1 + s.size, device="cuda")
    view = flat[1:].view(s.shape)
    view.copy_(to_dev(s))
    for m in (1, 70):
        got = qpl.qlinear_fp8b(to_dev_bf16(x)[:m], to_dev(w), view)
        assert np.array_equal(back(got), f64(f32_to_bf16_bits(y[:m].astype(np.float32))))


def test_outputs_past_2_31():
    # 2^31 outputs and more: 70000 rows of 30800 columns; the last rows compared
    M, K, N = 70000, 16, 30800
    rng = np.random.default_rng(0)
    x, w, s, _ = fp8b.exact_operands(rng, 64, K, N)
    dx = to_dev_bf16(x).repeat(M // 64 + 1, 1)[:M].contiguous()
    y = qpl.qlinear_fp8b(dx, to_dev(w), to_dev(s))
    want = f32_to_bf16_bits((f64(x) @ fp8b.dequant_weight(w, s).T).astype(np.float32))
    for m in (0, 34000, 69700, M - 1):
        assert np.array_equal(bf16_bits(y[m]), want[m % 64]), m


# ---- gated -----------------------------------------------------------------------------
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,H", GATED)
def test_gated(M, K, H, act):
    rng = np.random.default_rng(M + K + H)
    x, wg, wu = activation(rng, M, K), weight(rng, H, K), weight(rng, H, K)
    dx, gate, up = to_dev_bf16(x), layer(wg), layer(wu)
    h, g, u = qpl.qlinear_gated_fp8b(dx, gate, up, act=act, save=True)
    want = fp8b.gated(fp8b.dequant_act(*fp8b.quant_act(x)), fp8b.dequant_weight(*wg), fp8b.dequant_weight(*wu), act)
    for got, (ref, bound) in zip((h, g, u), want):
        within(back(got), ref, bound)
    # the same h without the projections, and a linear's projections bit for bit
    assert torch.equal(qpl.qlinear_gated_fp8b(dx, gate, up, act=act), h)


@pytest.mark.parametrize("M,K,H", GATED)
def test_gated_projections_exact(M, K, H):
    rng = np.random.default_rng(M)
    x, w, s, g = fp8b.exact_operands(rng, M, K, H)
    w2, s2 = np.roll(w, 1, axis=0), np.roll(s, 1, axis=0)
    u = f64(x) @ fp8b.dequant_weight(w2, s2).T
    _, gg, gu = qpl.qlinear_gated_fp8b(to_dev_bf16(x), layer((w, s)), layer((w2, s2)), save=True)
    assert np.array_equal(bf16_bits(gg), f32_to_bf16_bits(g.astype(np.float32)))
    assert np.array_equal(bf16_bits(gu), f32_to_bf16_bits(u.astype(np.float32)))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_extremes(act):
    # gates of +-2^100 and zero: act is the identity or zero, and nothing turns into NaN
    K, H = 128, 48
    x = np.zeros((6, K), np.float32)
    x[:, 0] = [2.0 ** 100, -2.0 ** 100, 1, -1, 0, 2.0 ** -100]
    w = np.zeros((H, K), np.float32)
    w[:, 0] = 1.0
    gate = layer(fp8b.quant_weight(bf16_round(w)))
    h, g, u = map(back, qpl.qlinear_gated_fp8b(to_dev_bf16(bf16_round(x)), gate, layer(fp8b.quant_weight(bf16_round(w * 2.0 ** -110))),
                                               act=act, save=True))
    assert np.isfinite(h).all() and np.array_equal(h[0], g[0] * u[0]) and (np.abs(h[1]) == 0).all() and (h[4] == 0).all()


# ---- gated backward ---------------------------------------------------------------------
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,K", PAIR)
def test_gated_backward(M, H, K, act):
    rng = np.random.default_rng(M + K + H)
    dh, g, u = (bf16_round((s * rng.standard_normal((M, H))).astype(np.float32)) for s in (1.0, 2.0, 1.0))
    wg, wu = weight(rng, H, K), weight(rng, H, K)
    gate_t, up_t = (dict(zip(("weight", "weight_scale"), qpl.transpose_fp8b(*map(to_dev, w)))) for w in (wg, wu))
    dx, dg, du = qpl.qlinear_gated_fp8b_backward(to_dev_bf16(dh), to_dev_bf16(g), to_dev_bf16(u), gate_t, up_t, act=act)
    for got, (ref, bound) in zip((dg, du), fp8b.gate_gradients(f64(dh), f64(g), f64(u), act)):
        within(back(got), ref, bound)
    # dx from the gradients that the call returned, and against the formula without their codes' rounding
    a, b = fp8b.dequant_weight(*wg), fp8b.dequant_weight(*wu)
    ref, bound = fp8b.gated_input_grad(bf16_bits(dg), bf16_bits(du), a, b)
    within(back(dx), ref, bound)
    true = back(dg) @ a + back(du) @ b
    codes = fp8b.code_error(bf16_bits(dg)) @ np.abs(a) + fp8b.code_error(bf16_bits(du)) @ np.abs(b)
    within(back(dx), true, bound + codes)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_backward_extremes(act):
    M, H, K = 8, 144, 16
    g = np.zeros((M, H), np.float32)
    g[:, :] = np.array([0, 2.0 ** 100, -2.0 ** 100, 90, -90, 12, -12, 1e-30], np.float32)[:, None]
    one = np.ones((M, H), np.float32)
    w = layer(fp8b.quant_weight(bf16_round(np.ones((K, H), np.float32))))
    dx, dg, du = map(back, qpl.qlinear_gated_fp8b_backward(*(to_dev_bf16(bf16_round(v)) for v in (one, g, one)), w, w, act=act))
    gb = f64(bf16_round(g))
    for got, (ref, bound) in zip((dg, du), fp8b.gate_gradients(one.astype(np.float64), gb, one.astype(np.float64), act)):
        within(got, ref, bound)
    assert np.isfinite(dx).all()


@pytest.mark.parametrize("M", [3, 300])
def test_gated_backward_in_place(M):
    rng = np.random.default_rng(M)
    H, K = 2064, 48
    dh, g, u = (to_dev_bf16(activation(rng, M, H)) for _ in range(3))
    w = [layer(weight(rng, K, H)) for _ in range(2)]
    want = qpl.qlinear_gated_fp8b_backward(dh, g, u, *w)
    for dg, du in (("g", "u"), ("dh", "g"), ("u", "dh")):
        t = dict(dh=dh.clone(), g=g.clone(), u=u.clone())
        got = qpl.qlinear_gated_fp8b_backward(t["dh"], t["g"], t["u"], *w, dg=t[dg], du=t[du])
        for a, b in zip(got, want):
            assert torch.equal(a, b), (dg, du)


def test_gated_backward_without_projections_gradients():
    import ctypes
    rng = np.random.default_rng(0)
    M, H, K = 40, 144, 48
    dh, g, u = (to_dev_bf16(activation(rng, M, H)) for _ in range(3))
    w = [layer(weight(rng, K, H)) for _ in range(2)]
    dx, _, _ = qpl.qlinear_gated_fp8b_backward(dh, g, u, *w)
    out = torch.empty_like(dx)
    ws = torch.empty(qpl.qlinear_gated_fp8b_backward_workspace_bytes(M, K, H), dtype=torch.uint8, device="cuda")
    c = [qpl.Fp8bWeight(v["weight"].data_ptr(), v["weight_scale"].data_ptr()) for v in w]
    assert qpl.load().qlinear_gated_fp8b_backward(dh.data_ptr(), g.data_ptr(), u.data_ptr(), M, K, H, ctypes.byref(c[0]),
                                                  ctypes.byref(c[1]), qpl.QPL_ACT_SILU, out.data_ptr(), None, None,
                                                  ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, dx)


# ---- gradient of a weight -----------------------------------------------------------------
GRAD = [(1, 16, 16), (5, 32, 48), (31, 128, 64), (32, 144, 272), (33, 256, 128), (130, 1040, 400), (64, 16, 2064),
        (515, 528, 784), (300, 4112, 4112), (1030, 5008, 4096), (4096, 64, 96), (9001, 16, 32)]


@pytest.mark.parametrize("M,N,K", GRAD)
def test_weight_grad_exact(M, N, K):
    # integers up to 8: every sum is below 2^24
    rng = np.random.default_rng(M + N)
    dy, x = (rng.integers(-8, 9, (M, w)).astype(np.float32) for w in (N, K))
    got = host(qpl.qlinear_weight_grad(to_dev_bf16(bf16_round(dy)), to_dev_bf16(bf16_round(x))))
    assert np.array_equal(got, dy.T @ x)


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (130, 1040, 400), (515, 528, 784), (4096, 64, 96)])
def test_weight_grad(M, N, K):
    rng = np.random.default_rng(M)
    dy, x = activation(rng, M, N), activation(rng, M, K)
    got = host(qpl.qlinear_weight_grad(to_dev_bf16(dy), to_dev_bf16(x))).astype(np.float64)
    within(got, *fp8b.weight_grad(dy, x))


# ---- used together ------------------------------------------------------------------------
def block(x, lay, scratch, out):
    """A feed-forward block, forward and backward, as a training step runs it."""
    gate, up, down, gate_t, up_t, down_t = lay
    h, g, u = qpl.qlinear_gated_fp8b(x, gate, up, h=out["h"], save=(out["g"], out["u"]), workspace=scratch)
    y = qpl.qlinear_fp8b(h, down["weight"], down["weight_scale"], y=out["y"], workspace=scratch)
    dh = qpl.qlinear_fp8b(y, down_t["weight"], down_t["weight_scale"], y=out["dh"], workspace=scratch)
    qpl.qlinear_gated_fp8b_backward(dh, g, u, gate_t, up_t, dx=out["dx"], dg=out["dg"], du=out["du"], workspace=scratch)
    qpl.qlinear_weight_grad(out["dg"], x, dw=out["dwg"])
    qpl.qlinear_weight_grad(out["du"], x, dw=out["dwu"])
    return out


def block_parts(seed, M, K, H):
    rng = np.random.default_rng(seed)
    lay = [layer(weight(rng, n, k)) for n, k in ((H, K), (H, K), (K, H))]
    lay += [dict(zip(("weight", "weight_scale"), qpl.transpose_fp8b(**v))) for v in lay]
    x = to_dev_bf16(activation(rng, M, K))
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")
    out = dict(h=e(M, H), g=e(M, H), u=e(M, H), y=e(M, K), dh=e(M, H), dx=e(M, K), dg=e(M, H), du=e(M, H),
               dwg=e(H, K, t=torch.float32), dwu=e(H, K, t=torch.float32))
    need = max(qpl.qlinear_workspace_bytes(qpl.QPL_FP8B, M, K, H), qpl.qlinear_workspace_bytes(qpl.QPL_FP8B, M, H, K),
               qpl.qlinear_gated_fp8b_backward_workspace_bytes(M, K, H))
    return x, lay, torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"), out


@pytest.mark.parametrize("M", [3, 40, 300])
def test_block_in_a_graph_against_eager(M):
    x, lay, ws, out = block_parts(M, M, 272, 400)
    eager = {k: v.clone() for k, v in block(x, lay, ws, out).items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block(x, lay, ws, out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, lay, ws, out)
    other = to_dev_bf16(activation(np.random.default_rng(99), M, 272))
    first = x.clone()
    for rep in range(4):
        src = first if rep % 2 == 0 else other
        x.copy_(src)
        for v in out.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        want = eager if rep % 2 == 0 else {k: v.clone() for k, v in block(x, lay, ws, out).items()}
        for k in got:
            assert torch.equal(got[k], want[k]), (rep, k)


def test_two_streams_at_once():
    parts = [block_parts(i, 200 + 60 * i, 272, 400) for i in range(2)]
    want = [{k: v.clone() for k, v in block(*p).items()} for p in parts]
    streams = [torch.cuda.Stream() for _ in parts]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(parts, streams):
            with torch.cuda.stream(s):
                block(*p)
    torch.cuda.synchronize()
    for p, w in zip(parts, want):
        for k in w:
            assert torch.equal(p[3][k], w[k]), k


def test_stream_argument():
    x, w, s, y = fp8b.exact_operands(np.random.default_rng(0), 70, 256, 130)
    st = torch.cuda.Stream()
    dx, dw, ds = to_dev_bf16(x), to_dev(w), to_dev(s)
    torch.cuda.synchronize()
    got = qpl.qlinear_fp8b(dx, dw, ds, stream=st)
    h = qpl.qlinear_gated_fp8b(dx, layer((w[:128], s[:1])), layer((w[:128], s[:1])), stream=st)
    st.synchronize()
    assert np.array_equal(bf16_bits(got), f32_to_bf16_bits(y.astype(np.float32)))
    assert torch.equal(h, qpl.qlinear_gated_fp8b(dx, layer((w[:128], s[:1])), layer((w[:128], s[:1]))))


@pytest.mark.parametrize("M,K,H", [(3, 272, 400), (300, 400, 656)])
def test_calls_repeat_bit_for_bit(M, K, H):
    x, lay, ws, out = block_parts(1, M, K, H)
    first = {k: v.clone() for k, v in block(x, lay, ws, out).items()}
    ws.zero_()
    again = block(x, lay, ws, out)
    for k in first:
        assert torch.equal(first[k], again[k]), k
