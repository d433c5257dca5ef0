"""Norm and rotation of queries and keys on the GPU against the CPU oracle in float64, within the bounds that the
oracle derives from the roundings of fp32 arithmetic and of the bf16 result."""
import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as qpl
from helpers import bf16_bits, host, to_dev, to_dev_bf16
from oracle import rope
from oracle.formats import bf16_bits_to_f32
from synthetic import bf16_round

pytestmark = pytest.mark.gpu
EPS = 1e-6


def f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def back(t):
    return f64(bf16_bits(t.contiguous()))


def within(got, ref, bound):
    bad = np.argwhere(~(np.abs(got - ref) <= bound))
    assert bad.size == 0, (len(bad), bad[:5].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])], bound[tuple(bad[0])])


class Case:
    def __init__(self, heads, kv, T, D, R, interleaved=False, axes=1, scale=1.0, far=4096, major="token", weights=True,
                 norm=True, seed=0):
        rng = np.random.default_rng(seed + T + D + R)
        self.T, self.D, self.R, self.scale, self.interleaved, self.norm = T, D, R, scale, interleaved, norm
        half = R // 2
        self.sections = None if axes == 1 else tuple([half // 4] + [1] * (axes - 2) + [half - half // 4 - axes + 2])
        pos = rng.integers(0, far, (T,) if axes == 1 else (T, axes)).astype(np.int32)
        pos.flat[0] = far - 1
        self.freq = (10000.0 ** (-np.arange(half) / max(half, 1))).astype(np.float32)
        self.turn = rope.turns(pos, self.freq, self.sections, scale) if R else np.ones((T, 0))
        self.host, self.dev = {}, {}
        for n, h in (("q", heads), ("k", kv), ("dq", heads), ("dk", kv)):
            b = bf16_round(rng.standard_normal((h, T, D)).astype(np.float32) * np.exp(rng.standard_normal((h, T, 1))).astype(np.float32))
            self.host[n] = b
            self.dev[n] = to_dev_bf16(b.transpose(1, 0, 2)).transpose(0, 1) if major == "token" else to_dev_bf16(b)
        for n in ("qw", "kw"):
            b = bf16_round((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)) if weights else None
            self.host[n], self.dev[n] = b, None if b is None else to_dev_bf16(b)
        self.pos, self.dfreq = to_dev(pos), to_dev(self.freq) if R else None

    def kw(self):
        return dict(eps=EPS, norm=self.norm, interleaved=self.interleaved, sections=self.sections, scale=self.scale)

    def forward(self, **kw):
        d = self.dev
        return qpl.qk_norm_rope(d["q"], d["k"], self.pos, self.dfreq, d["qw"], d["kw"], **self.kw(), **kw)

    def backward(self, **kw):
        d = self.dev
        return qpl.qk_norm_rope_backward(d["dq"], d["dk"], d["q"], d["k"], self.pos, self.dfreq, d["qw"], d["kw"],
                                         **self.kw(), **kw)

    def want(self, n):
        w = self.host[n + "w"]
        return rope.forward(f64(self.host[n]), None if w is None else f64(w), self.turn, self.interleaved, EPS, self.norm)

    def want_back(self, n):
        w = self.host[n + "w"]
        return rope.backward(f64(self.host["d" + n]), f64(self.host[n]), None if w is None else f64(w), self.turn,
                             self.interleaved, EPS, self.norm)


# every lane count (head_dim 16 to 512), parts of the head, both layouts, one token to many, several axes
CASES = [dict(heads=1, kv=1, T=1, D=16, R=16), dict(heads=3, kv=1, T=5, D=32, R=16), dict(heads=4, kv=2, T=7, D=48, R=32),
         dict(heads=8, kv=2, T=33, D=64, R=64), dict(heads=5, kv=5, T=19, D=80, R=16), dict(heads=12, kv=4, T=70, D=96, R=64),
         dict(heads=32, kv=8, T=1, D=128, R=128), dict(heads=32, kv=8, T=300, D=128, R=128), dict(heads=20, kv=20, T=77, D=128, R=32),
         dict(heads=6, kv=3, T=41, D=192, R=192), dict(heads=4, kv=1, T=130, D=256, R=64), dict(heads=3, kv=2, T=9, D=512, R=512),
         dict(heads=2, kv=2, T=3000, D=64, R=48), dict(heads=1, kv=70, T=40, D=16, R=16), dict(heads=5, kv=1, T=9001, D=32, R=32),
         dict(heads=32, kv=8, T=1500, D=128, R=128)]


@pytest.mark.parametrize("major", ["token", "head"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, interleaved, major):
    c = Case(**case, interleaved=interleaved, major=major, scale=1.25)
    q, k = c.forward()
    assert q.stride() == c.dev["q"].stride()
    within(back(q), *c.want("q"))
    within(back(k), *c.want("k"))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes,D,R", [(2, 64, 32), (3, 128, 128), (4, 96, 96)])
def test_axes(axes, D, R, interleaved):
    c = Case(6, 2, 45, D, R, interleaved=interleaved, axes=axes)
    for got, n in zip(c.forward(), "qk"):
        within(back(got), *c.want(n))
    out = c.backward()
    for i, n in enumerate("qk"):
        (dx, lim), (dw, wlim) = c.want_back(n)
        within(back(out[i]), dx, lim)
        within(host(out[2 + i]).astype(np.float64), dw, wlim)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_far_positions(far):
    # an angle of 2^31 radians in fp32 would be off by more than a turn
    c = Case(4, 2, 64, 64, 64, far=far)
    for got, n in zip(c.forward(), "qk"):
        within(back(got), *c.want(n))


def test_negative_positions_turn_back():
    c = Case(4, 2, 16, 64, 64)
    c.pos.neg_()
    c.turn = np.conj(c.turn)
    for got, n in zip(c.forward(), "qk"):
        within(back(got), *c.want(n))


@pytest.mark.parametrize("kw", [dict(norm=False, weights=False), dict(weights=False), dict(R=0)])
def test_parts_of_the_operation(kw):
    c = Case(**{**dict(heads=5, kv=2, T=33, D=96, R=64), **kw})
    for got, n in zip(c.forward(), "qk"):
        within(back(got), *c.want(n))
    out = c.backward()
    for i, n in enumerate("qk"):
        dx, dw = c.want_back(n)
        within(back(out[i]), *dx)
        if kw.get("weights", True):
            within(host(out[2 + i]).astype(np.float64), *dw)
        else:
            assert out[2 + i] is None


def test_queries_alone_and_one_weight():
    c = Case(5, 2, 33, 64, 64)
    q, k = qpl.qk_norm_rope(c.dev["q"], None, c.pos, c.dfreq, c.dev["qw"], **c.kw())
    assert k is None and torch.equal(q, c.forward()[0])
    out = qpl.qk_norm_rope_backward(c.dev["dq"], c.dev["dk"], c.dev["q"], c.dev["k"], c.pos, c.dfreq, None, c.dev["kw"], **c.kw())
    assert out[2] is None
    within(host(out[3]).astype(np.float64), *c.want_back("k")[1])
    c.host["qw"] = None
    within(back(out[0]), *c.want_back("q")[0])


def test_position_zero_is_the_norm_alone():
    c = Case(4, 2, 9, 64, 64)
    c.pos.zero_()
    a = c.forward()
    c.dfreq = None
    for x, y in zip(a, c.forward()):
        assert torch.equal(x, y)


def test_zero_heads():
    c = Case(4, 2, 9, 64, 64)
    c.dev["q"].zero_()
    q, _ = c.forward()
    assert not q.any()
    dq, _, dw, _ = c.backward()
    assert bool(torch.isfinite(dq).all()) and not dw.any()


@pytest.mark.parametrize("major", ["token", "head"])
def test_in_place(major):
    c = Case(12, 4, 70, 96, 64, major=major)
    want, grads = c.forward(), c.backward()
    d = {n: c.dev[n].clone() for n in ("dq", "dk")}
    out = c.backward(dq_out=c.dev["dq"], dk_out=c.dev["dk"])
    assert out[0] is c.dev["dq"]
    for a, b in zip(out, grads):
        assert torch.equal(a, b)
    for n in ("dq", "dk"):
        c.dev[n].copy_(d[n])
    out = c.forward(q_out=c.dev["q"], k_out=c.dev["k"])
    assert out[0] is c.dev["q"]
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def test_rows_of_a_longer_cache():
    # queries and keys as the fused QKV projection leaves them, among tokens that are there already
    c = Case(4, 2, 37, 64, 64, major="head")
    want = c.forward()
    big = [torch.full((h, 60, 64), 7.0, dtype=torch.bfloat16, device="cuda") for h in (4, 2)]
    for b, n in zip(big, "qk"):
        b[:, 5:42] = c.dev[n]
        c.dev[n] = b[:, 5:42]
    c.forward(q_out=c.dev["q"], k_out=c.dev["k"])
    for b, w in zip(big, want):
        assert torch.equal(b[:, 5:42], w)
        assert bool((b[:, :5] == 7).all()) and bool((b[:, 42:] == 7).all())


def test_slices_of_one_projection():
    # q and k as column ranges of one [tokens, (heads + 2 kv) head_dim] projection
    c = Case(4, 2, 21, 64, 64)
    p = torch.empty((21, 8, 64), dtype=torch.bfloat16, device="cuda")
    want = c.forward()
    p[:, :4], p[:, 4:6] = c.dev["q"].transpose(0, 1), c.dev["k"].transpose(0, 1)
    c.dev["q"], c.dev["k"] = p[:, :4].transpose(0, 1), p[:, 4:6].transpose(0, 1)
    for a, b in zip(c.forward(), want):
        assert torch.equal(a, b)


def test_a_head_shared_by_stride_zero():
    c = Case(1, 1, 9, 64, 64, major="head")
    shared = c.dev["q"].expand(3, 9, 64)
    q, _ = qpl.qk_norm_rope(shared, None, c.pos, c.dfreq, c.dev["qw"], q_out=torch.empty((3, 9, 64), dtype=torch.bfloat16, device="cuda"), **c.kw())
    one = c.forward()[0]
    for h in range(3):
        assert torch.equal(q[h], one[0])
    with pytest.raises(qpl.QPLError):
        qpl.qk_norm_rope(shared, None, c.pos, c.dfreq, c.dev["qw"], q_out=shared, **c.kw())


def test_refused_views():
    c = Case(2, 1, 9, 64, 64, major="head")
    with pytest.raises(ValueError, match="^q:"):
        qpl.qk_norm_rope(c.dev["q"].transpose(1, 2).contiguous().transpose(1, 2), None, c.pos, c.dfreq, **c.kw())
    with pytest.raises(ValueError, match="^positions:"):
        qpl.qk_norm_rope(c.dev["q"], None, c.pos.long(), c.dfreq, **c.kw())
    with pytest.raises(ValueError, match="^positions:"):
        qpl.qk_norm_rope(c.dev["q"], None, c.pos[:5], c.dfreq, **c.kw())
    with pytest.raises(ValueError, match="^k:"):
        qpl.qk_norm_rope(c.dev["q"], c.dev["k"][:, :5], c.pos, c.dfreq, **c.kw())
    with pytest.raises(ValueError, match="^q_weight:"):
        qpl.qk_norm_rope(c.dev["q"], None, c.pos, c.dfreq, c.dev["qw"].float(), **c.kw())
    odd = torch.empty(9 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 9, 64)
    with pytest.raises(qpl.QPLError):
        qpl.qk_norm_rope(odd, None, c.pos, c.dfreq, **c.kw())


@pytest.mark.parametrize("major", ["token", "head"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_backward(case, interleaved, major):
    c = Case(**case, interleaved=interleaved, major=major, scale=1.25)
    out = c.backward()
    for i, n in enumerate("qk"):
        (dx, lim), (dw, wlim) = c.want_back(n)
        within(back(out[i]), dx, lim)
        within(host(out[2 + i]).astype(np.float64), dw, wlim)


def test_offsets_past_2_31():
    # heads 2^31 elements apart and more, in one allocation
    T, D, far = 3, 64, (1 << 31) + 64
    buf = torch.empty(far + T * D, dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((2, T, D), (far, D, 1))
    c = Case(2, 1, T, D, 64, major="head")
    q.copy_(c.dev["q"])
    want, _ = c.forward()
    got, _ = qpl.qk_norm_rope(q, None, c.pos, c.dfreq, c.dev["qw"], q_out=q, **c.kw())
    assert torch.equal(got, want)


def test_projection_norm_and_rotation_in_a_graph():
    """The fused QKV projection writes q, k and v behind tokens that are there; the norm and rotation follow in place."""
    from oracle import fp8b
    rng = np.random.default_rng(3)
    M, K, heads, dim, off = 50, 272, 3, 64, 4
    x, w, s, _ = fp8b.exact_operands(rng, M, K, 3 * heads * dim)
    dx, dw, ds = to_dev_bf16(x), to_dev(w), to_dev(s)
    parts = [torch.zeros((heads, M + off, dim), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    ws = torch.empty(qpl.qlinear_workspace_bytes(qpl.QPL_FP8B, M, K, 3 * heads * dim), dtype=torch.uint8, device="cuda")
    pos = torch.arange(off, off + M, dtype=torch.int32, device="cuda")
    freq, scale = qpl.rope_frequencies(dim, scaling="yarn", factor=4.0, trained_tokens=32, device="cuda")
    g = to_dev_bf16(bf16_round((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32)))

    def step():
        qpl.qlinear_fp8b(dx, dw, ds, qkv=(*parts, off), workspace=ws)
        q, k = parts[0][:, off:], parts[1][:, off:]
        qpl.qk_norm_rope(q, k, pos, freq, g, g, scale=scale, q_out=q, k_out=k)

    step()
    eager = [p.clone() for p in parts]
    y = f64(x) @ fp8b.dequant_weight(w, s).T
    y = bf16_bits_to_f32(bf16_round(y.astype(np.float32))).astype(np.float64).reshape(M, 3, heads, dim)
    turn = rope.turns(np.arange(off, off + M), host(freq), scale=scale)
    for i in range(2):
        within(back(parts[i][:, off:]), *rope.forward(y[:, i].transpose(1, 0, 2), f64(bf16_bits(g)), turn, False, EPS))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for p in parts:
            p.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, e in zip(parts, eager):
            assert torch.equal(p, e)


def test_backward_on_streams_and_in_a_graph():
    cases = [Case(8, 2, 100 + 30 * i, 64, 32, seed=i) for i in range(2)]
    want = [c.backward() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [c.backward(stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    c, graph = cases[0], torch.cuda.CUDAGraph()
    ws = torch.empty(qpl.qk_norm_rope_backward_workspace_bytes(c.T, c.D), dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        out = c.backward(workspace=ws)
    for _ in range(3):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want[0]):
            assert torch.equal(x, y)
