"""Refusals of the block-scaled fp8 calls, the gradient of a weight and the norm and rotation of heads, on the host:
every status is forced before a device is touched, and the binding names the wrong tensor."""
import ctypes
import math

import pytest
import torch

import fp8b_instances as rule
import precision_quantized_linear_amd as qpl

OK, NULL, SHAPE, ALIGN, ARG, WORKSPACE, DEVICE, LAUNCH = range(8)
P = ctypes.c_void_p
A, B, C, D, E, F, G = (P(1 << i) for i in range(20, 27))   # aligned, never dereferenced
MIS = P((1 << 20) + 4)
ODD = P((1 << 20) + 2)    # arrays of scales need 4-byte alignment only
WS = 1 << 62
KMAX = 1 << 22


@pytest.fixture(scope="module")
def lib():
    return qpl.load()


def r256(b):
    return (b + 255) // 256 * 256


def weight(w=A, s=B):
    return ctypes.byref(qpl.Fp8bWeight(w, s))


def test_workspace_sizes():
    f = qpl.qlinear_workspace_bytes
    assert f(qpl.QPL_FP8B, 33, 48, 7) == r256(33 * 128) + r256(4 * 33)
    assert f(qpl.QPL_FP8B, 33, 1040, 7) == r256(33 * 1152) + r256(4 * 33 * 9)    # rows of whole lines
    assert f(qpl.QPL_FP8B, 4, 32, 4, 1) == 0                                     # no low rank
    assert f(qpl.QPL_FP8B, 1, 4096, 4) == 0                                      # a few rows: one launch, none needed
    assert f(qpl.QPL_FP8B, 40, KMAX - 16, 4) > 0 and f(qpl.QPL_FP8B, 40, KMAX, 4) == 0
    g = qpl.qlinear_gated_fp8b_workspace_bytes
    assert g(33, 1040, 48) == f(qpl.QPL_FP8B, 33, 1040, 48) and g(1, 64, 32) == 0 and g(33, 1040, 40) == 0
    b = qpl.qlinear_gated_fp8b_backward_workspace_bytes
    assert b(33, 48, 272) == r256(33 * 2 * 384) + r256(8 * 33 * 3)
    assert b(33, 48, 40) == b(33, 40, 48) == b(0, 48, 48) == 0
    assert b(1, 16, (1 << 21) - 128) > 0 and b(1, 16, (1 << 21) - 112) == 0
    q = qpl.qk_norm_rope_backward_workspace_bytes
    assert q(5, 128) == 5 * 8 * 128 and q(10 ** 6, 64) == 2048 * 8 * 64
    assert q(0, 64) == q(5, 24) == q(5, 528) == 0


def test_quantizer_refusals(lib):
    for fn in (lib.quant_act_fp8b, lib.quant_weight_fp8b):
        assert fn(None, 4, 16, B, C, None) == fn(A, 4, 16, None, C, None) == fn(A, 4, 16, B, None, None) == NULL
        assert fn(MIS, 4, 16, B, C, None) == fn(A, 4, 16, MIS, C, None) == fn(A, 4, 16, B, ODD, None) == ALIGN
        assert fn(A, 0, 16, B, C, None) == fn(A, 4, 24, B, C, None) == fn(A, 4, 0, B, C, None) == SHAPE
    t = lib.transpose_fp8b
    assert t(None, B, 16, 16, C, D, None) == t(A, B, 16, 16, C, None, None) == NULL
    assert t(MIS, B, 16, 16, C, D, None) == t(A, ODD, 16, 16, C, D, None) == ALIGN
    assert t(A, B, 24, 16, C, D, None) == t(A, B, 16, 24, C, D, None) == SHAPE


def test_linear_refusals(lib):
    def call(x=A, M=40, K=32, N=8, w=B, s=C, y=D, ws=E, nb=WS):
        return lib.qlinear_fp8b(x, M, K, N, w, s, y, ws, nb, None)
    for name in ("x", "w", "s", "y", "ws"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: ODD if name == "s" else MIS}) == ALIGN, name
    assert call(M=0) == call(K=24) == call(N=0) == call(K=KMAX) == call(M=1 << 31) == SHAPE
    assert call(nb=qpl.qlinear_workspace_bytes(qpl.QPL_FP8B, 40, 32, 8) - 1) == WORKSPACE
    e = qpl.Epilogue()
    for act in (qpl.QPL_ACT_SILU, 7):     # SiLU belongs to the gated block
        e.act = act
        assert lib.qlinear_fp8b_ex(A, 4, 32, 8, B, C, ctypes.byref(e), D, E, WS, None) == ARG
    e = qpl.Epilogue()
    e.q, e.k, e.v, e.heads, e.head_dim, e.tokens, e.token_offset = 1 << 24, 1 << 25, 1 << 26, 2, 16, 8, 5
    assert lib.qlinear_fp8b_ex(A, 4, 32, 96, B, C, ctypes.byref(e), None, E, WS, None) == SHAPE   # 5 + 4 > 8


def test_gated_refusals(lib):
    def call(x=A, M=40, K=32, H=48, g=weight(), u=weight(), act=qpl.QPL_ACT_SILU, h=C, sg=None, su=None, ws=E, nb=WS):
        return lib.qlinear_gated_fp8b(x, M, K, H, g, u, act, h, sg, su, ws, nb, None)
    for name in ("x", "h", "ws", "g", "u"):
        assert call(**{name: None}) == NULL, name
    assert call(sg=D) == call(su=D) == call(g=weight(None)) == call(u=weight(A, None)) == NULL
    for name in ("x", "h", "ws"):
        assert call(**{name: MIS}) == ALIGN, name
    assert call(g=weight(MIS)) == call(u=weight(A, ODD)) == call(sg=MIS, su=D) == ALIGN
    assert call(H=40) == call(K=24) == call(M=0) == call(K=KMAX) == SHAPE
    assert call(act=qpl.QPL_ACT_NONE) == call(act=9) == ARG
    assert call(nb=qpl.qlinear_gated_fp8b_workspace_bytes(40, 32, 48) - 1) == WORKSPACE


def test_gated_backward_refusals(lib):
    def call(dh=A, sg=B, su=C, M=4, K=32, H=48, g=weight(), u=weight(), act=qpl.QPL_ACT_SILU, dx=D, dg=E, du=F, ws=G, nb=WS):
        return lib.qlinear_gated_fp8b_backward(dh, sg, su, M, K, H, g, u, act, dx, dg, du, ws, nb, None)
    for name in ("dh", "sg", "su", "dx", "dg", "du", "ws", "g", "u"):
        assert call(**{name: None}) == NULL, name
    for name in ("dh", "sg", "su", "dx", "dg", "du", "ws"):
        assert call(**{name: MIS}) == ALIGN, name
    assert call(H=40) == call(K=24) == call(M=0) == call(H=1 << 21) == SHAPE
    assert call(act=qpl.QPL_ACT_NONE) == ARG
    assert call(nb=qpl.qlinear_gated_fp8b_backward_workspace_bytes(4, 32, 48) - 1) == WORKSPACE


def test_weight_grad_refusals(lib):
    def call(dy=A, x=B, M=4, N=48, K=32, dw=C):
        return lib.qlinear_weight_grad(dy, x, M, N, K, dw, None)
    for name in ("dy", "x", "dw"):
        assert call(**{name: None}) == NULL and call(**{name: MIS}) == ALIGN, name
    assert call(M=0) == call(N=40) == call(K=40) == call(N=0) == call(K=(1 << 23) + 16) == call(N=(1 << 23) + 16) == SHAPE


def heads(**kw):
    h = qpl.Heads(1 << 20, 1 << 21, 3, 640, 128, 640, 128)
    h.dx, h.dx_head_stride, h.dx_token_stride = 1 << 22, 640, 128
    for k, v in kw.items():
        setattr(h, k, v)
    return h


def rope(**kw):
    r = qpl.Rope(1 << 23, 1 << 24, 64, 1, (ctypes.c_int64 * 4)(32), 0, 1.0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


REF = ctypes.byref
BAD_HEADS = [(dict(x=None), NULL), (dict(x=(1 << 20) + 8), ALIGN), (dict(heads=0), SHAPE), (dict(heads=65537), SHAPE),
             (dict(x_head_stride=-8), SHAPE), (dict(x_token_stride=132), SHAPE), (dict(x_head_stride=1 << 40), SHAPE),
             (dict(x_token_stride=1 << 39), SHAPE), (dict(weight=(1 << 20) + 8), ALIGN)]
# written views in which two elements meet
MEETING = [(0, 128), (640, 0), (640, 120), (632, 128), (128, 256)]


def test_norm_rope_refusals(lib):
    def call(q=heads(), k=heads(), T=5, dim=128, norm=1, eps=1e-6, r=rope()):
        return lib.qk_norm_rope(None if q is None else REF(q), None if k is None else REF(k), T, dim, norm, eps,
                                None if r is None else REF(r), None)
    assert call(q=None) == NULL
    for kw, want in BAD_HEADS:
        assert call(q=heads(**kw)) == want and call(k=heads(**kw)) == want, kw
    assert call(q=heads(y=None)) == NULL and call(q=heads(y=(1 << 20) + 8)) == ALIGN
    for hs, ts in MEETING:
        assert call(q=heads(y_head_stride=hs, y_token_stride=ts)) == SHAPE, (hs, ts)
    assert call(T=0) == call(T=1 << 31) == call(dim=0) == call(dim=136) == call(dim=528) == SHAPE
    for eps in (0.0, -1.0, math.inf, math.nan):
        assert call(eps=eps) == ARG, eps
    assert call(norm=0, r=None) == ARG                              # nothing to do
    assert call(norm=0, r=rope(rotary_dim=0)) == ARG
    assert call(norm=0, q=heads(weight=1 << 20)) == ARG
    for kw, want in ((dict(positions=None), NULL), (dict(inv_freq=None), NULL), (dict(positions=(1 << 20) + 2), ALIGN),
                     (dict(inv_freq=(1 << 20) + 2), ALIGN), (dict(rotary_dim=144), SHAPE), (dict(rotary_dim=24), SHAPE),
                     (dict(rotary_dim=-16), SHAPE), (dict(axes=0), SHAPE), (dict(axes=5), SHAPE), (dict(scale=0.0), ARG),
                     (dict(scale=math.nan), ARG), (dict(scale=-1.0), ARG),
                     (dict(axes=2, sections=(ctypes.c_int64 * 4)(16, 15)), SHAPE),
                     (dict(axes=2, sections=(ctypes.c_int64 * 4)(-1, 33)), SHAPE),
                     (dict(axes=3, sections=(ctypes.c_int64 * 4)(16, 16, 1)), SHAPE)):
        assert call(r=rope(**kw)) == want, kw


def test_norm_rope_backward_refusals(lib):
    def call(q=heads(), k=heads(), T=5, dim=128, norm=1, eps=1e-6, r=rope(), ws=G, nb=WS):
        return lib.qk_norm_rope_backward(None if q is None else REF(q), None if k is None else REF(k), T, dim, norm, eps,
                                         None if r is None else REF(r), ws, nb, None)
    assert call(q=None) == NULL
    for kw, want in BAD_HEADS:
        assert call(q=heads(**kw)) == want and call(k=heads(**kw)) == want, kw
    assert call(q=heads(dx=None)) == NULL and call(k=heads(dx=(1 << 20) + 8)) == ALIGN
    for hs, ts in MEETING:
        assert call(k=heads(dx_head_stride=hs, dx_token_stride=ts)) == SHAPE, (hs, ts)
    w = dict(weight=1 << 20, dweight=1 << 25)
    assert call(q=heads(dweight=1 << 25)) == ARG
    assert call(q=heads(**w), ws=None) == NULL and call(q=heads(**w), ws=MIS) == ALIGN
    assert call(k=heads(weight=1 << 20, dweight=(1 << 25) + 2)) == ALIGN
    assert call(q=heads(**w), nb=5 * 8 * 128 - 1) == WORKSPACE
    assert call(eps=0.0) == call(norm=0, r=None) == ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="forces the no-device status; a GPU is present")
def test_good_calls_reach_the_device_check(lib):
    assert lib.quant_act_fp8b(A, 4, 16, B, C, None) == DEVICE
    assert lib.quant_weight_fp8b(A, 5, 16, B, MIS, None) == DEVICE
    assert lib.transpose_fp8b(A, B, 16, 32, C, D, None) == DEVICE
    assert lib.qlinear_fp8b(A, 1, 32, 7, B, MIS, D, None, 0, None) == DEVICE
    assert lib.qlinear_fp8b(A, 100, 32, 7, B, C, D, E, WS, None) == DEVICE
    assert lib.qlinear_gated_fp8b(A, 4, 32, 16, weight(), weight(), 2, C, None, None, None, 0, None) == DEVICE
    assert lib.qlinear_gated_fp8b(A, 40, 32, 16, weight(), weight(), 1, C, D, E, F, WS, None) == DEVICE
    assert lib.qlinear_gated_fp8b_backward(A, B, C, 1, 32, 16, weight(), weight(), 2, D, None, None, G, WS, None) == DEVICE
    assert lib.qlinear_weight_grad(A, B, 1, 16, 32, C, None) == DEVICE
    h, b = heads(weight=1 << 20), heads(weight=1 << 20, dweight=1 << 25)
    assert lib.qk_norm_rope(REF(h), None, 5, 128, 1, 1e-6, REF(rope()), None) == DEVICE
    assert lib.qk_norm_rope(REF(heads()), REF(heads(heads=1)), 5, 128, 0, 0.0, REF(rope()), None) == DEVICE
    assert lib.qk_norm_rope(REF(h), None, 5, 128, 1, 1e-6, None, None) == DEVICE
    t = heads(x_head_stride=128, x_token_stride=384, y_head_stride=128, y_token_stride=384)    # token-major
    assert lib.qk_norm_rope(REF(t), None, 5, 128, 1, 1e-6, REF(rope()), None) == DEVICE
    assert lib.qk_norm_rope(REF(heads(x_head_stride=0)), None, 5, 128, 1, 1e-6, REF(rope()), None) == DEVICE
    assert lib.qk_norm_rope_backward(REF(b), None, 5, 128, 1, 1e-6, REF(rope()), G, WS, None) == DEVICE
    assert lib.qk_norm_rope_backward(REF(heads()), None, 5, 128, 0, 0.0, REF(rope()), None, 0, None) == DEVICE


def test_frequencies():
    f, s = qpl.rope_frequencies(64, 10000.0)
    want = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    assert s == 1.0 and torch.equal(f, want.float())
    f, s = qpl.rope_frequencies(64, scaling="linear", factor=4.0)
    assert s == 1.0 and torch.equal(f, (want / 4).float())
    f, _ = qpl.rope_frequencies(64, scaling="ntk", factor=4.0)
    # the slowest channel turns 4 times slower, the fastest as before
    assert f[0] == 1.0 and abs(float(f[-1]) / float(want[-1]) - 0.25) < 1e-6
    f, s = qpl.rope_frequencies(64, scaling="yarn", factor=4.0, trained_tokens=4096)
    turns = 4096 * want / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    assert torch.allclose(f.double(), want * (keep + (1 - keep) / 4), rtol=2.0 ** -23)
    assert bool((keep == 0).any()) and bool((keep == 1).any()) and abs(s - (0.1 * math.log(4.0) + 1)) < 1e-7
    # the ends of the ramp are the caller's
    f, _ = qpl.rope_frequencies(64, scaling="yarn", factor=4.0, trained_tokens=4096, low_turns=1e5, high_turns=2e5)
    assert torch.equal(f, (want / 4).float())


def test_frequencies_refusals():
    for kw in (dict(rotary_dim=0), dict(rotary_dim=24), dict(rotary_dim=528), dict(base=1.0), dict(base=math.nan),
               dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=math.inf),
               dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, trained_tokens=10, low_turns=32.0)):
        with pytest.raises(qpl.QPLError):
            qpl.rope_frequencies(**{"rotary_dim": 64, **kw})
    with pytest.raises(ValueError, match="^scaling:"):
        qpl.rope_frequencies(64, scaling="other")


def test_binding_names_the_wrong_tensor():
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    w, s = torch.zeros((16, 32), dtype=torch.uint8), torch.zeros((1, 1))
    layer = dict(weight=w, weight_scale=s)
    q = torch.zeros((2, 4, 32), dtype=torch.bfloat16)
    pos, f = torch.zeros(4, dtype=torch.int32), torch.ones(16)
    with pytest.raises(ValueError, match="^x:"):       # on the host
        qpl.quant_act_fp8b(x)
    with pytest.raises(ValueError, match="^w:"):
        qpl.quant_weight_fp8b(x[0])
    with pytest.raises(ValueError, match="^weight:"):
        qpl.transpose_fp8b(w, s)
    with pytest.raises(ValueError, match="^weight:"):
        qpl.qlinear_fp8b(x, w[0], s)
    with pytest.raises(ValueError, match="^x:"):
        qpl.qlinear_fp8b(x, w, s)
    with pytest.raises(ValueError, match="^gate.weight:"):
        qpl.qlinear_gated_fp8b(x, dict(weight=w[0], weight_scale=s), layer)
    with pytest.raises(ValueError, match="^x:"):
        qpl.qlinear_gated_fp8b(x, layer, layer)
    with pytest.raises(ValueError, match="^dh:"):
        qpl.qlinear_gated_fp8b_backward(x, x, x, layer, layer)
    with pytest.raises(ValueError, match="^dy:"):
        qpl.qlinear_weight_grad(x[0], x)
    with pytest.raises(ValueError, match="^q:"):
        qpl.qk_norm_rope(q, None, pos, f)
    with pytest.raises(ValueError, match="^q:"):
        qpl.qk_norm_rope_backward(q, None, q[0], None, pos, f)


# sizes that the GPU tests multiply, and the kernels that the rule takes for them
LINEAR = [(1, 16, 1), (1, 4096, 257), (2, 48, 16), (16, 1024, 33), (16, 1040, 40), (3, 2000, 20000), (15, 80, 33),
          (17, 144, 63), (20, 2064, 100), (31, 400, 65), (33, 64, 8), (64, 400, 65), (65, 272, 1000), (127, 1040, 129),
          (129, 128, 256), (255, 512, 300), (300, 192, 513), (513, 336, 264), (515, 1040, 2001), (1025, 1200, 1032),
          (2100, 256, 2050), (2049, 528, 4103), (4500, 96, 5000), (2300, 400, 6000), (260, 20000, 40), (40, 8192, 24), (1500, 640, 6000), (1030, 272, 6000), (2050, 144, 6000), (300, 400, 1500),
          (64, 1040, 4112)]
GATED = [(1, 64, 16), (4, 2048, 272), (16, 1024, 64), (17, 144, 48), (33, 272, 400), (40, 4096, 16), (100, 512, 96),
         (130, 1040, 1008), (257, 384, 656), (700, 256, 1392), (1030, 400, 2064), (515, 272, 6000), (2050, 272, 3088)]
PAIR = [(1, 64, 16), (5, 400, 48), (17, 144, 272), (64, 1008, 528), (130, 2736, 1040), (300, 272, 2064),
        (257, 400, 4112), (1030, 656, 2064), (2050, 144, 4112), (2300, 272, 6000), (33, 4096, 272), (130, 144, 6000), (700, 1008, 6000)]


def test_sizes_reach_every_kernel():
    assert {rule.linear(*s) for s in LINEAR} == rule.every() | {-1}
    assert {rule.gated(*s) for s in GATED} == rule.every(gated=True) | {-1}
    assert {rule.pair(*s) for s in PAIR} == rule.every()
