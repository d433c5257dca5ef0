"""Refusals of the 8-bit integer linears and the experts' calls, on the host: every
status is forced before a device is touched, and the binding names the wrong tensor."""
import ctypes

import pytest
import torch

import precision_quantized_linear_amd as qpl

OK, NULL, SHAPE, ALIGN, ARG, WORKSPACE, DEVICE, LAUNCH = range(8)
P = ctypes.c_void_p
A, B, C, D, E, F = (P(1 << i) for i in range(20, 26))   # aligned, never dereferenced
MIS = P((1 << 20) + 4)
ODD = P((1 << 20) + 2)    # int32 and float arrays need 4-byte alignment only
WS = 1 << 62
KMAX = 1 << 17
PLACES = (1 << 31) - (1 << 16)


@pytest.fixture(scope="module")
def lib():
    return qpl.load()


def r256(b):
    return (b + 255) // 256 * 256


def test_workspace_sizes():
    assert qpl.qlinear_workspace_bytes(qpl.QPL_INT8, 33, 48, 7) == r256(33 * 48) + r256(4 * 33)
    assert qpl.qlinear_workspace_bytes(qpl.QPL_INT8, 33, 1040, 7) == r256(33 * 1152) + r256(4 * 33)   # rows of whole lines
    assert qpl.qlinear_workspace_bytes(qpl.QPL_INT8, 4, 32, 4, 1) == 0          # no low rank
    assert qpl.qlinear_workspace_bytes(qpl.QPL_INT8, 8, KMAX, 4) > 0
    assert qpl.qlinear_workspace_bytes(qpl.QPL_INT8, 8, KMAX + 16, 4) == 0      # int32 sums
    assert qpl.qlinear_workspace_bytes(qpl.QPL_INT8, 1, 4096, 4) == 0           # a few rows: one launch, none needed
    g = qpl.qlinear_grouped_int8_workspace_bytes
    assert g(100, 48, 7, 5) >= r256(4800) + r256(400)
    assert g(100, 24, 7, 5) == g(0, 48, 7, 5) == g(100, 48, 7, 0) == g(100, 48, 7, 65537) == 0
    assert g(PLACES, 16, 1, 1) == 0 and g(PLACES - 1, 16, 1, 1) > 0
    assert g(100, KMAX + 16, 7, 5) == 0
    m = qpl.qlinear_moe_int8_workspace_bytes
    assert m(7, 2, 48, 32, 24, 5) > g(14, 48, 32, 5)
    assert m(7, 2, 48, 24, 24, 5) == 0                                          # H % 16 != 0
    assert m(7, 0, 48, 32, 24, 5) == m(7, 257, 48, 32, 24, 5) == m(0, 2, 48, 32, 24, 5) == 0


def test_linear_refusals(lib):
    assert lib.quant_act_int8(None, 4, 16, None, B, C, None) == NULL
    assert lib.quant_act_int8(A, 4, 16, None, None, C, None) == NULL
    assert lib.quant_act_int8(A, 4, 16, MIS, B, C, None) == ALIGN
    assert lib.quant_act_int8(A, 4, 24, None, B, C, None) == SHAPE
    assert lib.quant_act_int8(A, 0, 16, None, B, C, None) == SHAPE
    assert lib.qlinear_int8(A, 4, 32, 8, B, C, None, None, E, WS, None) == NULL
    assert lib.qlinear_int8(A, 4, 32, 8, B, None, None, D, E, WS, None) == NULL
    assert lib.qlinear_int8(A, 4, 32, 8, B, MIS, None, D, E, WS, None) == ALIGN
    assert lib.qlinear_int8(A, 4, 32, 8, B, C, MIS, D, E, WS, None) == ALIGN
    assert lib.qlinear_int8(A, 4, 32, 0, B, C, None, D, E, WS, None) == SHAPE
    assert lib.qlinear_int8(A, 4, KMAX + 16, 8, B, C, None, D, E, WS, None) == SHAPE
    assert lib.qlinear_int8(A, 20, 32, 8, B, C, None, D, E, 256, None) == WORKSPACE
    assert lib.qlinear_int8(A, 20, 32, 8, B, C, None, D, None, 0, None) == NULL
    assert lib.qlinear_int8(A, 4, 32, 8, B, C, None, D, MIS, 0, None) == ALIGN
    e = qpl.Epilogue()
    e.act = 7
    assert lib.qlinear_int8_ex(A, 4, 32, 8, B, C, None, ctypes.byref(e), D, E, WS, None) == ARG
    e = qpl.Epilogue()
    e.q, e.k, e.v, e.heads, e.head_dim, e.tokens, e.token_offset = 1 << 24, 1 << 25, 1 << 26, 2, 16, 8, 5
    assert lib.qlinear_int8_ex(A, 4, 32, 96, B, C, None, ctypes.byref(e), None, E, WS, None) == SHAPE  # 5 + 4 > 8


def test_plan_and_combine_refusals(lib):
    assert lib.expert_plan(None, 4, 2, 3, B, C, D, None, 0, None) == NULL
    assert lib.expert_plan(A, 4, 2, 3, B, C, None, None, 0, None) == NULL
    assert lib.expert_plan(A, 4, 2, 3, ODD, C, D, None, 0, None) == ALIGN
    assert lib.expert_plan(A, 4, 2, 3, B, C, D, MIS, 0, None) == ALIGN
    need = qpl.expert_plan_workspace_bytes(1 << 16, 2, 300)
    assert need > 0 and qpl.expert_plan_workspace_bytes(4, 2, 3) == qpl.expert_plan_workspace_bytes(0, 2, 3) == 0
    assert lib.expert_plan(A, 1 << 16, 2, 300, B, C, D, None, 0, None) == NULL
    assert lib.expert_plan(A, 1 << 16, 2, 300, B, C, D, E, need - 1, None) == WORKSPACE
    for T, k, n in ((0, 2, 3), (4, 0, 3), (4, 257, 3), (4, 2, 0), (4, 2, 65537), (PLACES // 2, 2, 3)):
        assert lib.expert_plan(A, T, k, n, B, C, D, E, WS, None) == SHAPE, (T, k, n)
    assert lib.expert_combine(A, 8, 16, B, None, 4, 2, D, None) == NULL
    assert lib.expert_combine(MIS, 8, 16, B, C, 4, 2, D, None) == ALIGN
    assert lib.expert_combine(A, 8, 16, ODD, C, 4, 2, D, None) == ALIGN
    for R, N, T, k in ((0, 16, 4, 2), (8, 0, 4, 2), (8, 16, 0, 2), (8, 16, 4, 0), (PLACES, 16, 4, 2), (8, 16, 4, 257)):
        assert lib.expert_combine(A, R, N, B, C, T, k, D, None) == SHAPE, (R, N, T, k)


def test_grouped_refusals(lib):
    def call(x=A, M=8, K=32, N=16, n=4, w=B, ws=C, idx=None, R=8, off=D, act=0, y=E, scratch=F, nb=WS):
        return lib.qlinear_grouped_int8(x, M, K, N, n, w, ws, idx, R, off, act, y, scratch, nb, None)
    for name in ("x", "w", "ws", "off", "y", "scratch"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: ODD if name == "off" else MIS}) == ALIGN, name
    assert call(idx=ODD) == ALIGN
    assert call(K=24) == call(N=0) == call(n=0) == call(n=65537) == call(R=0) == call(M=0) == SHAPE
    assert call(R=9) == SHAPE                       # without an index every row comes from x
    assert call(idx=P(1 << 26), R=9, nb=0) == WORKSPACE
    assert call(K=KMAX + 16) == SHAPE
    assert call(N=(1 << 31) - 1, K=KMAX, n=4096) == SHAPE   # 2^60 weight elements
    assert call(act=2) == ARG
    assert call(nb=qpl.qlinear_grouped_int8_workspace_bytes(8, 32, 16, 4) - 1) == WORKSPACE


def test_moe_refusals(lib):
    def call(x=A, T=4, K=32, H=16, N=8, n=4, k=2, ids=B, wt=C, w1=A, s1=B, w2=C, s2=D, y=E, scratch=F, nb=WS):
        return lib.qlinear_moe_int8(x, T, K, H, N, n, k, ids, wt, w1, s1, w2, s2, y, scratch, nb, None)
    for name in ("x", "ids", "wt", "w1", "s1", "w2", "s2", "y", "scratch"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: ODD if name in ("ids", "wt") else MIS}) == ALIGN, name
    assert call(T=0) == call(K=24) == call(H=24) == call(N=0) == call(n=0) == call(k=0) == SHAPE
    assert call(nb=qpl.qlinear_moe_int8_workspace_bytes(4, 2, 32, 16, 8, 4) - 1) == WORKSPACE


@pytest.mark.skipif(torch.cuda.is_available(), reason="forces the no-device status; a GPU is present")
def test_good_calls_reach_the_device_check(lib):
    assert lib.quant_act_int8(A, 4, 16, None, B, C, None) == DEVICE
    assert lib.qlinear_int8(A, 4, 32, 8, B, C, None, D, E, WS, None) == DEVICE
    assert lib.qlinear_int8(A, 4, 32, 8, B, C, None, D, None, 0, None) == DEVICE
    assert lib.expert_plan(A, 4, 2, 3, B, C, D, None, 0, None) == DEVICE
    assert lib.expert_combine(A, 8, 16, B, C, 4, 2, D, None) == DEVICE
    assert lib.qlinear_grouped_int8(A, 8, 32, 16, 4, B, C, None, 8, D, 1, E, F, WS, None) == DEVICE
    assert lib.qlinear_moe_int8(A, 4, 32, 16, 8, 4, 2, B, C, A, B, C, D, E, F, WS, None) == DEVICE


def test_binding_names_the_wrong_tensor():
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    w, s = torch.zeros((8, 32), dtype=torch.int8), torch.zeros(8)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="^x:"):
        qpl.quant_act_int8(x[0])
    with pytest.raises(ValueError, match="^x:"):       # on the host
        qpl.qlinear_int8(x, w, s)
    with pytest.raises(ValueError, match="^weight:"):
        qpl.qlinear_int8(x, w[0], s)
    with pytest.raises(ValueError, match="^weight:"):
        qpl.qlinear_grouped_int8(x, w, s, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="^expert_ids:"):
        qpl.expert_plan(ids, 4)
    with pytest.raises(ValueError, match="^slot:"):
        qpl.expert_combine(x, ids[0], s)
    with pytest.raises(ValueError, match="^fc2.weight:"):
        qpl.qlinear_moe_int8(x, ids, torch.zeros((4, 2)), dict(weight=w[None], weight_scale=s[None]),
                             dict(weight=w, weight_scale=s))
