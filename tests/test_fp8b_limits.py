"""Sizes past which a grid of the block-scaled fp8 calls would have 2^32 threads or more: refused here, or (GPU) done in
slices."""
import ctypes

import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as qpl

SHAPE = 2
A, B, C, D = (ctypes.c_void_p(1 << i) for i in range(20, 24))


@pytest.fixture(autouse=True)
def give_back():
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


def test_refused_weights():
    lib = qpl.load()
    for K in ((1 << 31) - 112, (1 << 31) - 16):
        assert lib.quant_weight_fp8b(A, 1, K, B, C, None) == SHAPE
        assert lib.transpose_fp8b(A, B, 16, K, C, D, None) == SHAPE
    if not torch.cuda.is_available():
        K = (1 << 31) - 128
        assert lib.quant_weight_fp8b(A, 1, K, B, C, None) not in (0, SHAPE)
        assert lib.transpose_fp8b(A, B, 16, K, C, D, None) not in (0, SHAPE)


@pytest.mark.gpu
def test_quantizer_of_more_rows_than_a_grid_has():
    M, K = (1 << 26) + 5, 16
    x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    x[:, 3] = torch.arange(M, device="cuda") % 251 + 2
    q, s = qpl.quant_act_fp8b(x)
    top = (torch.arange(M, device="cuda") % 251 + 2).to(torch.bfloat16).float()
    assert torch.equal(s[:, 0], top * np.float32(1 / 448)) and bool((q[:, 3] == 0x7E).all())   # 448


@pytest.mark.gpu
def test_linear_of_more_rows_than_a_grid_has():
    # every row is one value, a power of two that differs from its neighbours', and the weight picks it out
    M, K, N = (1 << 26) + 5, 16, 3
    size = torch.exp2((torch.arange(M, device="cuda") % 13).float())
    x = (size[:, None] * torch.ones(K, device="cuda")).to(torch.bfloat16)
    w, s = qpl.quant_weight_fp8b(torch.eye(N, K, device="cuda").to(torch.bfloat16))
    y = qpl.qlinear_fp8b(x, w, s)
    assert bool((y == size[:, None]).all())


@pytest.mark.gpu
def test_gated_backward_of_more_rows_than_a_grid_has():
    # gates far to the right, where act is the identity: dg = dh u, du = dh g
    M, H, K = (1 << 26) + 5, 16, 16
    size = torch.exp2((torch.arange(M, device="cuda") % 13).float()).to(torch.bfloat16)
    dh = size[:, None].expand(M, H).contiguous()
    g, u = torch.full_like(dh, 128.0), torch.full_like(dh, 4.0)
    w = dict(zip(("weight", "weight_scale"), qpl.quant_weight_fp8b(torch.eye(K, H, device="cuda").to(torch.bfloat16))))
    dx, dg, du = qpl.qlinear_gated_fp8b_backward(dh, g, u, w, w)
    assert bool((dg == size[:, None] * 4).all()) and bool((du == size[:, None] * 128).all())
    assert torch.equal(dx, (size[:, None] * 132).expand(M, K))


@pytest.mark.gpu
def test_norm_and_rotation_of_more_tokens_than_a_grid_has():
    # one head of 272 channels, in place: eight tokens a workgroup.  The norm of a constant is one, up to eps.
    T, D = (1 << 27) + 3, 272
    free, _ = torch.cuda.mem_get_info()
    if free < 80 << 30:
        pytest.skip("73 GB of heads")
    x = torch.full((1, T, D), 2.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    qpl.qk_norm_rope(x, None, pos, torch.ones(8, device="cuda"), q_out=x)
    for part in x.view(-1).split(1 << 30):
        assert bool((part == 1).all())
