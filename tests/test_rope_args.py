"""Arguments of the norm and rotation of heads that no result could be right for, and the frequencies where torch's
default device is not the host."""
import ctypes

import pytest
import torch

import precision_quantized_linear_amd as qpl
from precision_quantized_linear_amd import _binding as binding

ARG = 4


@pytest.mark.parametrize("backward", [False, True])
def test_subnormal_eps(backward):
    lib = qpl.load()
    h = qpl.Heads(1 << 20, 1 << 21, 3, 640, 128, 640, 128, None, 1 << 22, 640, 128)

    def call(eps):
        args = (ctypes.byref(h), None, 5, 128, 1, eps, None)
        return lib.qk_norm_rope_backward(*args, None, 0, None) if backward else lib.qk_norm_rope(*args, None)
    for eps in (1e-38, 2.0 ** -127, 1e-40, 2.0 ** -149):
        assert call(eps) == ARG, eps
    if not torch.cuda.is_available():
        assert call(2.0 ** -126) not in (0, ARG)


def test_frequencies_under_another_default_device():
    # the library writes them on the host, wherever torch would put a new tensor
    want, scale = qpl.rope_frequencies(64, scaling="yarn", factor=4.0, trained_tokens=4096)
    with torch.device("meta"):
        got, s = qpl.rope_frequencies(64, scaling="yarn", factor=4.0, trained_tokens=4096)
    assert got.device.type == "cpu" and torch.equal(got, want) and s == scale


@pytest.mark.parametrize("sections", [(5,), (9,), (0,)])
def test_one_section_that_is_not_all_pairs(sections):
    pos, freq = torch.zeros((4, 1), dtype=torch.int32), torch.ones(8)
    assert binding._rope(pos, freq, 4, False, (8,), 1.0, -1) == binding._rope(pos[:, 0], freq, 4, False, None, 1.0, -1)
    with pytest.raises(ValueError, match="^sections:"):
        binding._rope(pos, freq, 4, False, sections, 1.0, -1)


@pytest.mark.gpu
def test_zero_heads_with_the_smallest_eps():
    x = torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda")
    for eps in (2.0 ** -126, 1e-30):
        y, _ = qpl.qk_norm_rope(x, None, None, None, eps=eps)
        dx, _, _, _ = qpl.qk_norm_rope_backward(torch.zeros_like(x), None, x, None, None, None, eps=eps)
        assert not y.any() and not dx.any()
    with pytest.raises(qpl.QPLError):
        qpl.qk_norm_rope(x, None, None, None, eps=1e-38)
