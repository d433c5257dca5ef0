"""The gradients of the norms' weights where the last group of tokens is not full, behind a kernel that left nothing but
NaNs in LDS: they are sums over the tokens that there are, whatever a workgroup finds in its LDS."""
import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as qpl
from helpers import host
from test_gpu_rope import Case, back, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def poison():
    """A transpose that turns over blocks of 0xFF bytes, four of which are a NaN in fp32, in the LDS of every CU."""
    w, s = torch.full((8192, 8192), 0xFF, dtype=torch.uint8, device="cuda"), torch.ones((64, 64), device="cuda")
    assert bool(torch.isnan(w.view(torch.float32)).all())
    t, ts = torch.empty_like(w), torch.empty_like(s)
    return lambda: qpl.transpose_fp8b(w, s, weight_t=t, weight_t_scale=ts)


@pytest.mark.parametrize("major", ["token", "head"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,kv,T,D,R", [(1, 1, 5, 16, 16), (3, 1, 9, 48, 32), (8, 2, 33, 64, 64), (6, 3, 41, 192, 192),
                                            (3, 2, 9, 512, 512), (32, 8, 33, 128, 128), (32, 8, 601, 128, 64),
                                            (32, 8, 1026, 128, 128), (32, 8, 2050, 128, 128)])
def test_sums_over_a_last_group_that_is_not_full(poison, heads, kv, T, D, R, interleaved, major):
    c = Case(heads, kv, T, D, R, interleaved=interleaved, major=major, scale=1.25)
    want = [c.want_back(n) for n in "qk"]
    torch.cuda.synchronize()
    for _ in range(2):
        poison()
        out = c.backward()
        for i in range(2):
            (dx, lim), (dw, wlim) = want[i]
            within(back(out[i]), dx, lim)
            within(host(out[2 + i]).astype(np.float64), dw, wlim)


@pytest.mark.parametrize("T", [5, 33, 601])
def test_forward_behind_it(poison, T):
    c = Case(8, 2, T, 64, 64)
    want = [c.want(n) for n in "qk"]
    poison()
    for got, w in zip(c.forward(), want):
        within(back(got), *w)
