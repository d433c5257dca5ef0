"""8-bit integer linear on the GPU against the CPU oracle: codes and scales bit for bit,
and outputs bit for bit too, because the int32 sums are exact and the roundings after
them (to fp32, two fp32 products, bf16) leave one value for each element.  GELU outputs
lie in the interval that those roundings and an fp32 GELU allow."""
import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as qpl
from helpers import adversarial_rows, bf16_bits, host, to_dev, to_dev_bf16
from oracle.formats import bf16_bits_to_f32
from oracle.int8 import gelu_bounds, qlinear_int8_bits, qlinear_int8_ref, quant_int8
from oracle.quant import smooth_bf16
from synthetic import bf16_round, smooth_factors

pytestmark = pytest.mark.gpu


def operands(M, K, N, seed=0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.integers(0, K, max(K // 100, 1))] *= 10
    w = rng.integers(-128, 128, (N, K)).astype(np.int8)
    return bf16_round(x), w, rng.uniform(1e-4, 2e-3, N).astype(np.float32)


def linear(x, w, ws, **kw):
    return qpl.qlinear_int8(to_dev_bf16(x), to_dev(w), to_dev(ws), **kw)


# ---- quantizer -----------------------------------------------------------------------
@pytest.mark.parametrize("K", [16, 48, 512, 520 * 2, 4096, 12288, 16384])
def test_quantizer_adversarial(K):
    x = adversarial_rows(K, seed=K)
    q, s = qpl.quant_act_int8(to_dev_bf16(x))
    wq, ws = quant_int8(x)
    assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)


def test_quantizer_every_significand_pair():
    # rows of maximum j 2^e hold every significand at nine exponents, both signs; ties included
    i = np.arange(128, 256, dtype=np.float64)
    small = np.concatenate([i * 2.0 ** -p for p in range(1, 10)])
    for e in (-120, 0, 100):
        rows = [np.concatenate([np.minimum(i, j), small, -np.minimum(i, j), -small]) * 2.0 ** e
                for j in range(128, 256)]
        x = bf16_round(np.stack(rows).astype(np.float32))
        q, s = qpl.quant_act_int8(to_dev_bf16(x))
        wq, ws = quant_int8(x)
        assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws), e


@pytest.mark.parametrize("M,K", [(1, 64), (5, 4096), (9, 15232)])
def test_quantizer_smoothed(M, K):
    x, _, _ = operands(M, K, 1)
    lam = smooth_factors("svdq_w4a4", K=K)
    q, s = qpl.quant_act_int8(to_dev_bf16(x), smooth=to_dev(lam))
    wq, ws = quant_int8(smooth_bf16(x, lam))
    assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)


def test_quantizer_ignores_rows_around_a_view():
    x, _, _ = operands(9, 128, 1)
    q, s = qpl.quant_act_int8(to_dev_bf16(x)[2:7])
    wq, ws = quant_int8(x[2:7])
    assert np.array_equal(host(q), wq) and np.array_equal(host(s), ws)


# ---- linear ---------------------------------------------------------------------------
SHAPES = [(1, 16, 1), (1, 4096, 257), (2, 48, 16), (15, 80, 33), (16, 128, 64), (17, 144, 63), (31, 2064, 100),
          (33, 64, 8), (64, 400, 65), (65, 272, 1000), (127, 1040, 129), (129, 128, 256), (255, 512, 300),
          (1, 32768, 100), (2, 16384, 530), (4, 8192, 48), (4, 8208, 33), (3, 2000, 20000), (1, 32784, 9),
          (5, 64, 70), (16, 2048, 300),
          (16, 2064, 50), (8, 4096, 70), (9, 3600, 40), (13, 1008, 8200), (11, 2560, 77),
          (1, 16384, 90), (1, 16400, 90), (16, 1024, 4100), (16, 1040, 64), (4, 4096, 20000), (5, 3120, 40), (7, 2048, 30),
          (300, 192, 513), (513, 336, 264), (1025, 1200, 1032), (2100, 256, 2050), (4500, 96, 5000), (3, 131072, 20),
          (260, 20000, 40), (150, 131072, 130), (2, 4096, 100003)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear(M, K, N):
    x, w, ws = operands(M, K, N, seed=M + K + N)
    y = linear(x, w, ws)
    xq, xs = quant_int8(x)
    want = qlinear_int8_bits(xq, xs, w, ws)
    bad = np.argwhere(bf16_bits(y) != want)
    assert bad.size == 0, (len(bad), bad[:5].tolist())


def test_largest_sums_stay_exact():
    # K = 2^17, every product 127 * -128: the sum is -2130706432, close to -2^31
    x = np.full((2, 131072), 0x3F80, np.uint16)
    w = np.full((3, 131072), -128, np.int8)
    ws = np.array([1.0, 0.5, 1e-6], np.float32)
    y = linear(x, w, ws)
    xq, xs = quant_int8(x)
    assert np.array_equal(bf16_bits(y), qlinear_int8_bits(xq, xs, w, ws))


@pytest.mark.parametrize("M", [1, 4, 16, 40, 300, 1100])
def test_linear_smoothed_and_gelu(M):
    K, N = 512, 1030
    x, w, ws = operands(M, K, N, seed=M)
    lam = smooth_factors("svdq_w4a4", K=K)
    y = bf16_bits_to_f32(bf16_bits(linear(x, w, ws, smooth=to_dev(lam), act="gelu_tanh"))).astype(np.float64)
    xq, xs = quant_int8(smooth_bf16(x, lam))
    lo, hi = gelu_bounds(qlinear_int8_ref(xq, xs, w, ws))
    assert np.all((y >= lo) & (y <= hi))


@pytest.mark.parametrize("M,heads,head_dim,offset", [(1, 2, 8, 0), (37, 3, 64, 5), (300, 4, 128, 12), (1030, 8, 128, 1)])
def test_qkv(M, heads, head_dim, offset):
    d, K, tokens = heads * head_dim, 160, M + offset + 3
    x, w, ws = operands(M, K, 3 * d, seed=M)
    q, k, v = (torch.full((heads, tokens, head_dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    out = linear(x, w, ws, qkv=(q, k, v, offset))
    y = linear(x, w, ws)
    assert out[0] is q and out[1] is k and out[2] is v
    for p, t in enumerate((q, k, v)):
        part = y[:, p * d:(p + 1) * d].reshape(M, heads, head_dim).transpose(0, 1)
        assert torch.equal(t[:, offset:offset + M], part)
        assert bool((t[:, :offset] == 7).all()) and bool((t[:, offset + M:] == 7).all())


def test_zero_rows_give_zeros():
    x, w, ws = operands(70, 256, 90)
    x[::3] = 0x8000
    y = bf16_bits_to_f32(bf16_bits(linear(x, w, ws)))
    assert not y[::3].any() and y[1::3].any()


@pytest.mark.parametrize("M,N,K", [(16, 134217750, 16), (33, 67108869, 16), (40000, 65536, 64)])
def test_outputs_past_2_31_elements(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand((N,), generator=g, device="cuda") * 1e-3 + 1e-4
    y = qpl.qlinear_int8(x, w, ws)
    rows = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    cols = torch.cat([torch.arange(0, 40), torch.randint(0, N, (400,)), torch.arange(N - 40, N)]).cuda()
    got = bf16_bits(y[rows][:, cols].contiguous())
    xq, xs = quant_int8(bf16_bits(x[rows].contiguous()))
    assert np.array_equal(got, qlinear_int8_bits(xq, xs, host(w[cols]), host(ws[cols])))


def test_outputs_and_workspace_of_the_caller():
    x, w, ws = operands(50, 176, 72)
    xd, wd, sd = to_dev_bf16(x), to_dev(w), to_dev(ws)
    y = torch.empty((50, 72), dtype=torch.bfloat16, device="cuda")
    need = qpl.qlinear_workspace_bytes(qpl.QPL_INT8, 50, 176, 72)
    work = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    assert qpl.qlinear_int8(xd, wd, sd, y=y, workspace=work) is y
    xq, xs = quant_int8(x)
    assert np.array_equal(bf16_bits(y), qlinear_int8_bits(xq, xs, w, ws))
    assert np.all(host(work)[need:] == 0x5A)
    with pytest.raises(qpl.QPLError):
        qpl.qlinear_int8(xd, wd, sd, workspace=work[:need - 1])
    with pytest.raises(ValueError, match="^y:"):
        qpl.qlinear_int8(xd, wd, sd, y=y.float())
    with pytest.raises(ValueError, match="^workspace:"):
        qpl.qlinear_int8(xd, wd, sd, workspace=work.cpu())


@pytest.mark.parametrize("M", [3, 600])
def test_streams_and_graphs(M):
    x, w, ws = operands(M, 640, 770)
    x2 = operands(M, 640, 770, seed=9)[0]
    xd, wd, sd = to_dev_bf16(x), to_dev(w), to_dev(ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ys = [qpl.qlinear_int8(xd, wd, sd, stream=side) for _ in range(3)] + [qpl.qlinear_int8(xd, wd, sd)]
    torch.cuda.synchronize()
    want = {k: qlinear_int8_bits(*quant_int8(v), w, ws) for k, v in ((0, x), (1, x2))}
    assert all(np.array_equal(bf16_bits(y), want[0]) for y in ys)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = qpl.qlinear_int8(xd, wd, sd)
    for i in (0, 1, 0, 1, 1):
        xd.copy_(to_dev_bf16((x, x2)[i]))
        y.zero_()
        graph.replay()
        eager = qpl.qlinear_int8(xd, wd, sd)
        torch.cuda.synchronize()
        assert np.array_equal(bf16_bits(y), want[i]) and torch.equal(y, eager)
