"""The plan for more than 1024 experts, in slices of them: against a stable sort, at the
borders of slices, chunks and of the rule that chooses between the forms."""
import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as qpl
from helpers import host, to_dev
from oracle.int8 import plan_ref


def sorted_plan(ids, E):
    """plan_ref by a stable sort, for many choices."""
    k = ids.reshape(-1).astype(np.int64)
    ok = (k >= 0) & (k < E)
    order = np.argsort(np.where(ok, k, E), kind="stable")[:ok.sum()]
    slot, row_index = np.full(k.size, -1, np.int32), np.full(k.size, -1, np.int32)
    slot[order] = np.arange(order.size)
    row_index[:order.size] = order // ids.shape[1]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(k[ok], minlength=E))])
    return row_index, slot.reshape(ids.shape), offsets


def draw(T, topk, E, kind, seed=0):
    rng = np.random.default_rng(seed + T)
    if kind == "border":                                  # the experts at both ends of every slice
        ends = np.unique(np.clip(np.concatenate([np.arange(0, E + 1024, 1024) + d for d in (-1, 0, 1)]), -1, E))
        return rng.choice(ends, (T, topk)).astype(np.int32)
    if kind == "last":
        return np.full((T, topk), E - 1, np.int32)
    if kind == "none":
        return np.full((T, topk), E, np.int32)
    ids = rng.integers(-E // 8 if kind == "invalid" else 0, E + (E // 8 if kind == "invalid" else 0), (T, topk))
    ids = ids.astype(np.int32)
    if kind == "invalid":
        ids[0, 0], ids[-1, -1] = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    return ids


def test_the_sort_is_the_plan():
    for kind in ("invalid", "border", "last", "none"):
        ids = draw(50, 3, 1030, kind)
        assert all(np.array_equal(a, b) for a, b in zip(sorted_plan(ids, 1030), plan_ref(ids, 1030)))


def test_no_plan_reads_all_choices_for_each_of_many_experts():
    # the form without a workspace reads all choices once per expert: only where that is little
    for T, topk, E in ((1 << 20, 2, 2049), (1 << 20, 8, 65536), ((1 << 23) - 256, 255, 65536), (4097, 1, 4096),
                       (1, 1, 65536), (12289, 1, 257)):
        assert qpl.expert_plan_workspace_bytes(T, topk, E) > 0, (T, topk, E)
    for T, topk, E in ((2048, 1, 8192), (6144, 2, 1024), (8192, 1, 2048), (32767, 1, 256), (1, 1, 1)):
        assert qpl.expert_plan_workspace_bytes(T, topk, E) == 0, (T, topk, E)


SIZES = [(4096, 3, 1024, "invalid"), (12289, 1, 257, "invalid"), (12288, 1, 256, "random"), (6000, 2, 700, "last"),
         (8192, 1, 2048, "border"), (2048, 1, 8192, "invalid"), (8193, 4, 513, "random"), (15000, 2, 256, "none"),
         (1, 1, 65536, "random"), (1, 1, 8193, "last"), (4096, 1, 8192, "invalid"), (4097, 1, 1025, "invalid"),
         (4097, 1, 2048, "border"), (2049, 2, 2049, "border"), (33, 7, 9000, "invalid"), (700, 8, 65535, "border"),
         (3000, 3, 4097, "last"), (3000, 3, 4097, "none"), (20011, 5, 1500, "invalid"), (1 << 20, 2, 2049, "invalid"),
         (70000, 8, 65536, "invalid"), (1 << 19, 3, 1025, "border")]


@pytest.mark.gpu
@pytest.mark.parametrize("T,topk,E,kind", SIZES)
def test_plan_in_slices(T, topk, E, kind):
    ids = draw(T, topk, E, kind)
    need = qpl.expert_plan_workspace_bytes(T, topk, E)
    work = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    n = T * topk
    outs = [torch.full((k + 64,), 7, dtype=torch.int32, device="cuda") for k in (n, n, E + 1)]
    qpl.expert_plan(to_dev(ids), E, row_index=outs[0][:n], slot=outs[1][:n].view(T, topk), offsets=outs[2][:E + 1],
                    workspace=work[:need] if need else None)
    for name, got, want in zip(("row_index", "slot", "offsets"), outs, sorted_plan(ids, E)):
        assert np.array_equal(host(got)[:want.size], want.reshape(-1)), name
        assert np.all(host(got)[want.size:] == 7), name
    assert np.all(host(work)[need:] == 0x5A)


@pytest.mark.gpu
def test_slices_in_a_graph_and_in_the_mlp():
    T, topk, E, K, H, N = 300, 2, 8300, 32, 16, 24
    ids = to_dev(draw(T, topk, E, "invalid"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = qpl.expert_plan(ids, E)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    wt = torch.rand((T, topk), generator=g, device="cuda")
    f1, f2 = (dict(weight=torch.randint(-127, 128, (E, a, b), generator=g, device="cuda", dtype=torch.int8),
                   weight_scale=torch.rand((E, a), generator=g, device="cuda") * 1e-2) for a, b in ((H, K), (N, H)))
    for seed in range(4):
        ids.copy_(to_dev(draw(T, topk, E, "invalid", seed)))
        for t in outs:
            t.zero_()
        graph.replay()
        row_index, slot, offsets = qpl.expert_plan(ids, E)
        assert all(np.array_equal(host(a), b) for a, b in zip(outs, sorted_plan(host(ids), E)))
        assert all(torch.equal(a, b) for a, b in zip(outs, (row_index, slot, offsets)))
        h = qpl.qlinear_grouped_int8(x, f1["weight"], f1["weight_scale"], offsets, row_index=row_index, act="gelu_tanh")
        y = qpl.expert_combine(qpl.qlinear_grouped_int8(h, f2["weight"], f2["weight_scale"], offsets), slot, wt)
        assert torch.equal(qpl.qlinear_moe_int8(x, ids, wt, f1, f2), y) and bool(y.any())


def test_refusals_without_a_workspace():
    # no device: a call that passes every check before it reports that
    if torch.cuda.is_available():
        pytest.skip("forces the no-device status; a GPU is present")
    import ctypes
    lib, p = qpl.load(), ctypes.c_void_p(1 << 20)
    null, device = 1, 6
    for T, topk, E, want in ((4, 2, 65536, device), (32767, 1, 1024, device), (1 << 19, 1, 65536, device),
                             ((1 << 19) + 1, 1, 65536, null), (1 << 20, 8, 65536, null), (32768, 1, 1024, null),
                             (1 << 16, 2, 300, null)):
        assert lib.expert_plan(p, T, topk, E, p, p, p, None, 0, None) == want, (T, topk, E)
        need = qpl.expert_plan_workspace_bytes(T, topk, E)
        assert need > 0 and lib.expert_plan(p, T, topk, E, p, p, p, p, need - 1, None) == 5
        assert lib.expert_plan(p, T, topk, E, p, p, p, p, need, None) == device


@pytest.mark.gpu
@pytest.mark.parametrize("T,topk,E,kind", [(4, 2, 65536, "invalid"), (20011, 1, 700, "invalid"), (9000, 3, 1500, "border"),
                                           (5000, 2, 4097, "last")])
def test_plan_without_a_workspace(T, topk, E, kind):
    assert qpl.expert_plan_workspace_bytes(T, topk, E) > 0
    ids = draw(T, topk, E, kind)
    d = to_dev(ids)
    outs = [torch.full((k,), 7, dtype=torch.int32, device="cuda") for k in (T * topk, T * topk, E + 1)]
    status = qpl.load().expert_plan(d.data_ptr(), T, topk, E, *(t.data_ptr() for t in outs), None, 0,
                                    torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0
    for name, got, want in zip(("row_index", "slot", "offsets"), outs, sorted_plan(ids, E)):
        assert np.array_equal(host(got), want.reshape(-1)), name
