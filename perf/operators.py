"""Measured cases of the 8-bit integer linears: dense, grouped by expert, and what routes tokens to the experts.

``run`` computes a case in plain torch operations (``own`` false) or through the package's entry points
(``own`` true); both take what ``prepare`` makes.  The operators:

* linear   y = act((q_x q_w^T) s_x s_w), with q_x, s_x each row's 8-bit codes and scale:
           a = max |x|, s = a / 127, q = rint(127 x / a) (ties to even; a zero row has s = 0 and codes 0);
           optionally x is first divided by smoothing factors and rounded to bf16, and the result can go
           through GELU (tanh form) or be split into q, k and v [heads, tokens, head_dim];
* grouped  the same product with rows sorted by expert, a weight for each expert, and rows gathered from x;
* plan     router choices [tokens, k] -> rows sorted by expert (stable), each choice's place, and the
           experts' first rows;
* combine  out[t] = sum_j weight[t, j] y[slot[t, j]];
* moe      plan, grouped product with GELU, grouped product, combine: a GELU MLP of experts.
"""
import math

import torch

own = False

BF16 = torch.bfloat16


# ---- cases -------------------------------------------------------------------------------------------
def listed():
    return [
        # one token through a square projection: a single-user decoding step
        dict(name="linear_token", op="linear", M=1, K=4096, N=4096, form="plain", smooth=False),
        # a decoding batch through an up-projection with smoothing factors and GELU
        dict(name="linear_batch", op="linear", M=24, K=4096, N=12288, form="gelu", smooth=True),
        # a chunk of a prompt, with no size a multiple of a tile
        dict(name="linear_chunk", op="linear", M=515, K=2080, N=5003, form="plain", smooth=False),
        # a long prompt through a fused QKV projection, written after 512 tokens that are there already
        dict(name="linear_prompt_qkv", op="linear", M=4096, K=4096, N=12288, form="qkv", smooth=False, heads=32),
        # decoding 32 sequences, 8 of 64 experts each: most experts see a handful of rows
        dict(name="grouped_decode", op="grouped", T=32, topk=8, E=64, K=2048, N=1536, gelu=True, skew=1.0),
        # a prompt over 32 experts, unevenly used
        dict(name="grouped_prompt", op="grouped", T=4096, topk=4, E=32, K=2048, N=4096, gelu=False, skew=1.0),
        # a few tokens through a whole MLP of experts
        dict(name="moe_decode", op="moe", T=7, topk=4, E=16, K=2048, H=1408, N=2048, skew=0.5),
        # a prompt through it
        dict(name="moe_prompt", op="moe", T=2048, topk=4, E=32, K=2048, H=1408, N=2048, skew=0.5),
        # router choices of a decoding step and of a batch of long prompts
        dict(name="plan_decode", op="plan", T=32, topk=8, E=64, skew=1.0),
        dict(name="plan_prompt", op="plan", T=16384, topk=8, E=256, skew=1.0),
        # the experts' rows back to their tokens, for a decoding step and a prompt
        dict(name="combine_decode", op="combine", T=37, topk=8, N=2048),
        dict(name="combine_prompt", op="combine", T=8192, topk=4, N=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "moe", "plan", "combine"])
    if op == "linear":
        form = rng.choice(["plain", "gelu", "qkv"])
        c = dict(op=op, M=_log(rng, 1, 4608), K=16 * _log(rng, 4, 512), form=form, smooth=rng.random() < 0.3)
        if form == "qkv":
            c["heads"] = _log(rng, 1, 32)
            c["N"] = 3 * 128 * c["heads"]
        else:
            c["N"] = _log(rng, 64, 12288)
        while c["M"] * c["K"] * c["N"] > 4096 * 4096 * 12288:
            c["M"] = c["M"] // 2 + 1
        return c
    E = _log(rng, 2, 128)
    topk = min(E, rng.randint(1, 8))
    skew = rng.choice([0.0, 0.5, 1.0])
    if op == "grouped":
        return dict(op=op, T=_log(rng, 1, 4096), topk=min(topk, 4), E=min(E, 64), K=16 * _log(rng, 16, 128),
                    N=_log(rng, 256, 4096), gelu=rng.random() < 0.5, skew=skew)
    if op == "moe":
        return dict(op=op, T=_log(rng, 1, 2048), topk=min(topk, 4), E=min(E, 32), K=16 * _log(rng, 32, 128),
                    H=16 * _log(rng, 16, 88), N=_log(rng, 256, 2048), skew=skew)
    if op == "plan":
        return dict(op=op, T=_log(rng, 1, 16384), topk=topk, E=E, skew=skew)
    return dict(op=op, T=_log(rng, 1, 8192), topk=min(topk, 4), N=_log(rng, 64, 4096))


# ---- inputs ------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activation(g, M, K):
    """N(0, 1) with one channel in a hundred ten times larger, as transformer activations have them."""
    x = torch.randn((M, K), generator=g, device="cuda")
    outlier = torch.randperm(K, generator=g, device="cuda")[: max(K // 100, 1)]
    x[:, outlier] *= 10.0
    return x.to(BF16)


def _weight(g, *shape):
    """Codes int8 [..., K] and scales float32 [...] of an N(0, 0.02) weight."""
    w = torch.randn(shape, generator=g, device="cuda") * 0.02
    a = w.abs().amax(-1, keepdim=True)
    return torch.round(w * (127.0 / a)).to(torch.int8), (a / 127.0).squeeze(-1).contiguous()


def _choices(g, T, topk, E, skew):
    """topk different experts of each token, some experts more popular than others."""
    score = torch.rand((T, E), generator=g, device="cuda").log().neg().log().neg()
    score += skew * torch.randn((E,), generator=g, device="cuda")
    return score.topk(topk, dim=1).indices.to(torch.int32)


def _sorted(ids, E):
    """(row_index, slot, offsets) of the choices, in torch."""
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(flat.numel(), device=flat.device)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum((flat[:, None] == torch.arange(E, device=flat.device)).sum(0), 0)
    return ((order // ids.shape[1]).to(torch.int32), slot.reshape(ids.shape).to(torch.int32),
            offsets.to(torch.int32))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = _activation(g, M, K)
        s["w"], s["ws"] = _weight(g, N, K)
        s["smooth"] = (0.25 * torch.randn((K,), generator=g, device="cuda")).exp() if case["smooth"] else None
        if case["form"] == "qkv":
            s["qkv"] = [torch.zeros((case["heads"], M + 512, N // 3 // case["heads"]), dtype=BF16, device="cuda")
                        for _ in range(3)]
    elif op in ("grouped", "moe"):
        E = case["E"]
        s["x"] = _activation(g, case["T"], case["K"])
        s["ids"] = _choices(g, case["T"], case["topk"], E, case["skew"])
        if op == "grouped":
            s["w"], s["ws"] = _weight(g, E, case["N"], case["K"])
            s["row_index"], _, s["offsets"] = _sorted(s["ids"], E)
            s["bounds"] = s["offsets"].tolist()
        else:
            s["w1"], s["ws1"] = _weight(g, E, case["H"], case["K"])
            s["w2"], s["ws2"] = _weight(g, E, case["N"], case["H"])
            s["weights"] = torch.randn(s["ids"].shape, generator=g, device="cuda").softmax(1)
    elif op == "plan":
        s["ids"] = _choices(g, case["T"], case["topk"], case["E"], case["skew"])
    else:
        T, k, N = case["T"], case["topk"], case["N"]
        s["y"] = torch.randn((T * k, N), generator=g, device="cuda").to(BF16)
        s["slot"] = torch.randperm(T * k, generator=g, device="cuda").reshape(T, k).to(torch.int32)
        s["weights"] = torch.randn((T, k), generator=g, device="cuda").softmax(1)
    return s


# ---- plain forms -------------------------------------------------------------------------------------
def _quantize(x, smooth=None):
    """Codes as float32 values and scales [M, 1]; the codes in 64 bits, because 127 x / a can lie on a border."""
    v = x.float()
    if smooth is not None:
        v = (v / smooth).to(BF16).float()
    a = v.abs().amax(1, keepdim=True)
    q = torch.round(v.double() * 127.0 / a.double())
    return torch.where(a > 0, q, torch.zeros_like(q)).float(), a / 127.0


def _gelu(v):
    return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))


def _product(q, s, w, ws, gelu):
    v = (q @ w.float().t()) * s * ws
    return (_gelu(v) if gelu else v).to(BF16)


def _grouped(x, w, ws, row_index, bounds, gelu):
    q, s = _quantize(x)
    row = row_index.long()
    y = torch.empty((row.numel(), w.shape[1]), dtype=BF16, device=x.device)
    for e in range(w.shape[0]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            y[lo:hi] = _product(q[row[lo:hi]], s[row[lo:hi]], w[e], ws[e], gelu)
    return y


def _combine(y, slot, weights):
    return (y[slot.long()].float() * weights[..., None]).sum(1).to(BF16)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import precision_quantized_linear_amd as qpl
        if op == "linear":
            if c["form"] == "qkv":
                return qpl.qlinear_int8(state["x"], state["w"], state["ws"], smooth=state["smooth"],
                                        qkv=(*state["qkv"], 512))
            return qpl.qlinear_int8(state["x"], state["w"], state["ws"], smooth=state["smooth"],
                                    act="gelu_tanh" if c["form"] == "gelu" else None)
        if op == "grouped":
            return qpl.qlinear_grouped_int8(state["x"], state["w"], state["ws"], state["offsets"],
                                            row_index=state["row_index"], act="gelu_tanh" if c["gelu"] else None)
        if op == "moe":
            return qpl.qlinear_moe_int8(state["x"], state["ids"], state["weights"],
                                        dict(weight=state["w1"], weight_scale=state["ws1"]),
                                        dict(weight=state["w2"], weight_scale=state["ws2"]))
        if op == "plan":
            return qpl.expert_plan(state["ids"], c["E"])
        return qpl.expert_combine(state["y"], state["slot"], state["weights"])
    if op == "linear":
        q, s = _quantize(state["x"], state["smooth"])
        y = _product(q, s, state["w"], state["ws"], c["form"] == "gelu")
        if c["form"] == "qkv":
            heads = c["heads"]
            for part, out in zip(y.chunk(3, dim=1), state["qkv"]):
                out[:, 512:] = part.reshape(c["M"], heads, -1).transpose(0, 1)
            return tuple(state["qkv"])
        return y
    if op == "grouped":
        return _grouped(state["x"], state["w"], state["ws"], state["row_index"], state["bounds"], c["gelu"])
    if op == "moe":
        row_index, slot, offsets = _sorted(state["ids"], c["E"])
        bounds = offsets.tolist()
        h = _grouped(state["x"], state["w1"], state["ws1"], row_index, bounds, True)
        rows = torch.arange(h.shape[0], device=h.device)
        y = _grouped(h, state["w2"], state["ws2"], rows, bounds, False)
        return _combine(y, slot, state["weights"])
    if op == "plan":
        return _sorted(state["ids"], c["E"])
    return _combine(state["y"], state["slot"], state["weights"])


# ---- what a pass cannot do without -------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return dict(bytes=2 * M * K + N * K + 4 * N + 2 * M * N + (4 * K if case["smooth"] else 0), flops=2 * M * N * K)
    if op == "plan":
        return dict(bytes=12 * case["T"] * case["topk"] + 4 * (case["E"] + 1), flops=case["T"] * case["topk"])
    T, k, N = case["T"], case["topk"], case["N"]
    R = T * k
    if op == "combine":
        return dict(bytes=2 * R * N + 8 * R + 2 * T * N, flops=2 * R * N)
    # the weights of at most min(E, R) experts are read; expected number of them for even use
    E, K = case["E"], case["K"]
    used = E * (1.0 - (1.0 - k / E) ** T)
    if op == "grouped":
        return dict(bytes=int(2 * T * K + used * N * (K + 4) + 4 * R + 4 * (E + 1) + 2 * R * N), flops=2 * R * N * K)
    H = case["H"]
    return dict(bytes=int(2 * T * K + used * (H * (K + 4) + N * (H + 4)) + 8 * R + 2 * T * N),
                flops=2 * R * H * (K + N))


# ---- the definition in 64 bits -----------------------------------------------------------------------
def _codes64(x, smooth=None):
    v = x.to(torch.float64)
    if smooth is not None:
        # the smoothed activation is a bf16 tensor by definition: a correctly rounded fp32 quotient, then bf16
        v = (v / smooth.to(torch.float64)).to(torch.float32).to(BF16).to(torch.float64)
    top = v.abs().max(dim=1, keepdim=True).values
    codes = torch.zeros_like(v)
    live = top[:, 0] > 0
    codes[live] = (127.0 * v[live] / top[live]).round()
    return codes, top / 127.0


def _gelu64(v):
    u = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
    return v / (1.0 + torch.exp(-2.0 * u))


def _experts64(codes, scales, choice, w, ws, gelu):
    """Rows codes[i] scales[i] times the weight of expert choice[i], in 64 bits."""
    y = torch.zeros((codes.shape[0], w.shape[1]), dtype=torch.float64, device=codes.device)
    for e in range(w.shape[0]):
        rows = (choice == e).nonzero()[:, 0]
        if rows.numel():
            v = torch.mm(codes[rows], w[e].to(torch.float64).t().contiguous())
            v = v * scales[rows] * ws[e].to(torch.float64)
            y[rows] = _gelu64(v) if gelu else v
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "linear":
        codes, scale = _codes64(s["x"], s["smooth"])
        v = torch.mm(codes, s["w"].to(torch.float64).t().contiguous()) * scale * s["ws"].to(torch.float64)
        if case["form"] == "gelu":
            return _gelu64(v)
        if case["form"] == "qkv":
            heads, M = case["heads"], case["M"]
            out = torch.zeros((3, heads, M + 512, v.shape[1] // 3 // heads), dtype=torch.float64, device=v.device)
            out[:, :, 512:] = v.reshape(M, 3, heads, -1).permute(1, 2, 0, 3)
            return tuple(out)
        return v
    if op == "combine":
        T, k = s["slot"].shape
        out = torch.zeros((T, s["y"].shape[1]), dtype=torch.float64, device=s["y"].device)
        for j in range(k):
            out += s["weights"][:, j:j + 1].to(torch.float64) * s["y"][s["slot"][:, j].long()].to(torch.float64)
        return out
    codes, scale = _codes64(s["x"])
    k = case["topk"]
    choice = s["ids"].reshape(-1)
    if op == "grouped":
        choice, order = torch.sort(choice, stable=True)
        token = order // k
        return _experts64(codes[token], scale[token], choice, s["w"], s["ws"], case["gelu"])
    # the hidden activation is a bf16 tensor by definition
    token = torch.arange(choice.numel(), device=choice.device) // k
    h = _experts64(codes[token], scale[token], choice, s["w1"], s["ws1"], True).to(BF16)
    codes, scale = _codes64(h)
    y = _experts64(codes, scale, choice, s["w2"], s["ws2"], False).to(BF16).to(torch.float64)
    return (y.reshape(-1, k, y.shape[1]) * s["weights"].to(torch.float64)[..., None]).sum(1)
