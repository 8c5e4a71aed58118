"""The operators of a mixture-of-experts layer for any number of tokens: what is measured.

Four operators, in the order in which a layer uses them:

- norm:   a row's residual, an addend and its routed expert rows are added, the sum is normalised
          (root mean square) and given in BF16 and in 8 bits with scales;
- route:  router logits to picks, weights and the tokens grouped by expert;
- swiglu: the gate/up product of every expert with its own rows, the clamped SwiGLU and the
          8-bit hidden with scales, in one step;
- gemm:   the product of every expert with its own rows (the down projection).

`run` computes them in elementary torch operations, or with `own` set through the package's calls.
"""

import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
EPS = 2.0**-20
LIMIT = 7.0


def listed():
    return [
        # one decoded token between two layers: the residual and the attention's output, FP8 for the experts
        {"name": "norm decode", "op": "norm", "T": 1, "D": 7168, "delta": True, "k": 0, "quant": "fp8"},
        # a prompt's tokens behind the experts: eight routed rows each are weighted and added on the way
        {"name": "norm routed prompt", "op": "norm", "T": 4096, "D": 7168, "delta": False, "k": 8, "quant": "fp8"},
        # a prompt's latents in MXFP8, an odd number of them
        {"name": "norm latent mxfp8", "op": "norm", "T": 8191, "D": 3584, "delta": True, "k": 0, "quant": "mxfp8"},
        # one decoded token's routing
        {"name": "route decode", "op": "route", "T": 1, "E": 256, "k": 8, "bf16": False},
        # a long prompt's routing
        {"name": "route prompt", "op": "route", "T": 16384, "E": 256, "k": 8, "bf16": False},
        # many small experts, BF16 logits, an odd number of tokens
        {"name": "route many experts", "op": "route", "T": 4095, "E": 896, "k": 16, "bf16": True},
        # four decoded tokens: weights of some thirty experts are read for one row each
        {"name": "swiglu decode", "op": "swiglu", "T": 4, "E": 256, "k": 8, "K": 7168, "N": 2048, "skew": 0.0, "quant": "fp8"},
        # a batch of short prompts over many small experts: about ten rows each
        {"name": "swiglu many experts", "op": "swiglu", "T": 511, "E": 896, "k": 16, "K": 3584, "N": 1024, "skew": 0.5, "quant": "fp8"},
        # a long prompt: some hundred rows for each expert, unevenly spread
        {"name": "swiglu prompt", "op": "swiglu", "T": 8192, "E": 256, "k": 8, "K": 7168, "N": 2048, "skew": 0.5, "quant": "fp8"},
        # the smallest product: one token's eight down projections
        {"name": "gemm decode", "op": "gemm", "T": 1, "E": 256, "k": 8, "K": 2048, "N": 7168, "skew": 0.0, "quant": "fp8", "gather": False},
        # MXFP8 latents through one GPU's share of experts, rows gathered
        {"name": "gemm latent mxfp8", "op": "gemm", "T": 1237, "E": 56, "k": 2, "K": 3584, "N": 2048, "skew": 0.5, "quant": "mxfp8", "gather": True},
        # a long prompt's down projection
        {"name": "gemm prompt", "op": "gemm", "T": 8192, "E": 256, "k": 8, "K": 2048, "N": 7168, "skew": 0.5, "quant": "fp8", "gather": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "swiglu", "swiglu", "gemm", "gemm"])
    if op == "norm":
        k = rng.choice([0, 0, rng.randint(1, 16)])
        D = 128 * _log(rng, 2, 64)
        return {"op": op, "T": max(1, min(_log(rng, 1, 16384), 2**28 // ((k + 2) * D))), "D": D, "delta": rng.random() < 0.7 or not k,
                "k": k, "quant": rng.choice(["fp8", "mxfp8"])}
    if op == "route":
        E = _log(rng, 8, 1024)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 16)), "bf16": rng.random() < 0.5}
    E = _log(rng, 4, 256)
    case = {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(E, 8)), "K": 128 * _log(rng, 2, 56),
            "N": 128 * _log(rng, 2, 16 if op == "swiglu" else 56), "skew": rng.choice([0.0, 0.5, 1.0]), "quant": rng.choice(["fp8", "fp8", "mxfp8"])}
    if op == "gemm":
        case["N"] = min(case["N"], 128 * (7168 * 2048 // 128 // case["K"]))  # no expert larger than the listed ones
        case["gather"] = rng.random() < 0.5
    return case


# ---- inputs -------------------------------------------------------------------------------------


def _blocks(v, block):
    return v.view(*v.shape[:-1], v.shape[-1] // block, block)


def _fp8(v):
    """FP8 codes and FP32 scales per 128 values of v (FP32)."""
    b = _blocks(v, 128)
    s = b.abs().amax(-1, keepdim=True).clamp_min(1e-10) / 448.0
    return (b * (1.0 / s)).clamp(-448.0, 448.0).to(F8).view(v.shape), s.squeeze(-1)


def _mx_shared(amax):
    """The shared exponent of MXFP8 blocks with these maxima."""
    return torch.where(amax > 0, (torch.frexp(amax)[1] - 1 - 8).clamp(-127, 127), -127)


def _mxfp8(v):
    """MXFP8 codes and shared exponents (int32) per 32 values of v (FP32)."""
    b = _blocks(v, 32)
    e = _mx_shared(b.abs().amax(-1, keepdim=True))
    return torch.ldexp(b, -e).clamp(-448.0, 448.0).to(F8).view(v.shape), e.squeeze(-1)


def _rows(gen, T, D):
    """Activations: Gaussian, with another size for each token."""
    size = torch.exp2(torch.randn(T, 1, generator=gen, device=DEV))
    return torch.randn(T, D, generator=gen, device=DEV) * size


def _weights(gen, E, N, K):
    """FP8 expert weights [E, N, K], such that the products come out of the order of one, and their 128 x 128 scales."""
    w = torch.empty(E, N, K, dtype=F8, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        w[e : e + n] = (torch.randn(n, N, K, generator=gen, device=DEV) * 107.0).clamp_(-448.0, 448.0).to(F8)
    s = torch.rand(E, N // 128, K // 128, generator=gen, device=DEV) * 1.5 + 0.5
    return w, s / (107.0 * math.sqrt(K))


def _grouped(gen, T, E, k, skew):
    """offsets [E + 1], the token of each grouped row, and the longest group."""
    z = torch.empty(T, E, device=DEV).exponential_(generator=gen).log_().neg_() + skew * torch.randn(E, generator=gen, device=DEV)
    ids = z.topk(k, dim=-1).indices.flatten()
    count = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = count.cumsum(0)
    rows = (torch.sort(ids, stable=True).indices // k).to(torch.int32)
    return offsets, rows, int(count.max())


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] == "norm":
        T, D, k = c["T"], c["D"], c["k"]
        s["residual"] = _rows(gen, T, D).to(torch.bfloat16)
        s["gamma"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device=DEV)).to(torch.bfloat16)
        s["delta"] = _rows(gen, T, D).to(torch.bfloat16) if c["delta"] else None
        s["y"] = s["pos"] = s["weights"] = None
        if k:  # routed rows lie in the experts' order: each token's k rows are anywhere
            s["y"] = torch.randn(T * k, D, generator=gen, device=DEV).to(torch.bfloat16)
            s["pos"] = torch.randperm(T * k, generator=gen, device=DEV).to(torch.int32).view(T, k)
            w = torch.rand(T, k, generator=gen, device=DEV) + 0.05
            s["weights"] = w / w.sum(-1, keepdim=True) * 2.5
        return s
    if c["op"] == "route":
        z = torch.randn(c["T"], c["E"], generator=gen, device=DEV) * 2.0
        s["logits"] = z.to(torch.bfloat16) if c["bf16"] else z
        s["bias"] = torch.randn(c["E"], generator=gen, device=DEV) * 0.1
        return s
    T, E, k, K = c["T"], c["E"], c["k"], c["K"]
    s["offsets"], s["rows"], s["longest"] = _grouped(gen, T, E, k, c["skew"])
    if c["op"] == "gemm" and not c["gather"]:
        s["rows"] = None
    x = _rows(gen, T * k if s["rows"] is None else T, K)
    if c["quant"] == "fp8":
        s["x"], s["x_scale"] = _fp8(x)
    else:
        s["x"], e = _mxfp8(x)
        s["x_scale"] = (e + 127).to(torch.uint8)
    s["w"], s["w_scale"] = _weights(gen, E, c["N"] * (2 if c["op"] == "swiglu" else 1), K)
    return s


# ---- the operators in plain operations ----------------------------------------------------------


def _norm(s, real):
    """The sums and the statistics in 64 bits; the normalised row in `real`'s steps. Returns the sum, the row, its codes and scales."""
    h = s["residual"].double()
    if s["delta"] is not None:
        h = h + s["delta"].double()
    if s["y"] is not None:
        h = h + (s["weights"].double().unsqueeze(-1) * s["y"].double()[s["pos"].long()]).sum(1)
    h = h.to(real)
    rstd = (1.0 / (h.double().square().mean(-1, keepdim=True) + EPS).sqrt()).to(real)
    return h, (h * rstd) * s["gamma"].to(real)


def _plain_norm(s):
    h, v = _norm(s, torch.float32)
    if s["case"]["quant"] == "fp8":
        q, scale = _fp8(v)
    else:
        q, e = _mxfp8(v)
        scale = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return {"residual": h.to(torch.bfloat16), "out": v.to(torch.bfloat16), "q": q, "scale": scale}


def _plain_route(s):
    k, E = s["case"]["k"], s["case"]["E"]
    score = (1.0 / (1.0 + torch.exp(-s["logits"].double()))).float()
    ids = torch.sort(score + s["bias"], dim=-1, descending=True, stable=True).indices[:, :k]  # equal keys: the lower expert
    picked = score.gather(1, ids)
    weights = picked / picked.sum(-1, keepdim=True) * 2.5
    flat, order = torch.sort(ids.flatten(), stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.searchsorted(flat, torch.arange(E + 1, device=flat.device))
    return {"ids": ids.to(torch.int32), "weights": weights, "offsets": offsets.to(torch.int32),
            "rows": (order // k).to(torch.int32), "pos": pos.to(torch.int32).view(-1, k)}


def _plain_x(s, real):
    x = s["x"].to(real)
    if s["case"]["quant"] == "fp8":
        scale, block = s["x_scale"].to(real), 128
    else:
        e = s["x_scale"].to(torch.int32) - 127
        scale, block = torch.ldexp(torch.ones_like(e, dtype=real), e), 32
    x = (_blocks(x, block) * scale.unsqueeze(-1)).view(x.shape)
    return x if s["rows"] is None else x[s["rows"].long()]


def _plain_w(w, scale, real):
    n, N, K = w.shape
    return (w.to(real).view(n, N // 128, 128, K // 128, 128) * scale.to(real)[:, :, None, :, None]).view(n, N, K)


def _plain_products(s):
    """Each grouped row times its expert's weights, in FP32."""
    offsets, E = s["offsets"].long(), s["case"]["E"]
    x = _plain_x(s, torch.float32)
    R = x.shape[0]
    row = torch.arange(R, device=x.device)
    expert = torch.searchsorted(offsets, row, right=True) - 1
    if R < E:  # few rows: the weights of each row's own expert
        w = _plain_w(s["w"][expert], s["w_scale"][expert], torch.float32)
        return torch.bmm(w, x.unsqueeze(-1)).squeeze(-1)
    at = offsets[:-1, None] + torch.arange(s["longest"], device=x.device)  # every group as long as the longest
    y = torch.bmm(x[at.clamp_max(R - 1)], _plain_w(s["w"], s["w_scale"], torch.float32).transpose(1, 2))
    return y[expert, row - offsets[expert]]


def _act(y):
    I = y.shape[-1] // 2  # rows of the first half are up, of the second gate
    up, gate = y[:, :I].clamp(-LIMIT, LIMIT), y[:, I:].clamp_max(LIMIT)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_swiglu(s):
    q, scale = _fp8(_act(_plain_products(s)))
    return {"q": q, "scale": scale}


def _plain_gemm(s):
    return {"y": _plain_products(s).to(torch.bfloat16)}


# ---- the framework's calls ----------------------------------------------------------------------


def _own_norm(s):
    import fp8_block_scaled_moe_amd as moe

    residual, out, q, scale = moe.add_rmsnorm_quant(s["residual"], s["gamma"], EPS, delta=s["delta"], y=s["y"], pos=s["pos"],
                                                    weights=s["weights"], quant=s["case"]["quant"])
    if s["case"]["quant"] == "mxfp8":
        scale = scale.view(torch.float8_e8m0fnu).float()
    return {"residual": residual, "out": out, "q": q.view(F8), "scale": scale}


def _own_route(s):
    import fp8_block_scaled_moe_amd as moe

    r = moe.route_rows(s["logits"], s["bias"], top_k=s["case"]["k"], routed_scale=2.5)
    return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "rows": r.rows, "pos": r.pos}


def _own_swiglu(s):
    import fp8_block_scaled_moe_amd as moe

    q, scale = moe.grouped_swiglu(s["x"], s["x_scale"], s["w"], s["w_scale"], s["offsets"], limit=LIMIT, rows=s["rows"])
    return {"q": q.view(F8), "scale": scale}


def _own_gemm(s):
    import fp8_block_scaled_moe_amd as moe

    return {"y": moe.grouped_gemm(s["x"], s["x_scale"], s["w"], s["w_scale"], s["offsets"], rows=s["rows"])}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "route": _own_route, "swiglu": _own_swiglu, "gemm": _own_gemm}[op](state)
    return {"norm": _plain_norm, "route": _plain_route, "swiglu": _plain_swiglu, "gemm": _plain_gemm}[op](state)


# ---- what a pass cannot do without --------------------------------------------------------------


def work(case):
    c, T = case, case["T"]
    if c["op"] == "norm":
        D, k = c["D"], c["k"]
        read = T * D * 2 * (1 + bool(c["delta"]) + k) + T * k * 8 + D * 2
        return {"bytes": read + T * D * (2 + 2 + 1) + T * D // (32 if c["quant"] == "mxfp8" else 128) * (1 if c["quant"] == "mxfp8" else 4),
                "flops": T * D * (6 + 2 * k)}
    if c["op"] == "route":
        E, k = c["E"], c["k"]
        return {"bytes": T * E * (2 if c["bf16"] else 4) + E * 8 + T * k * 16, "flops": T * E * 6}
    E, k, K = c["E"], c["k"], c["K"]
    R, N = T * k, c["N"] * (2 if c["op"] == "swiglu" else 1)
    touched = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token picks, on average
    tokens = T if c["op"] == "swiglu" or c["gather"] else R
    read = touched * (N * K + N * K // 4096) + tokens * (K + K // 32) + R * 4 + E * 4
    wrote = R * c["N"] * (1 + 1 / 32 if c["op"] == "swiglu" else 2)
    return {"bytes": read + wrote, "flops": 2.0 * R * N * K}


# ---- the definitions in 64 bits -----------------------------------------------------------------


def _to_grid8(v):
    """The nearest e4m3 value of each v (FP64), ties to the even code, none over 448."""
    a = v.abs().clamp_max(448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0**-6))) - 3)
    return torch.round(a / step) * step * torch.sign(v)


def _exact_norm(case, seed):
    s = prepare(case, seed)
    T, D, k = case["T"], case["D"], case["k"]
    total = s["residual"].to(torch.float64).clone()
    if case["delta"]:
        total += s["delta"].to(torch.float64)
    for j in range(k):
        total += s["weights"][:, j : j + 1].to(torch.float64) * s["y"][s["pos"][:, j].long()].to(torch.float64)
    root = torch.sqrt((total * total).sum(1, keepdim=True) / D + EPS)
    v = total / root * s["gamma"].to(torch.float64)
    block = 128 if case["quant"] == "fp8" else 32
    largest = v.reshape(T, D // block, block).abs().max(-1).values
    if case["quant"] == "fp8":
        scale = torch.clamp_min(largest, 1e-10) / 448.0
    else:
        scale = torch.exp2(torch.floor(torch.log2(largest)).clamp(-119, 135) - 8)
    q = _to_grid8(v / scale.repeat_interleave(block, 1))
    # an MXFP8 scale is a power of two that the FP32 row decides: next to one, 64 bits have no say
    return {"residual": total, "out": v, "q": q, "scale": scale if case["quant"] == "fp8" else None}


def _exact_route(case, seed):
    s = prepare(case, seed)
    z = s["logits"].to(torch.float64)
    score = torch.special.expit(z)
    key = score.to(torch.float32) + s["bias"]  # the keys are compared in FP32
    left, picks = key.clone(), []
    for _ in range(case["k"]):
        best = left.max(1, keepdim=True).values
        e = (left == best).to(torch.int8).argmax(1, keepdim=True)
        left.scatter_(1, e, float("-inf"))
        picks.append(e)
    ids = torch.cat(picks, 1)
    picked = score.gather(1, ids)
    rows, pos, offsets, at = [], torch.zeros(ids.numel(), dtype=torch.int64, device=ids.device), [0], 0
    flat = ids.reshape(-1)
    for e in range(case["E"]):
        mine = torch.nonzero(flat == e).reshape(-1)
        rows.append(mine // case["k"])
        pos[mine] = torch.arange(mine.numel(), device=ids.device) + at
        at += mine.numel()
        offsets.append(at)
    return {"ids": ids, "weights": 2.5 * picked / picked.sum(1, keepdim=True), "offsets": torch.tensor(offsets), "rows": torch.cat(rows),
            "pos": pos.view(ids.shape)}


def _exact_products(s, case):
    """Group after group, block of 128 after block, in FP64."""
    K, N = case["K"], s["w"].shape[1]
    ends = s["offsets"].tolist()
    y = torch.zeros(ends[-1], N, dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        x = (s["x"][s["rows"][lo:hi].long()] if s["rows"] is not None else s["x"][lo:hi]).to(torch.float64)
        xs = s["x_scale"][s["rows"][lo:hi].long()] if s["rows"] is not None else s["x_scale"][lo:hi]
        xs = xs.to(torch.float64) if case["quant"] == "fp8" else torch.exp2(xs.to(torch.float64) - 127)
        x = x * xs.repeat_interleave(K // xs.shape[1], 1)
        w = s["w"][e].to(torch.float64)
        w = w * s["w_scale"][e].to(torch.float64).repeat_interleave(128, 0).repeat_interleave(128, 1)
        y[lo:hi] = x @ w.t()
    return y


def exact(case, seed):
    if case["op"] == "norm":
        return _exact_norm(case, seed)
    if case["op"] == "route":
        return _exact_route(case, seed)
    s = prepare(case, seed)
    y = _exact_products(s, case)
    if case["op"] == "gemm":
        return {"y": y}
    up, gate = y[:, : case["N"]], y[:, case["N"] :]
    up, gate = torch.clamp(up, min=-LIMIT, max=LIMIT), torch.minimum(gate, torch.full_like(gate, LIMIT))
    act = up * gate * torch.special.expit(gate)
    largest = act.reshape(act.shape[0], -1, 128).abs().max(-1).values
    scale = torch.clamp_min(largest, 1e-10) / 448.0
    return {"q": _to_grid8(act / scale.repeat_interleave(128, 1)), "scale": scale}
