"""Speed cases of the routed-layer operators: scored routing with its gradient,
the gradient of the weighted combine, MXFP4 quantisation and the indirect
expert product with both operands in MXFP4.

Each case can be run in two forms.  With `own` false, `run` computes the
operator from elementary torch operations; with `own` true it makes the
framework's calls.  `exact` is the operator's definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SZ = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------------- cases
def _route(**kw):
    c = dict(op="route", T=1, E=256, k=8, dtype="f32", score="sigmoid", bias=True, n_groups=1, topk_groups=1,
             group_score="max", normalize=True, scale=1.0, pad=0)
    c.update(kw)
    return c


def _route_bwd(**kw):
    c = dict(op="route_backward", T=1, E=256, k=8, dtype="f32", score="sigmoid", normalize=True, scale=1.0)
    c.update(kw)
    return c


def _combine_bwd(**kw):
    c = dict(op="combine_backward", T=1, k=8, n=2048, ddst=True)
    c.update(kw)
    return c


def _quant(**kw):
    c = dict(op="quantize", rows=1, n=2048, dtype="bf16")
    c.update(kw)
    return c


def _product(**kw):
    c = dict(op="product", T=1, E=256, k=8, n_in=2048, n_out=512, dtype="bf16", mode="broadcast", routing="uniform")
    c.update(kw)
    return c


def listed():
    return [
        # one generated token through the router of a 256-expert layer that picks 4 of 8 groups
        _route(name="route_one_token", n_groups=8, topk_groups=4, group_score="top2", scale=2.5),
        # the same router over a 4096-token prompt
        _route(name="route_prompt_groups", T=4096, n_groups=8, topk_groups=4, group_score="top2", scale=2.5),
        # a batch through a 128-expert top-4 softmax router whose half-precision logits are columns of a wider
        # matrix product (rows 16 elements apart from contiguous)
        _route(name="route_batch_softmax", T=8191, E=128, k=4, dtype="bf16", score="softmax", bias=False,
               normalize=False, pad=16),
        # training the 256-expert router on a 4096-token prompt: gradient of the chosen experts' logits
        _route_bwd(name="route_backward_sigmoid", T=4096, scale=2.5),
        # training a 128-expert softmax router with unnormalised weights: every logit has a gradient
        _route_bwd(name="route_backward_softmax", T=16384, E=128, k=4, dtype="bf16", score="softmax",
                   normalize=False),
        # gradient of the combine of a 64-expert layer's outputs, 512 tokens
        _combine_bwd(name="combine_backward_512", T=512, k=6, n=2048),
        # the same over a 4096-token prompt of the 7168-wide layer
        _combine_bwd(name="combine_backward_4096", T=4096, k=8, n=7168),
        # activations of a decode batch
        _quant(name="quantize_decode_rows", rows=8, n=7168, dtype="f32"),
        # the gate matrices of a 64-expert layer, converted once when a model is loaded
        _quant(name="quantize_expert_stack", rows=64 * 1408, n=2048),
        # four tokens being generated, 256 experts of width 512
        _product(name="product_decode", T=4),
        # per-slot product over 8192 tokens with a few popular experts, sizes that end inside a tile
        _product(name="product_skewed", T=8192, E=128, k=4, n_in=2880, n_out=2880, mode="per_slot", routing="zipf"),
        # gate product of a 4096-token prompt, 256 experts
        _product(name="product_prompt", T=4096, n_in=7168, n_out=2048, routing="skew"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "combine_backward", "quantize", "product"])
    if op == "route":
        n_groups = rng.choice([1, 1, 2, 4, 8, 12])
        size = _log_int(rng, 3, 512 // n_groups)
        topk_groups = rng.randint(1, n_groups)
        E = n_groups * size
        return _route(T=_log_int(rng, 1, 16384), E=E, k=rng.randint(2, min(16, topk_groups * size)),
                      dtype=rng.choice(["f32", "bf16", "f16"]), score=rng.choice(["sigmoid", "softmax"]),
                      bias=rng.random() < 0.6, n_groups=n_groups, topk_groups=topk_groups,
                      group_score=rng.choice(["max", "top2"]), normalize=rng.random() < 0.6,
                      scale=rng.choice([1.0, 2.5]), pad=rng.choice([0, 0, 1, 16]))
    if op == "route_backward":
        E = _log_int(rng, 4, 512)
        return _route_bwd(T=_log_int(rng, 1, 16384), E=E, k=rng.randint(2, min(16, E)),
                          dtype=rng.choice(["f32", "bf16", "f16"]), score=rng.choice(["sigmoid", "softmax"]),
                          normalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
    if op == "combine_backward":
        T, k = _log_int(rng, 1, 8192), rng.randint(1, 10)
        n = _log_int(rng, 100, min(8192, 4096 * 8 * 7168 // (T * k)))
        return _combine_bwd(T=T, k=k, n=n - n % 4 if rng.random() < 0.7 else n, ddst=rng.random() < 0.7)
    if op == "quantize":
        rows = _log_int(rng, 1, 100000)
        return _quant(rows=rows, n=32 * _log_int(rng, 1, min(256, 64 * 1408 * 64 // rows)),
                      dtype=rng.choice(["f32", "bf16", "f16"]))
    while True:
        E = rng.choice([8, 32, 60, 64, 128, 256])
        c = _product(T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, 8), n_in=32 * _log_int(rng, 4, 224),
                     n_out=_log_int(rng, 100, 4096), dtype=rng.choice(["f32", "bf16", "f16"]),
                     mode=rng.choice(["broadcast", "per_slot"]), routing=rng.choice(["uniform", "skew", "zipf"]))
        w = work(c)
        if w["bytes"] < 2.4e9 and w["flops"] < 0.9e12 and E * c["n_in"] * c["n_out"] < 256 * 2048 * 7168:
            return c


# --------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _pick(scores, k):
    """ids int32 [T][k] of the k largest scores of each row."""
    return torch.topk(scores, k, dim=-1).indices.to(torch.int32).contiguous()


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "route":
        T, E = case["T"], case["E"]
        # router logits of a trained layer: unit-scale rows over a mild preference per expert
        wide = (torch.randn(T, E + case["pad"], generator=g, device="cuda") * 1.5
                + torch.randn(E + case["pad"], generator=g, device="cuda") * 0.5).to(_DT[case["dtype"]])
        return dict(logits=wide[:, :E], bias=_randn(g, E, std=0.05) if case["bias"] else None)
    if op == "route_backward":
        T, E, k = case["T"], case["E"], case["k"]
        logits = _randn(g, T, E, dtype=_DT[case["dtype"]], std=1.5)
        noise = _randn(g, E, std=0.05)
        return dict(logits=logits, ids=_pick(logits.float() + noise, k), dweights=_randn(g, T, k))
    if op == "combine_backward":
        T, k, n = case["T"], case["k"], case["n"]
        w = torch.softmax(_randn(g, T, k), dim=-1)
        return dict(dy=_randn(g, T, n, std=0.1), dst=_randn(g, T, k, n), weights=w)
    if op == "quantize":
        # rows of unlike magnitude, as channels of a weight matrix or tokens have
        rows, n = case["rows"], case["n"]
        mag = torch.exp2(_randn(g, rows, 1) * 2.0)
        return dict(x=(_randn(g, rows, n) * mag * 0.05).to(_DT[case["dtype"]]))
    T, E, k, n_in, n_out = (case[a] for a in ("T", "E", "k", "n_in", "n_out"))
    rows = T if case["mode"] == "broadcast" else T * k
    if case["routing"] == "zipf":
        pop = -1.2 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        pop = pop[torch.randperm(E, generator=g, device="cuda")]
    elif case["routing"] == "skew":
        pop = _randn(g, E, std=0.5)
    else:
        pop = torch.zeros(E, device="cuda")
    gumbel = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)))
    # MXFP4 blocks: scale byte around 2^-7, then 16 bytes of codes
    blocks = torch.randint(0, 256, (E, n_out, n_in // 32, 17), generator=g, device="cuda", dtype=torch.uint8)
    blocks[..., 0] = torch.randint(117, 123, (E, n_out, n_in // 32), generator=g, device="cuda", dtype=torch.uint8)
    return dict(blocks=blocks, x=_randn(g, rows, n_in, dtype=_DT[case["dtype"]]), ids=_pick(pop + gumbel, k))


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import indirect_expert_matmul_b200 as moe
        op = case["op"]
        if op == "route":
            s["ids"] = torch.empty(case["T"], case["k"], dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty(case["T"], case["k"], device="cuda")
        elif op == "route_backward":
            s["out"] = torch.empty(case["T"], case["E"], dtype=_DT[case["dtype"]], device="cuda")
        elif op == "combine_backward":
            s["dw"] = torch.empty(case["T"], case["k"], device="cuda")
            s["dd"] = torch.empty_like(s["dst"]) if case["ddst"] else None
        elif op == "quantize":
            s["out"] = torch.empty(case["rows"], case["n"] // 32, 17, dtype=torch.uint8, device="cuda")
            s["values"] = torch.empty_like(s["x"])
        else:
            E, n_out, n_in = case["E"], case["n_out"], case["n_in"]
            s["W"] = moe.weights_prepare(s["blocks"], E, n_out, n_in, wtype="mxfp4")
            s["ws"] = moe.workspace(case["T"], case["k"], E, n_in, x_dtype=s["x"].dtype)
            s["out"] = torch.empty(case["T"], case["k"], n_out, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _scores(logits, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_route(s, c):
    # 64 bits: the choice depends on which of two close keys is larger
    p = _scores(s["logits"].double(), c["score"])
    key = p if s["bias"] is None else p + s["bias"].double()
    T, E, G = c["T"], c["E"], c["n_groups"]
    if G > 1:
        per = key.view(T, G, E // G)
        if c["group_score"] == "top2":
            gs = torch.sort(per, dim=-1, descending=True).values[..., :2].sum(-1)
        else:
            gs = per.amax(-1)
        chosen = torch.sort(gs, dim=-1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, chosen, True)
        key = torch.where(open_.repeat_interleave(E // G, 1), key, -math.inf)
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = p.gather(1, ids)
    if c["normalize"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _plain_route_backward(s, c):
    l, ids, g = s["logits"].float(), s["ids"].long(), s["dweights"] * c["scale"]
    p = _scores(l, c["score"])
    pc = p.gather(1, ids)
    if c["normalize"]:
        tot = pc.sum(-1, keepdim=True)
        q = pc / tot
        gp = (g - (g * q).sum(-1, keepdim=True)) / tot  # gradient of the chosen scores
    else:
        gp = g
    dp = torch.zeros_like(p).scatter_add_(1, ids, gp)
    if c["score"] == "sigmoid":
        dl = dp * p * (1.0 - p)
    else:
        dl = p * (dp - (dp * p).sum(-1, keepdim=True))
    return dl.to(s["logits"].dtype)


def _plain_combine_backward(s, c):
    dw = (s["dy"][:, None, :] * s["dst"]).sum(-1)
    if not c["ddst"]:
        return (dw,)
    return dw, s["weights"][:, :, None] * s["dy"][:, None, :]


def _scale_of(byte):
    """2^(byte - 127) as float32, from its bits (byte 0 is the subnormal 2^-127)."""
    b = byte.to(torch.int32)
    return torch.where(b == 0, 0x00400000, b << 23).view(torch.float32)


def _quantize(x):
    """(codes uint8 [..., 32], scale bytes) of blocks of 32 float32 values."""
    amax = x.abs().amax(-1)
    _, e = torch.frexp(amax)  # amax = m * 2^e, m in [1/2, 1): floor(log2 amax) = e - 1
    byte = torch.where(amax > 0, (e - 3 + 127).clamp(0, 254), 0).to(torch.uint8)
    r = (x / _scale_of(byte)[..., None]).abs()
    code = torch.signbit(x).to(torch.uint8) * 8
    # round to nearest on 0, .5, 1, 1.5, 2, 3, 4, 6; ties to the even code
    code += (r > 0.25).to(torch.uint8) + (r >= 0.75).to(torch.uint8) + (r > 1.25).to(torch.uint8)
    code += (r >= 1.75).to(torch.uint8) + (r > 2.5).to(torch.uint8) + (r >= 3.5).to(torch.uint8)
    code += (r > 5.0).to(torch.uint8)
    return code, byte


_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(code, byte):
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), device=code.device)
    return grid[code.long()] * _scale_of(byte)[..., None]


def _plain_quantize(s, c):
    x = s["x"].float().view(c["rows"], -1, 32)
    code, byte = _quantize(x)
    packed = code[..., :16] | (code[..., 16:] << 4)
    return torch.cat([byte[..., None], packed], -1), _values(code, byte).view(c["rows"], c["n"]).to(s["x"].dtype)


def _unpack(blocks):
    """(codes, scale bytes) of MXFP4 blocks [..., n/32, 17]."""
    q = blocks[..., 1:]
    return torch.cat([q & 15, q >> 4], -1), blocks[..., 0]


def _plain_product(s, c):
    x, ids, T, k = s["x"], s["ids"], c["T"], c["k"]
    xq = _values(*_quantize(x.float().view(x.shape[0], -1, 32))).view(x.shape[0], -1)
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=c["E"]).tolist()
    out = torch.empty(T * k, c["n_out"], device=x.device)
    p = 0
    for e, n in enumerate(counts):
        if n:
            slots = order[p:p + n]
            rows = slots // k if c["mode"] == "broadcast" else slots
            out[slots] = xq[rows] @ _values(*_unpack(s["blocks"][e])).view(c["n_out"], c["n_in"]).t()
            p += n
    return out.view(T, k, c["n_out"])


_PLAIN = dict(route=_plain_route, route_backward=_plain_route_backward, combine_backward=_plain_combine_backward,
              quantize=_plain_quantize, product=_plain_product)


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return _PLAIN[op](state, c)
    import indirect_expert_matmul_b200 as moe
    if op == "route":
        return moe.route_scored(state["logits"], c["k"], bias=state["bias"], score=c["score"],
                                n_groups=c["n_groups"], topk_groups=c["topk_groups"], group_score=c["group_score"],
                                normalize=c["normalize"], scale=c["scale"], ids=state["ids"],
                                weights=state["weights"])
    if op == "route_backward":
        return moe.route_scored_backward(state["logits"], state["ids"], state["dweights"], score=c["score"],
                                         normalize=c["normalize"], scale=c["scale"], out=state["out"])
    if op == "combine_backward":
        dw, dd = moe.combine_backward(state["dy"], state["dst"], state["weights"], need_ddst=c["ddst"],
                                      dweights=state["dw"], ddst=state["dd"])
        return (dw, dd) if c["ddst"] else (dw,)
    if op == "quantize":
        return moe.mxfp4_quantize(state["x"], out=state["out"], values=state["values"])
    return moe.mul_mat_id_mx4(state["W"], c["E"], c["n_out"], c["n_in"], state["x"], state["ids"], mode=c["mode"],
                              ws=state["ws"], out=state["out"])


# ----------------------------------------------------------------------- work
def work(case):
    """What one pass cannot do without: inputs read once, outputs written once."""
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return dict(bytes=T * E * _SZ[case["dtype"]] + (4 * E if case["bias"] else 0) + T * k * 8, flops=4 * T * E)
    if op == "route_backward":
        T, E, k, z = case["T"], case["E"], case["k"], _SZ[case["dtype"]]
        # only an unnormalised softmax needs the logits that were not chosen
        read = T * E * z if case["score"] == "softmax" and not case["normalize"] else T * k * z
        return dict(bytes=read + T * E * z + T * k * 8, flops=4 * read // z + 8 * T * k)
    if op == "combine_backward":
        T, k, n = case["T"], case["k"], case["n"]
        w = T * k * n * 4 + T * k * 4 if case["ddst"] else 0
        return dict(bytes=T * k * n * 4 + T * n * 4 + T * k * 4 + w, flops=(3 if case["ddst"] else 2) * T * k * n)
    if op == "quantize":
        m = case["rows"] * case["n"]
        return dict(bytes=2 * m * _SZ[case["dtype"]] + m // 32 * 17, flops=3 * m)
    T, E, k, n_in, n_out = (case[a] for a in ("T", "E", "k", "n_in", "n_out"))
    touched = E * (1.0 - (1.0 - k / E) ** T)  # experts that receive a slot, for a uniform choice
    rows = T if case["mode"] == "broadcast" else T * k
    return dict(bytes=int(touched * n_out * (n_in // 32) * 17) + rows * n_in * _SZ[case["dtype"]] + T * k * 4
                + T * k * n_out * 4, flops=2 * T * k * n_in * n_out)


# ---------------------------------------------------------------------- exact
def _exact_route(s, c):
    l = s["logits"].double().cpu().numpy()
    if c["score"] == "sigmoid":
        p = np.exp(-np.logaddexp(0.0, -l))
    else:
        m = l.max(1, keepdims=True)
        p = np.exp(l - m - np.log(np.exp(l - m).sum(1, keepdims=True)))
    key = p if s["bias"] is None else p + s["bias"].double().cpu().numpy()
    T, E, G = c["T"], c["E"], c["n_groups"]
    size = E // G
    if G > 1:
        ordered = np.sort(key.reshape(T, G, size), axis=2)
        gs = ordered[:, :, -1] + (ordered[:, :, -2] if c["group_score"] == "top2" else 0.0)
        # rank of a group: the groups that beat it, by score and then by index
        ahead = (gs[:, :, None] < gs[:, None, :]) | (
            (gs[:, :, None] == gs[:, None, :]) & (np.arange(G)[None, :, None] > np.arange(G)[None, None, :]))
        shut = ahead.sum(2) >= c["topk_groups"]
        key = np.where(np.repeat(shut, size, axis=1), -np.inf, key)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :c["k"]]
    w = np.take_along_axis(p, ids, 1)
    if c["normalize"]:
        w = w / w.sum(1, keepdims=True)
    return torch.from_numpy(ids.astype(np.int32)), torch.from_numpy(w * c["scale"])


def _exact_route_backward(s, c):
    # d(weight i)/d(logit j) written out for the slots of each token
    l, ids = s["logits"].double(), s["ids"].long()
    g = s["dweights"].double()
    lc = l.gather(1, ids)
    out = torch.zeros_like(l)
    if c["score"] == "sigmoid":
        p = torch.sigmoid(lc)
        slope = 1.0 - p  # d log p / d logit
        w = p / p.sum(1, keepdim=True) if c["normalize"] else p
        dlog = g * w
        if c["normalize"]:
            dlog = dlog - w * dlog.sum(1, keepdim=True)
        return out.scatter_add_(1, ids, c["scale"] * dlog * slope)
    if c["normalize"]:
        w = torch.softmax(lc, 1)
        return out.scatter_add_(1, ids, c["scale"] * w * (g - (g * w).sum(1, keepdim=True)))
    w = torch.exp(lc - torch.logsumexp(l, 1, keepdim=True))
    out.scatter_add_(1, ids, g * w)
    return c["scale"] * (out - torch.softmax(l, 1) * (g * w).sum(1, keepdim=True))


def _exact_combine_backward(s, c):
    dy, dst = s["dy"].double(), s["dst"].double()
    dw = torch.einsum("tkn,tn->tk", dst, dy)
    return (dw, torch.einsum("tk,tn->tkn", s["weights"].double(), dy)) if c["ddst"] else (dw,)


def _exact_round(x):
    """Nearest E2M1 multiples of the block scale (64-bit values), codes and scale exponents."""
    amax = x.abs().amax(-1, keepdim=True)
    ex = torch.floor(torch.log2(amax.clamp_min(2.0 ** -200)))
    ex = ex + (torch.exp2(ex + 1) <= amax).double() - (torch.exp2(ex) > amax).double()
    ex = torch.where(amax > 0, (ex - 2).clamp(-127, 127), -127.0)
    scale = torch.exp2(ex)
    r = x.abs() / scale
    # spacing of the grid around r: 1/2 below 2, 1 from 2 to 4, 2 above; torch.round takes ties to even
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))
    r = (torch.round(r / step) * step).clamp_max(6.0)
    return torch.copysign(r, x), scale, ex


def _exact_quantize(s, c):
    x = s["x"].double().view(c["rows"], -1, 32)
    r, scale, ex = _exact_round(x)
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    code = torch.bucketize(r.abs(), grid).to(torch.int32) + 8 * torch.signbit(r).to(torch.int32)
    packed = code[..., :16] + 16 * code[..., 16:]
    return torch.cat([(ex + 127).to(torch.int32), packed], -1).to(torch.uint8), (r * scale).view(c["rows"], c["n"])


def _exact_product(s, c):
    x = s["x"].double().view(s["x"].shape[0], -1, 32)
    r, scale, _ = _exact_round(x)
    xq = (r * scale).view(x.shape[0], -1)
    del x, r
    T, k = c["T"], c["k"]
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), dtype=torch.float64, device=xq.device)
    out = torch.zeros(T, k, c["n_out"], dtype=torch.float64, device=xq.device)
    for e in range(c["E"]):
        t, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        b = s["blocks"][e].int()
        w = torch.empty(c["n_out"], c["n_in"] // 32, 32, dtype=torch.float64, device=xq.device)
        w[..., :16] = grid[b[..., 1:] % 16]
        w[..., 16:] = grid[b[..., 1:] // 16]
        w *= torch.exp2(b[..., :1].double() - 127)
        out[t, slot] = xq[t if c["mode"] == "broadcast" else t * k + slot] @ w.view(c["n_out"], -1).t()
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    return dict(route=_exact_route, route_backward=_exact_route_backward, combine_backward=_exact_combine_backward,
                quantize=_exact_quantize, product=_exact_product)[case["op"]](s, case)
