"""The mixture-of-experts operators as measured: routing, token dispatch and
combine, and the grouped MX product with its epilogue, each forward and
backward.

With ``own`` false, ``run`` computes an operator from elementary torch
operations in 32 bits; with ``own`` true it calls the package's entry point.
Both take the state ``prepare`` made.  ``exact`` computes the same outputs in
64 bits from the definitions, apart from the plain forms.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32
NEG = float("-inf")
GATED = {"swiglu": "silu", "geglu": "gelu"}


# --------------------------------------------------------------- the cases

def listed():
    return [
        # routing of one decode step of a small batch
        {"name": "route_decode", "op": "route", "tokens": 7, "experts": 64, "k": 6, "score": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "renormalize": True, "scale": 1.0, "dtype": "bf16", "pad": 0.0},
        # routing of a long prefill: sigmoid scores, balance bias, 4 of 8 groups, float router logits
        {"name": "route_prefill", "op": "route", "tokens": 32768, "experts": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "renormalize": True, "scale": 2.5, "dtype": "f32", "pad": 0.0},
        # a training step's router gradient, an odd token count, some tokens padding
        {"name": "route_grad", "op": "route_grad", "tokens": 16385, "experts": 128, "k": 4, "score": "softmax",
         "bias": False, "groups": 1, "topk_groups": 1, "renormalize": False, "scale": 1.0, "dtype": "bf16",
         "pad": 0.03},
        # decode: a small batch's tokens into expert order as MXFP8
        {"name": "dispatch_decode", "op": "dispatch", "tokens": 33, "experts": 64, "k": 6, "hidden": 7168,
         "out": "e4m3", "dtype": "bf16", "pad": 0.0},
        # prefill: the MoE layer's hidden width, eight experts a token
        {"name": "dispatch_prefill", "op": "dispatch", "tokens": 8192, "experts": 32, "k": 8, "hidden": 7168,
         "out": "e4m3", "dtype": "bf16", "pad": 0.0},
        # prefill: the experts' outputs back to the tokens, onto the residual stream
        {"name": "combine_prefill", "op": "combine", "tokens": 8192, "k": 8, "hidden": 7168, "dtype": "bf16",
         "residual": True, "pad": 0.0},
        # training: the combine's gradients, odd sizes, some slots dropped
        {"name": "combine_grad", "op": "combine_grad", "tokens": 4099, "k": 6, "hidden": 4097, "dtype": "bf16",
         "residual": False, "pad": 0.05},
        # decode: one token's eight experts, gate and up products
        {"name": "ffn_token", "op": "product", "rows": 8, "experts": 32, "k": 7168, "n": 2048, "act": "swiglu",
         "bias": False, "residual": False, "keep_z": False, "b_fmt": "e2m1", "dtype": "bf16"},
        # decode of a batch: the down product with bias and residual
        {"name": "ffn_batch", "op": "product", "rows": 192, "experts": 32, "k": 2048, "n": 7168, "act": "none",
         "bias": True, "residual": True, "keep_z": False, "b_fmt": "e2m1", "dtype": "bf16"},
        # the MoE layer's training forward: gate and up products, pre-activation kept
        {"name": "ffn_train", "op": "product", "rows": 32768, "experts": 8, "k": 7168, "n": 2048, "act": "swiglu",
         "bias": True, "residual": False, "keep_z": True, "b_fmt": "e2m1", "dtype": "bf16"},
        # one shared expert, ragged rows and columns
        {"name": "ffn_ragged", "op": "product", "rows": 4099, "experts": 1, "k": 4096, "n": 4095, "act": "gelu",
         "bias": True, "residual": True, "keep_z": False, "b_fmt": "e2m1", "dtype": "bf16"},
        # the MoE layer's training backward through the activation, with the bias gradient
        {"name": "act_grad", "op": "act_grad", "rows": 32768, "experts": 8, "n": 2048, "act": "swiglu",
         "bias": True, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "dispatch", "combine", "combine_grad", "product", "product", "product",
                     "act_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    pad = rng.choice([0.0, 0.0, 0.04])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * max(2, _log_int(rng, 4, 512) // groups)
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(12, experts // groups * topk_groups))
        return {"op": op, "tokens": _log_int(rng, 1, 32768), "experts": experts, "k": k,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "topk_groups": topk_groups, "renormalize": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5]),
                "dtype": dtype, "pad": pad}
    if op in ("dispatch", "combine", "combine_grad"):
        k = rng.randint(1, 8)
        hidden = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            hidden = max(32, hidden // 32 * 32)
        tokens = min(_log_int(rng, 1, 16384), (8192 * 8 * 7168) // (2 * k * hidden))
        if op == "dispatch":
            return {"op": op, "tokens": tokens, "experts": max(k, _log_int(rng, 4, 256)), "k": k, "hidden": hidden,
                    "out": rng.choice(["e4m3", "e4m3", "same"]), "dtype": dtype, "pad": pad}
        return {"op": op, "tokens": tokens, "k": k, "hidden": hidden, "dtype": dtype,
                "residual": op == "combine" and rng.random() < 0.5, "pad": pad}
    act = rng.choice(["none", "relu", "silu", "gelu", "swiglu", "swiglu", "geglu"])
    experts = _log_int(rng, 1, 32)
    if op == "act_grad":
        return {"op": op, "rows": _log_int(rng, 1, 32768), "experts": experts, "n": _log_int(rng, 32, 2048),
                "act": act if act != "none" else "silu", "bias": rng.random() < 0.5, "dtype": dtype}
    k = 32 * _log_int(rng, 4, 224)
    n = _log_int(rng, 32, 4096)
    if rng.random() < 0.6:
        n = max(32, n // 32 * 32)
    return {"op": op, "rows": _log_int(rng, 1, 16384), "experts": experts, "k": k, "n": n, "act": act,
            "bias": rng.random() < 0.5, "residual": rng.random() < 0.4, "keep_z": rng.random() < 0.3,
            "b_fmt": rng.choice(["e2m1", "e2m1", "e2m1", "e4m3"]), "dtype": "bf16"}


def work(case):
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    op = c["op"]
    if op in ("route", "route_grad"):
        t, e, k = c["tokens"], c["experts"], c["k"]
        if op == "route":
            return {"bytes": t * e * es + t * k * 8 + (4 * e if c["bias"] else 0), "flops": 4 * t * e}
        # renormalised weights or sigmoid scores depend on the chosen logits alone
        dense = c["score"] == "softmax" and not c["renormalize"]
        return {"bytes": t * e * es + (t * e if dense else t * k) * es + t * k * 8, "flops": 6 * t * (e if dense else k)}
    if op == "dispatch":
        t, k, h = c["tokens"], c["k"], c["hidden"]
        out = t * k * (h * es if c["out"] == "same" else h + -(-h // BLOCK))
        return {"bytes": t * h * es + out + 8 * t * k + 8 * c["experts"], "flops": 3 * t * h}
    if op in ("combine", "combine_grad"):
        t, k, h = c["tokens"], c["k"], c["hidden"]
        rows = t * k * h * es
        if op == "combine":
            return {"bytes": rows + t * h * es * (2 if c["residual"] else 1) + 8 * t * k, "flops": 2 * t * k * h}
        return {"bytes": 2 * rows + t * h * es + 12 * t * k, "flops": 3 * t * k * h}
    gated = c["act"] in GATED
    n, i = (2 * c["n"], c["n"]) if gated else (c["n"], c["n"])
    m = c["rows"]
    if op == "act_grad":
        return {"bytes": m * es * (2 * n + i) + (4 * n * c["experts"] if c["bias"] else 0), "flops": 10 * m * n}
    k, busy = c["k"], min(c["experts"], m)
    b = n * (k // 2 if c["b_fmt"] == "e2m1" else k) + n * (k // BLOCK)
    return {"bytes": m * (k + k // BLOCK) + busy * b + m * i * es * (2 if c["residual"] else 1)
            + (m * n * es if c["keep_z"] else 0) + (4 * n * busy if c["bias"] else 0), "flops": 2 * m * n * k}


# --------------------------------------------------------------- inputs

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _mxfp8(x):
    """MXFP8 E4M3 of the last dimension's blocks of 32: (codes, E8M0 bytes)."""
    h = x.shape[-1]
    nb = -(-h // BLOCK)
    xb = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - h)).unflatten(-1, (nb, BLOCK))
    e8 = ((xb.abs().amax(-1).view(torch.int32) >> 23) - 8).clamp(min=0)
    q = (xb * ((254 - e8) << 23).view(torch.float32).unsqueeze(-1)).clamp(-448.0, 448.0)
    q = q.flatten(-2)[..., :h].to(torch.float8_e4m3fn)
    return q.contiguous().view(torch.uint8), e8.to(torch.uint8)


def _mxfp4(w):
    """Packed E2M1 nibbles and E8M0 bytes of the last dimension's blocks of 32."""
    wb = w.unflatten(-1, (-1, BLOCK))
    e8 = ((wb.abs().amax(-1).view(torch.int32) >> 23) - 2).clamp(min=0)
    a = wb * ((254 - e8) << 23).view(torch.float32).unsqueeze(-1)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = (torch.bucketize(a.abs(), mids, out_int32=True) + 8 * (a < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), e8.to(torch.uint8)


def _undecided(logits, bias, case):
    """Tokens whose choice 32-bit scores do not settle: two of the values that
    decide it are closer than rounding, but not equal."""
    l = logits.double()
    s = torch.softmax(l, -1) if case["score"] == "softmax" else torch.sigmoid(l)
    v = s + bias.double() if bias is not None else s
    near = 4e-6 * v.abs().amax(-1, keepdim=True)
    bad = torch.zeros(v.shape[0], dtype=torch.bool, device=DEV)
    if case["groups"] > 1:
        gv = v.unflatten(-1, (case["groups"], -1)).topk(min(2, v.shape[-1] // case["groups"]), -1).values.sum(-1)
        order = gv.sort(-1, descending=True)
        if case["topk_groups"] < case["groups"]:
            at = case["topk_groups"]
            gap = order.values[:, at - 1] - order.values[:, at]
            bad |= (gap > 0) & (gap < 2 * near[:, 0])
        keep = torch.zeros_like(gv, dtype=torch.bool).scatter_(-1, order.indices[:, :case["topk_groups"]], True)
        v = v.masked_fill(~keep.repeat_interleave(v.shape[-1] // case["groups"], -1), NEG)
    top = v.topk(min(case["k"] + 1, v.shape[-1]), -1).values
    gap = top[:, :-1] - top[:, 1:]
    return bad | ((gap > 0) & (gap < near)).any(-1)


def _logits(g, case):
    t, e, dt = case["tokens"], case["experts"], _type(case)
    bias = 0.1 * _randn(g, e) if case["bias"] else None
    logits = (1.5 * _randn(g, t, e)).to(dt)
    if bias is not None or case["groups"] > 1:
        for _ in range(20):
            at = _undecided(logits, bias, case).nonzero()[:, 0]
            if not at.numel():
                break
            logits[at] = (1.5 * _randn(g, at.numel(), e)).to(dt)
    if case["pad"] > 0:  # padding tokens: no expert may take them
        logits[torch.rand(t, generator=g, device=DEV) < case["pad"]] = NEG
    return logits, bias


def _ids(g, tokens, experts, k, pad):
    """k distinct experts a token, some of them more popular; padding tokens -1."""
    v = _randn(g, tokens, experts) + 0.5 * _randn(g, experts)
    ids = v.topk(k, -1).indices.to(torch.int32)
    if pad > 0:
        ids[torch.rand(tokens, generator=g, device=DEV) < pad] = -1
    return ids.contiguous()


def _counts(g, rows, experts):
    """Rows an expert: one each of distinct experts for few rows, a skewed split for many."""
    if rows <= experts:
        hit = torch.randperm(experts, generator=g, device=DEV)[:rows]
        return torch.zeros(experts, dtype=torch.int64, device=DEV).index_fill_(0, hit, 1)
    p = torch.softmax(0.3 * _randn(g, experts), -1)
    ends = (p.double().cumsum(0) / p.double().sum() * rows).round().long()
    ends[-1] = rows
    return torch.diff(ends, prepend=ends.new_zeros(1))


def prepare(case, seed):
    g, op, dt = _gen(seed), case["op"], _type(case)
    st = dict(case)
    if op in ("route", "route_grad"):
        st["logits"], st["bias_t"] = _logits(g, case)
        t, e, k = case["tokens"], case["experts"], case["k"]
        st["weights"] = torch.empty(t, k, device=DEV)
        st["ids"] = torch.empty(t, k, dtype=torch.int32, device=DEV)
        if op == "route_grad":
            st["ids"] = _route(st)["ids"]
            st["grad_weights"] = _randn(g, t, k)
            st["grad_logits"] = torch.empty(t, e, dtype=dt, device=DEV)
        return st
    if op in ("dispatch", "combine", "combine_grad"):
        t, k, h = case["tokens"], case["k"], case["hidden"]
        e = case.get("experts", 64 if k <= 64 else k)
        ids = _ids(g, t, e, k, case["pad"])
        st["ids"] = ids
        if op == "dispatch":
            st["x"] = _randn(g, t, h).to(dt)
            st["group_list"] = torch.empty(e, dtype=torch.int64, device=DEV)
            st["slot_rows"] = torch.empty(t, k, dtype=torch.int32, device=DEV)
            # rows past the dispatched ones are not written
            if case["out"] == "same":
                st["y"] = torch.zeros(t * k, h, dtype=dt, device=DEV)
            else:
                st["q"] = torch.zeros(t * k, h, dtype=torch.uint8, device=DEV)
                st["scales"] = torch.zeros(t * k, -(-h // BLOCK), dtype=torch.uint8, device=DEV)
            return st
        st["slot_rows"] = _plan(ids, e)[1]
        st["h"] = _randn(g, t * k, h).to(dt)
        w = torch.rand(t, k, generator=g, device=DEV) + 0.05
        st["weights"] = w / w.sum(-1, keepdim=True)
        if op == "combine":
            st["res"] = _randn(g, t, h).to(dt) if case["residual"] else None
            st["y"] = torch.empty(t, h, dtype=dt, device=DEV)
        else:
            st["grad_y"] = _randn(g, t, h).to(dt)
            st["grad_h"] = torch.zeros(t * k, h, dtype=dt, device=DEV)
            st["grad_weights"] = torch.empty(t, k, device=DEV)
        return st
    m, e = case["rows"], case["experts"]
    n, i = (2 * case["n"], case["n"]) if case["act"] in GATED else (case["n"], case["n"])
    st["group_list"] = _counts(g, m, e)
    if op == "act_grad":
        st["z"] = (1.2 * _randn(g, m, n)).to(dt)
        st["grad_c"] = _randn(g, m, i).to(dt)
        st["grad_z"] = torch.empty(m, n, dtype=dt, device=DEV)
        st["grad_bias"] = torch.empty(e, n, device=DEV) if case["bias"] else None
        return st
    k = case["k"]
    st["a"], st["a_scales"] = _mxfp8(_randn(g, m, k).to(torch.bfloat16))
    kb = k // 2 if case["b_fmt"] == "e2m1" else k
    st["b"] = torch.empty(e, n, kb, dtype=torch.uint8, device=DEV)
    st["b_scales"] = torch.empty(e, n, k // BLOCK, dtype=torch.uint8, device=DEV)
    for j in range(e):
        w = (_randn(g, n, k) * k ** -0.5).to(torch.bfloat16)
        st["b"][j], st["b_scales"][j] = _mxfp4(w.float()) if case["b_fmt"] == "e2m1" else _mxfp8(w)
    st["bias_t"] = 0.2 * _randn(g, e, n) if case["bias"] else None
    st["res"] = _randn(g, m, i).to(dt) if case["residual"] else None
    st["c"] = torch.empty(m, i, dtype=dt, device=DEV)
    st["z"] = torch.empty(m, n, dtype=dt, device=DEV) if case["keep_z"] else None
    # the largest group, which the plain product pads every group to
    st["capacity"] = int(st["group_list"].max())
    return st


# --------------------------------------------------------------- one pass

def run(st):
    op = st["op"]
    if own:
        return _own(st)
    if op == "route":
        return _route(st)
    if op == "route_grad":
        return _route_grad(st)
    if op == "dispatch":
        return _dispatch(st)
    if op == "combine":
        return _combine(st)
    if op == "combine_grad":
        return _combine_grad(st)
    if op == "product":
        return _product(st)
    return _act_grad(st)


def _own(st):
    import mxfp4_fake_quantization_amd as M
    op = st["op"]
    if op == "route":
        M.mxfp4_moe_route(st["logits"], st["weights"], st["ids"], bias=st["bias_t"], score=st["score"],
                          num_groups=st["groups"], topk_groups=st["topk_groups"], renormalize=st["renormalize"],
                          scale=st["scale"])
        return {"weights": st["weights"], "ids": st["ids"]}
    if op == "route_grad":
        M.mxfp4_moe_route_bwd(st["grad_weights"], st["logits"], st["ids"], st["grad_logits"], score=st["score"],
                              renormalize=st["renormalize"], scale=st["scale"])
        return {"grad_logits": st["grad_logits"]}
    if op == "dispatch":
        M.mxfp4_moe_plan(st["ids"], st["group_list"], st["slot_rows"])
        out = {"group_list": st["group_list"], "slot_rows": st["slot_rows"]}
        if st["out"] == "same":
            M.mxfp4_moe_dispatch(st["x"], st["slot_rows"], y=st["y"])
            return {**out, "y": st["y"]}
        M.mxfp4_moe_dispatch(st["x"], st["slot_rows"], q=st["q"], scales=st["scales"], fmt="e4m3")
        return {**out, **_values(st["q"], st["scales"])}
    if op == "combine":
        M.mxfp4_moe_combine(st["h"], st["slot_rows"], st["y"], weights=st["weights"], residual=st["res"])
        return {"y": st["y"]}
    if op == "combine_grad":
        M.mxfp4_moe_combine_bwd(st["grad_y"], st["h"], st["slot_rows"], st["weights"], st["grad_h"],
                                st["grad_weights"])
        return {"grad_h": st["grad_h"], "grad_weights": st["grad_weights"]}
    if op == "product":
        M.mxfp4_grouped_matmul_act(st["a"], st["a_scales"], st["b"], st["b_scales"], st["c"],
                                   group_list=st["group_list"], act=st["act"], bias=st["bias_t"],
                                   residual=st["res"], z=st["z"], a_fmt="e4m3", b_fmt=st["b_fmt"])
        return {"c": st["c"], "z": st["z"]}
    M.mxfp4_act_bwd(st["grad_c"], st["z"], st["grad_z"], act=st["act"], grad_bias=st["grad_bias"],
                    group_list=st["group_list"])
    return {"grad_z": st["grad_z"], "grad_bias": st["grad_bias"]}


def _values(q, scales):
    """The codes and block scales as the numbers they hold."""
    return {"q": q.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


# --------------------------------------------------------------- plain forms

def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(-1, keepdim=True)
    ex = torch.exp(l - torch.where(top == NEG, 0.0, top))
    total = ex.sum(-1, keepdim=True)
    return ex / torch.where(total == 0, 1.0, total)


def _route(st):
    l = st["logits"].float()
    s = _scores(l, st["score"])
    if st["bias_t"] is None and st["groups"] == 1:
        v = l
    else:
        v = s if st["bias_t"] is None else s + st["bias_t"]
        v = torch.where(l > NEG, v, NEG)
    if st["groups"] > 1:
        two = v.unflatten(-1, (st["groups"], -1)).sort(-1, descending=True).values[..., :2]
        gv = torch.where(two[..., 0] > NEG, torch.where(two > NEG, two, 0.0).sum(-1), NEG)
        best = gv.sort(dim=-1, descending=True, stable=True).indices[..., :st["topk_groups"]]
        keep = torch.zeros_like(gv, dtype=torch.bool).scatter_(-1, best, True)
        v = torch.where(keep.repeat_interleave(v.shape[-1] // st["groups"], -1), v, NEG)
    order = v.sort(dim=-1, descending=True, stable=True)
    at, live = order.indices[:, :st["k"]], order.values[:, :st["k"]] > NEG
    w = torch.where(live, s.gather(-1, at), 0.0)
    if st["renormalize"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    return {"weights": w * st["scale"], "ids": torch.where(live, at, -1).to(torch.int32)}


def _route_grad(st):
    l, ids = st["logits"].float(), st["ids"].long()
    live, at = ids >= 0, ids.clamp(min=0)
    s = _scores(l, st["score"])
    p = torch.where(live, s.gather(-1, at), 0.0)
    d = torch.where(live, st["grad_weights"], 0.0) * st["scale"]
    if st["renormalize"]:
        total = p.sum(-1, keepdim=True)
        total = torch.where(total == 0, 1.0, total)
        d = (d - (d * p / total).sum(-1, keepdim=True)) / total
        d = torch.where(live, d, 0.0)
    if st["score"] == "sigmoid":
        g = torch.zeros_like(l).scatter_add_(-1, at, d * p * (1.0 - p))
    else:
        ds = torch.zeros_like(l).scatter_add_(-1, at, d)
        g = s * (ds - (d * p).sum(-1, keepdim=True))
    return {"grad_logits": g.to(st["logits"].dtype)}


def _plan(ids, experts):
    flat = ids.reshape(-1).long()
    e = torch.where(flat < 0, experts, flat)
    order = e.sort(stable=True, dim=0).indices
    rows = torch.empty_like(order)
    rows[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, e, torch.ones_like(e))
    return counts[:experts], torch.where(flat < 0, -1, rows).to(torch.int32).view(ids.shape)


def _to_rows(values, slot_rows):
    """values [T, ...] (one a token) or [T, k, ...] (one a slot) at their slots' rows; the others stay zero."""
    t, k = slot_rows.shape
    at = torch.where(slot_rows < 0, t * k, slot_rows).long().reshape(-1)
    out = torch.zeros(t * k + 1, values.shape[-1], dtype=values.dtype, device=values.device)
    if values.dim() == 2:
        values = values.unsqueeze(1).expand(t, k, -1)
    out[at] = values.reshape(t * k, -1)
    return out[:t * k]


def _dispatch(st):
    counts, slot_rows = _plan(st["ids"], st["experts"])
    out = {"group_list": counts, "slot_rows": slot_rows}
    if st["out"] == "same":
        return {**out, "y": _to_rows(st["x"], slot_rows)}
    q, scales = _mxfp8(st["x"])
    return {**out, **_values(_to_rows(q, slot_rows), _to_rows(scales, slot_rows))}


def _combine(st):
    rows = st["slot_rows"].long()
    live = (rows >= 0).unsqueeze(-1)
    hk = st["h"].float()[rows.clamp(min=0)]
    y = torch.where(live, st["weights"].unsqueeze(-1) * hk, 0.0).sum(1)
    if st["res"] is not None:
        y = y + st["res"].float()
    return {"y": y.to(st["h"].dtype)}


def _combine_grad(st):
    rows = st["slot_rows"].long()
    live = rows >= 0
    dy = st["grad_y"].float().unsqueeze(1)
    hk = st["h"].float()[rows.clamp(min=0)]
    gw = torch.where(live, (hk * dy).sum(-1), 0.0)
    gh = (st["weights"].unsqueeze(-1) * dy).to(st["h"].dtype)
    return {"grad_h": _to_rows(gh, st["slot_rows"]), "grad_weights": gw}


def _fp4_values(b, scales):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=b.device)
    table = torch.cat([table, -table])
    w = torch.stack([table[(b & 15).int()], table[(b >> 4).int()]], -1).flatten(-2)
    return (w.unflatten(-1, (-1, BLOCK)) * scales.view(torch.float8_e8m0fnu).float().unsqueeze(-1)).flatten(-2)


def _fp8_values(q, scales):
    v = q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, BLOCK))
    return (v * scales.view(torch.float8_e8m0fnu).float().unsqueeze(-1)).flatten(-2)


def _act(x, name):
    if name == "relu":
        return x.clamp(min=0.0)
    if name == "silu":
        return x / (1.0 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * 0.5 ** 0.5))
    return x


def _act_slope(x, name):
    if name == "relu":
        return (x > 0).to(x.dtype)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return s * (1.0 + x * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(x * 0.5 ** 0.5)) + x * torch.exp(-0.5 * x * x) * (2.0 * math.pi) ** -0.5
    return torch.ones_like(x)


def _row_groups(counts, rows):
    ends = counts.cumsum(0)
    at = torch.arange(rows, device=counts.device)
    g = torch.searchsorted(ends, at, right=True)
    return g, at - (ends - counts)[g]


def _product(st):
    m, e, cap = st["rows"], st["experts"], st["capacity"]
    a = _fp8_values(st["a"], st["a_scales"])
    g, place = _row_groups(st["group_list"], m)
    values = _fp4_values if st["b_fmt"] == "e2m1" else _fp8_values
    if m <= e:  # the rows' own experts
        z = (values(st["b"][g], st["b_scales"][g]) @ a.unsqueeze(-1)).squeeze(-1)
    else:       # every expert, its rows padded to the largest group
        w = values(st["b"], st["b_scales"])
        padded = torch.zeros(e * cap, a.shape[-1], device=a.device)
        padded[g * cap + place] = a
        z = torch.bmm(padded.view(e, cap, -1), w.transpose(1, 2)).view(e * cap, -1)[g * cap + place]
    if st["bias_t"] is not None:
        z = z + st["bias_t"][g]
    if st["act"] in GATED:
        gate, up = z.chunk(2, -1)
        c = _act(gate, GATED[st["act"]]) * up
    else:
        c = _act(z, st["act"])
    if st["res"] is not None:
        c = c + st["res"].float()
    dt = st["c"].dtype
    return {"c": c.to(dt), "z": z.to(dt) if st["keep_z"] else None}


def _act_grad(st):
    z, dc = st["z"].float(), st["grad_c"].float()
    if st["act"] in GATED:
        gate, up = z.chunk(2, -1)
        name = GATED[st["act"]]
        dz = torch.cat([dc * up * _act_slope(gate, name), dc * _act(gate, name)], -1)
    else:
        dz = dc * _act_slope(z, st["act"])
    gb = None
    if st["grad_bias"] is not None:
        g, _ = _row_groups(st["group_list"], st["rows"])
        member = (g == torch.arange(st["experts"], device=z.device).unsqueeze(-1)).float()
        gb = member @ dz
    return {"grad_z": dz.to(st["z"].dtype), "grad_bias": gb}


# --------------------------------------------------------------- 64 bits

def _bits_fp8(q):
    """E4M3 values from sign, exponent and mantissa bits."""
    q = q.long()
    e, m = (q >> 3) & 15, (q & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, torch.ldexp(1.0 + m / 8.0, e - 7))
    return torch.where(q >= 128, -v, v)


def _bits_fp4(b):
    c = torch.empty(*b.shape[:-1], 2 * b.shape[-1], dtype=torch.long, device=b.device)
    c[..., 0::2], c[..., 1::2] = b & 15, b >> 4
    m = c & 7
    v = torch.where(m < 2, 0.5 * m.double(), torch.ldexp(1.0 + 0.5 * (m & 1).double(), (m >> 1) - 1))
    return torch.where(c >= 8, -v, v)


def _times_scale(v, scales):
    two = torch.ldexp(torch.ones_like(scales, dtype=torch.float64), scales.long() - 127)
    return v * two.repeat_interleave(BLOCK, -1)


def _act64(x, name):
    """(value, slope) of an activation."""
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x)), (x > 0).double()
    if name == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * (1 - s)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-x / math.sqrt(2.0))
        return x * cdf, cdf + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    return x, torch.ones_like(x)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op in ("route", "route_grad"):
        l = st["logits"].double()
        dead = torch.isneginf(l)
        gone = dead.all(-1, keepdim=True)
        if case["score"] == "sigmoid":
            s = torch.sigmoid(l)
        else:
            s = torch.softmax(l.masked_fill(gone, 0.0), -1).masked_fill(gone, 0.0)
        if op == "route":
            v = s if st["bias_t"] is None else s + st["bias_t"].double()
            if st["bias_t"] is None and case["groups"] == 1:
                v = l
            v = v.masked_fill(dead, NEG)
            if case["groups"] > 1:
                t, size = v.shape[0], v.shape[1] // case["groups"]
                gv = v.view(t, case["groups"], size).topk(min(2, size), -1).values.sum(-1)
                out = gv.sort(dim=-1, descending=True, stable=True).indices[:, case["topk_groups"]:]
                dropped = torch.zeros_like(gv).scatter_(1, out, 1.0) > 0
                v = v.view(t, case["groups"], size).masked_fill(dropped.unsqueeze(-1), NEG).view(t, -1)
            ids = v.sort(dim=-1, descending=True, stable=True).indices[:, :case["k"]]
            none = torch.isneginf(v.gather(-1, ids))
            w = s.gather(-1, ids).masked_fill(none, 0.0)
            if case["renormalize"]:
                w = torch.nan_to_num(w / w.sum(-1, keepdim=True), nan=0.0)
            return {"weights": w * case["scale"], "ids": ids.masked_fill(none, -1).to(torch.int32)}
        # the gradient through autograd in 64 bits
        x = l.masked_fill(gone, 0.0).requires_grad_(True)
        s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, -1)
        live = st["ids"] >= 0
        w = s.gather(-1, st["ids"].long().clamp(min=0)) * live
        if case["renormalize"]:
            w = w / w.sum(-1, keepdim=True).masked_fill(~live.any(-1, keepdim=True), 1.0)
        (w * st["grad_weights"].double() * live * case["scale"]).sum().backward()
        return {"grad_logits": x.grad.masked_fill(gone, 0.0)}
    if op in ("dispatch", "combine", "combine_grad"):
        t, k, h = case["tokens"], case["k"], case["hidden"]
        if op == "dispatch":
            flat = st["ids"].reshape(-1)
            rows = torch.full_like(flat, -1)
            at, counts = 0, []
            for e in range(case["experts"]):
                mine = (flat == e).nonzero()[:, 0]
                rows[mine] = torch.arange(at, at + mine.numel(), device=DEV, dtype=rows.dtype)
                at += mine.numel()
                counts.append(mine.numel())
            out = {"group_list": torch.tensor(counts), "slot_rows": rows.view(t, k)}
            if case["out"] == "same":
                y = torch.zeros(t * k, h, dtype=torch.float64, device=DEV)
                live = (rows >= 0).nonzero()[:, 0]
                y[rows[live].long()] = st["x"].double()[live // k]
                return {**out, "y": y}
            return {**out, "q": None, "scales": None}
        rows = st["slot_rows"].long()
        if op == "combine":
            y = torch.zeros(t, h, dtype=torch.float64, device=DEV) if st["res"] is None else st["res"].double()
            for j in range(k):
                live = rows[:, j] >= 0
                part = st["h"][rows[:, j].clamp(min=0)].double() * st["weights"][:, j:j + 1].double()
                y += part.masked_fill(~live.unsqueeze(-1), 0.0)
            return {"y": y}
        gh = torch.zeros(t * k, h, dtype=torch.float64, device=DEV)
        gw = torch.zeros(t, k, dtype=torch.float64, device=DEV)
        for j in range(k):
            live = (rows[:, j] >= 0).nonzero()[:, 0]
            dy = st["grad_y"][live].double()
            gh[rows[live, j]] = dy * st["weights"][live, j:j + 1].double()
            gw[live, j] = torch.linalg.vecdot(dy, st["h"][rows[live, j]].double())
        return {"grad_h": gh, "grad_weights": gw}
    gated = case["act"] in GATED
    name = GATED.get(case["act"], case["act"])
    counts = st["group_list"].tolist()
    if op == "act_grad":
        z, dc, n = st["z"].double(), st["grad_c"].double(), case["n"]
        if gated:
            f, slope = _act64(z[:, :n], name)
            dz = torch.cat([dc * slope * z[:, n:], dc * f], -1)
        else:
            dz = dc * _act64(z, name)[1]
        gb = torch.stack([p.sum(0) for p in dz.split(counts)]) if case["bias"] else None
        return {"grad_z": dz, "grad_bias": gb}
    at, zs = 0, []
    for e, count in enumerate(counts):
        if not count:
            continue
        a = _times_scale(_bits_fp8(st["a"][at:at + count]), st["a_scales"][at:at + count])
        b = _bits_fp4(st["b"][e]) if case["b_fmt"] == "e2m1" else _bits_fp8(st["b"][e])
        z = torch.mm(a, _times_scale(b, st["b_scales"][e]).t())
        zs.append(z if st["bias_t"] is None else z + st["bias_t"][e].double())
        at += count
    z = torch.cat(zs)
    c = _act64(z[:, :case["n"]], name)[0] * z[:, case["n"]:] if gated else _act64(z, name)[0]
    if st["res"] is not None:
        c = c + st["res"].double()
    return {"c": c, "z": z if case["keep_z"] else None}
