"""Low-rank adapters beside a shared projection and the global gradient norm
with clipping, as measured: the adapters of many requests in one call, their
backward pass, the norm over many tensors, and the clipped gradients.

With ``own`` false, ``run`` computes an operator from elementary torch
operations in 32 bits (long sums in 64); with ``own`` true it calls the
package's entry point.  Both take the state ``prepare`` made.  ``exact``
computes the same outputs in 64 bits from the definitions, adapter by adapter.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of one request, a square projection
        {"name": "adapter_token", "op": "adapter", "tokens": 1, "requests": 1, "adapters": 8, "none": 0, "rank": 16,
         "in": 4096, "out": 4096, "base": True, "save": False, "slice": False, "dtype": "bf16"},
        # one decode step of a batch, nearly every request with an adapter of its own, the widest projection
        {"name": "adapter_decode", "op": "adapter", "tokens": 64, "requests": 64, "adapters": 48, "none": 4, "rank": 16,
         "in": 8192, "out": 28672, "base": True, "save": False, "slice": False, "dtype": "bf16"},
        # prompts' chunks of several requests, odd sizes, columns of a fused projection's output
        {"name": "adapter_mixed", "op": "adapter", "tokens": 1531, "requests": 37, "adapters": 24, "none": 3,
         "rank": 12, "in": 4095, "out": 4097, "base": True, "save": False, "slice": True, "dtype": "bf16"},
        # prefill of long prompts
        {"name": "adapter_prefill", "op": "adapter", "tokens": 8192, "requests": 16, "adapters": 16, "none": 0,
         "rank": 32, "in": 7168, "out": 7168, "base": True, "save": False, "slice": False, "dtype": "bf16"},
        # a training forward of one adapter in fp32, its inner values kept for the backward pass
        {"name": "adapter_f32", "op": "adapter", "tokens": 4096, "requests": 1, "adapters": 1, "none": 0, "rank": 8,
         "in": 4096, "out": 4096, "base": True, "save": True, "slice": False, "dtype": "f32"},
        # a training backward of one adapter
        {"name": "grad_one", "op": "adapter_grad", "tokens": 16384, "requests": 1, "adapters": 1, "none": 0,
         "rank": 16, "in": 4096, "out": 4096, "base": True, "dtype": "bf16"},
        # several adapters trained side by side, some sequences without one
        {"name": "grad_many", "op": "adapter_grad", "tokens": 8191, "requests": 12, "adapters": 4, "none": 2,
         "rank": 64, "in": 7168, "out": 2048, "base": True, "dtype": "bf16"},
        # a small fp32 training batch of odd sizes
        {"name": "grad_ragged", "op": "adapter_grad", "tokens": 333, "requests": 5, "adapters": 3, "none": 0,
         "rank": 5, "in": 1025, "out": 515, "base": False, "dtype": "f32"},
        # the gradients of a tiny QAT model: two 32 x 64 weights and two vectors
        {"name": "norm_tiny", "op": "norm", "tensors": 4, "kind": "model", "rank": 0, "in": 64, "out": 32, "p": "2",
         "packed": False, "dtype": "f32"},
        # the weight gradients of four layers' projections
        {"name": "norm_layers", "op": "norm", "tensors": 8, "kind": "model", "rank": 0, "in": 4096, "out": 7168,
         "p": "2", "packed": False, "dtype": "bf16"},
        # the gradients of a model's adapters: hundreds of small tensors
        {"name": "clip_adapters", "op": "clip", "tensors": 448, "kind": "adapters", "rank": 16, "in": 4096,
         "out": 4096, "p": "2", "packed": False, "max_norm": 1.0, "dtype": "f32"},
        # the gradients of large weights
        {"name": "clip_weights", "op": "clip", "tensors": 8, "kind": "model", "rank": 0, "in": 8192, "out": 28672,
         "p": "2", "packed": False, "max_norm": 1.0, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapter", "adapter", "adapter", "adapter_grad", "adapter_grad", "norm", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "clip"):
        kind = rng.choice(["model", "adapters"])
        n_in, n_out, rank = _log_int(rng, 32, 8192), _log_int(rng, 32, 8192), rng.choice([4, 8, 15, 16, 64])
        size = (n_in + 1) * n_out if kind == "model" else rank * (n_in + n_out)
        case = {"op": op, "tensors": min(_log_int(rng, 1, 700), 2 + 200_000_000 // size), "kind": kind, "rank": rank,
                "in": n_in, "out": n_out, "p": rng.choice(["2", "2", "2", "1", "inf"]),
                "packed": rng.random() < 0.4, "dtype": dtype}
        return case if op == "norm" else {**case, "max_norm": rng.choice([0.5, 1.0, 1e6])}
    rank = rng.choice([1, 4, 7, 8, 8, 16, 16, 16, 24, 32, 64, 64, 96, 128])
    n_in, n_out = _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
    if rng.random() < 0.6:
        n_in, n_out = max(32, n_in // 32 * 32), max(32, n_out // 32 * 32)
    tokens = min(_log_int(rng, 1, 8192), 8192 * 7168 // max(n_in, n_out))
    if dtype == "f32":
        tokens = max(1, min(tokens, 4096 * 4096 // max(n_in, n_out), 4096 * 4096 * 64 // ((n_in + n_out) * rank)))
    adapters = max(1, min(_log_int(rng, 1, 64 if op == "adapter" else 8), 512 // rank))
    requests = tokens if op == "adapter" and tokens <= 128 and rng.random() < 0.7 else min(tokens, _log_int(rng, 1, 40))
    case = {"op": op, "tokens": tokens, "requests": requests, "adapters": adapters,
            "none": rng.choice([0, 0, requests // 8]), "rank": rank, "in": n_in, "out": n_out,
            "base": rng.random() < 0.7, "dtype": dtype}
    if op == "adapter":
        case["save"], case["slice"] = rng.random() < 0.3, rng.random() < 0.3
    return case


def _sizes(case):
    """Elements of each tensor: weights and vectors by turns, or the two matrices of each adapter."""
    n, i, o, r = case["tensors"], case["in"], case["out"], case["rank"]
    two = (i * o, i) if case["kind"] == "model" else (r * i, o * r)
    return [two[j % 2] for j in range(n)]


def work(case):
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] in ("norm", "clip"):
        n = sum(_sizes(c))
        return {"bytes": n * es * (1 if c["op"] == "norm" else 2) + 4, "flops": 2 * n}
    t, r, i, o = c["tokens"], c["rank"], c["in"], c["out"]
    used = min(c["adapters"], c["requests"] - c["none"])
    weights = used * r * (i + o) * es
    if c["op"] == "adapter":
        return {"bytes": t * es * (i + o * (2 if c["base"] else 1)) + weights + 4 * t + (4 * t * r if c["save"] else 0),
                "flops": 2 * t * r * (i + o)}
    return {"bytes": t * es * (o + i * (3 if c["base"] else 2)) + weights + c["adapters"] * r * (i + o) * es
            + 4 * t + 4 * t * r, "flops": 4 * t * r * (i + o)}


# --------------------------------------------------------------- inputs

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _ids(g, case):
    """The adapter of every token: each request a run of tokens, `none` of the
    requests without an adapter, the others taking the adapters in turn."""
    t, n = case["tokens"], case["requests"]
    cuts = torch.randperm(t - 1, generator=g, device=DEV)[:n - 1] + 1 if n > 1 else torch.empty(0, device=DEV).long()
    starts = torch.zeros(t, dtype=torch.int64, device=DEV)
    starts[cuts] = 1
    of = torch.arange(n, device=DEV) - case["none"]
    of = torch.where(of < 0, -1, of % case["adapters"])[torch.randperm(n, generator=g, device=DEV)]
    return of[starts.cumsum(0)].to(torch.int32)


def prepare(case, seed):
    g, op, dt = torch.Generator(device=DEV), case["op"], _type(case)
    g.manual_seed(seed)
    st = dict(case)
    if op in ("norm", "clip"):
        # tensors one after the other in a flat buffer, as gradient buckets hold them: end to end (packed), or each
        # from a boundary of 64 elements.  Layers differ in the size of their gradients.
        sizes, at, places = _sizes(case), 0, []
        for n in sizes:
            places.append((at, n))
            at += n if case["packed"] else -(-n // 64) * 64
        st["flat"] = torch.zeros(at, dtype=dt, device=DEV)
        level = torch.exp(1.2 * _randn(g, len(sizes)) - 7.0).tolist()
        for (p, n), s in zip(places, level):
            st["flat"][p:p + n] = (s * _randn(g, n)).to(dt)
        st["grads"] = [st["flat"][p:p + n] for p, n in places]
        st["norm"] = torch.empty(1, device=DEV)
        if op == "clip":
            # a gradient above the bound, as clipping meets it (unless the bound is out of reach)
            st["flat"] *= 40.0
            st["flat_out"] = torch.zeros_like(st["flat"])
            st["outs"] = [st["flat_out"][p:p + n] for p, n in places]
        return st
    t, r, i, o, n = case["tokens"], case["rank"], case["in"], case["out"], case["adapters"]
    st["ids"] = _ids(g, case)
    st["x"] = _randn(g, t, i).to(dt)
    st["a"] = (i ** -0.5 * _randn(g, n, r, i)).to(dt)
    st["b"] = (0.05 * _randn(g, n, o, r)).to(dt)
    st["scale"] = 0.5 + 1.5 * torch.rand(n, generator=g, device=DEV)
    if op == "adapter":
        wide = 2 * o if case["slice"] else o          # the columns after another projection's
        st["base_t"] = _randn(g, t, wide).to(dt)[:, wide - o:] if case["base"] else None
        st["y"] = torch.empty(t, wide, dtype=dt, device=DEV)[:, wide - o:]
        st["u"] = torch.empty(t, r, device=DEV) if case["save"] else None
        return st
    st["base_t"] = _randn(g, t, i).to(dt) if case["base"] else None
    st["grad_y"] = _randn(g, t, o).to(dt)
    u = st["x"].float() @ st["a"].float().view(n * r, i).t()
    at = st["ids"].long().clamp(min=0).view(t, 1, 1).expand(t, 1, r)
    st["u"] = torch.where(st["ids"].view(t, 1) >= 0, u.view(t, n, r).gather(1, at).squeeze(1), 0.0)
    st["grad_x"] = torch.empty(t, i, dtype=dt, device=DEV)
    st["grad_a"], st["grad_b"] = torch.empty_like(st["a"]), torch.empty_like(st["b"])
    return st


# --------------------------------------------------------------- one pass

def run(st):
    op = st["op"]
    if own:
        return _own(st)
    if op == "adapter":
        return _adapter(st)
    if op == "adapter_grad":
        return _adapter_grad(st)
    norm = _norm(st)
    if op == "norm":
        return {"norm": norm}
    coef = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": norm, "out": (st["flat"].float() * coef).to(st["flat"].dtype)}


def _own(st):
    import mxfp4_fake_quantization_amd as M
    op = st["op"]
    if op == "adapter":
        M.mxfp4_adapter_fwd(st["x"], st["a"], st["b"], st["y"], ids=st["ids"], scale=st["scale"], base=st["base_t"],
                            u=st["u"])
        return {"y": st["y"], "u": st["u"]}
    if op == "adapter_grad":
        M.mxfp4_adapter_bwd(st["grad_y"], st["a"], st["b"], x=st["x"], u=st["u"], ids=st["ids"], scale=st["scale"],
                            grad_x=st["grad_x"], grad_a=st["grad_a"], grad_b=st["grad_b"], base=st["base_t"])
        return {"grad_x": st["grad_x"], "grad_a": st["grad_a"], "grad_b": st["grad_b"]}
    if op == "norm":
        M.mxfp4_grad_norm(st["grads"], st["norm"], norm_type=float(st["p"]))
        return {"norm": st["norm"]}
    M.mxfp4_grad_clip(st["grads"], st["max_norm"], st["norm"], outs=st["outs"], norm_type=float(st["p"]))
    return {"norm": st["norm"], "out": st["flat_out"]}


# --------------------------------------------------------------- plain forms
#
# All adapters' columns side by side, those of other adapters masked out.

def _own_columns(st):
    n, r = st["adapters"], st["rank"]
    of = torch.arange(n, device=DEV).repeat_interleave(r)
    mine = st["ids"].unsqueeze(-1) == of
    a = st["a"].float().view(n * r, -1)
    b = st["b"].float().permute(1, 0, 2).reshape(-1, n * r).contiguous()
    return mine, a, b, st["scale"].repeat_interleave(r)


def _adapter(st):
    mine, a, b, scale = _own_columns(st)
    u = torch.where(mine, st["x"].float() @ a.t(), 0.0)
    y = (u * scale) @ b.t()
    if st["base_t"] is not None:
        y = st["base_t"].float() + y
    kept = u.view(-1, st["adapters"], st["rank"]).sum(1) if st["save"] else None
    return {"y": y.to(st["x"].dtype), "u": kept}


def _adapter_grad(st):
    mine, a, b, scale = _own_columns(st)
    gy, dt = st["grad_y"].float(), st["grad_y"].dtype
    n, r = st["adapters"], st["rank"]
    du = torch.where(mine, (gy @ b) * scale, 0.0)
    gx = du @ a
    if st["base_t"] is not None:
        gx = st["base_t"].float() + gx
    ga = du.t() @ st["x"].float()
    u = torch.where(mine, st["u"].repeat(1, n) * scale, 0.0)
    gb = (u.t() @ gy).view(n, r, -1).transpose(1, 2)
    return {"grad_x": gx.to(dt), "grad_a": ga.view_as(st["a"]).to(dt), "grad_b": gb.contiguous().to(dt)}


def _norm(st):
    v = st["flat"].float().abs()
    if st["p"] == "inf":
        return v.max().view(1)
    if st["p"] == "1":
        return v.sum(dtype=torch.float64).float().view(1)
    return v.square().sum(dtype=torch.float64).sqrt().float().view(1)


# --------------------------------------------------------------- 64 bits

def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op in ("norm", "clip"):
        p = float(case["p"])
        per = torch.stack([torch.linalg.vector_norm(v, ord=p, dtype=torch.float64) for v in st["grads"]])
        norm = torch.linalg.vector_norm(per, ord=p).view(1)
        if op == "norm":
            return {"norm": norm}
        return {"norm": norm, "out": st["flat"].double() * torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0)}
    x, s = st["x"].double(), st["scale"].double()
    ids = st["ids"].long()
    rows = [(ids == j).nonzero()[:, 0] for j in range(case["adapters"])]
    if op == "adapter":
        y = torch.zeros(case["tokens"], case["out"], dtype=torch.float64, device=DEV)
        if case["base"]:
            y += st["base_t"].double()
        u = torch.zeros(case["tokens"], case["rank"], dtype=torch.float64, device=DEV)
        for j, at in enumerate(rows):
            if at.numel():
                u[at] = torch.mm(x[at], st["a"][j].double().t())
                y[at] += s[j] * torch.mm(u[at], st["b"][j].double().t())
        return {"y": y, "u": u if case["save"] else None}
    gy = st["grad_y"].double()
    gx = st["base_t"].double() if case["base"] else torch.zeros_like(x)
    ga, gb = st["a"].double() * 0.0, st["b"].double() * 0.0
    for j, at in enumerate(rows):
        if at.numel():
            du = s[j] * torch.mm(gy[at], st["b"][j].double())
            gx[at] += torch.mm(du, st["a"][j].double())
            ga[j] = torch.mm(du.t(), x[at])
            gb[j] = s[j] * torch.mm(gy[at].t(), st["u"][at].double())
    return {"grad_x": gx, "grad_a": ga, "grad_b": gb}
