"""A W4A8 mixture-of-experts feed-forward layer on the library's calls.

Every token goes to k of E experts, each two products around an activation
(usually gated): weights in MXFP4 along the reduction dimension, activations
in MXFP8, group by group in one launch.  The README of the amct PR describes
the recipe (quantize w1 / w2 and the permuted inputs before the grouped
product), the hyper-parallel page's FakeW4A8GroupedLinear the three products
of a training step.

- ``MoESpec``: routing (score, groups, renormalisation, scale) and activation.
- ``PackedExperts``: weights quantized once, for serving:
      experts = PackedExperts(w1, w2, MoESpec(k=8)); y = experts(x, logits, residual=x)
- ``moe_ffn``: the same layer from float weights, with gradients for x, the
  router's logits, both weights and both biases, for quantization-aware
  training (the weights' and activations' quantization is passed straight
  through, the products of the backward pass are quantized as the page does:
  each operand along the dimension that its product sums).
- ``MoELayer``: ``moe_ffn`` with its parameters and a router, as a module.

x is [tokens, hidden] bfloat16; w1 [E, 2 I or I, hidden] (gate rows, then up
rows), w2 [E, hidden, I]; biases float32 [E, rows of the weight].  hidden and I
are multiples of 32.  A token whose logits are all -inf goes to no expert.
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import torch
import torch.nn.functional as F
from torch import nn
from torch.autograd.function import once_differentiable

from . import (ACTIVATIONS, GROUP_K, kmajor_k_blocks, mxfp4_act_bwd, mxfp4_grouped_matmul, mxfp4_grouped_matmul_act,
               mxfp4_moe_combine, mxfp4_moe_combine_bwd, mxfp4_moe_dispatch, mxfp4_moe_plan, mxfp4_moe_route,
               mxfp4_moe_route_bwd, mxfp4_quant_pack, mxfp4_quant_pack_kmajor, mxfp8_kmajor_k_blocks, mxfp8_quant,
               mxfp8_quant_kmajor)

__all__ = ["MoESpec", "PackedExperts", "MoELayer", "moe_ffn"]


@dataclasses.dataclass(frozen=True)
class MoESpec:
    """Routing of each token to ``k`` experts (see mxfp4_moe_route) and the
    experts' activation (a name of ACTIVATIONS)."""

    k: int = 2
    score: str = "softmax"
    num_groups: int = 1
    topk_groups: Optional[int] = None
    renormalize: bool = True
    scale: float = 1.0
    act: str = "swiglu"

    def __post_init__(self):
        if self.act not in ACTIVATIONS:
            raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {self.act!r}")

    @property
    def gated(self) -> bool:
        return bool(ACTIVATIONS[self.act] & 4)


def _check_shapes(x, logits, w1, w2, spec):
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise ValueError("x must be a 2-D bfloat16 tensor [tokens, hidden]")
    experts, n1, hidden = w1.shape
    inner = n1 // 2 if spec.gated else n1
    if hidden % 32 or inner % 32 or n1 != inner * (2 if spec.gated else 1):
        raise ValueError(f"hidden {hidden} and the inner width {inner} must be multiples of 32")
    if tuple(w2.shape) != (experts, hidden, inner):
        raise ValueError(f"w2 must be [{experts}, {hidden}, {inner}], got {list(w2.shape)}")
    if x.shape[1] != hidden or tuple(logits.shape) != (x.shape[0], experts):
        raise ValueError(f"x must be [tokens, {hidden}] and logits [tokens, {experts}]")


def _pack(w):
    """MXFP4 of the last dimension's blocks: codes and scales of w's rank."""
    w = w.contiguous()
    codes = torch.empty(*w.shape[:-1], w.shape[-1] // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(*w.shape[:-1], w.shape[-1] // 32, dtype=torch.uint8, device=w.device)
    mxfp4_quant_pack(w, codes, scales)
    return codes, scales


def _pack_t(w):
    """MXFP4 of w [E, rows, cols] along its rows, K-major: [cols, E * rows]
    codes and scales, and the strides of an expert in them."""
    e, rows, cols = w.shape
    kb = kmajor_k_blocks(e * rows, 32)
    codes = torch.empty(cols, kb * 16, dtype=torch.uint8, device=w.device)
    scales = torch.empty(cols, kb, dtype=torch.uint8, device=w.device)
    mxfp4_quant_pack_kmajor(w.contiguous().view(e * rows, cols), codes, scales)
    return codes, scales, (rows // 2, rows // 32)


def _mxfp8(x):
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    s = torch.empty(x.shape[0], x.shape[1] // 32, dtype=torch.uint8, device=x.device)
    mxfp8_quant(x, q, s)
    return q, s


def _mxfp8_t(x, group_list):
    """MXFP8 down each group's rows, K-major: the operand of a product over them."""
    kb = mxfp8_kmajor_k_blocks(x.shape[0], group_list.numel())
    q = torch.empty(x.shape[1], kb * 32, dtype=torch.uint8, device=x.device)
    s = torch.empty(x.shape[1], kb, dtype=torch.uint8, device=x.device)
    mxfp8_quant_kmajor(x, q, s, group_list=group_list)
    return q, s


def _route(logits, spec, balance):
    tokens, experts = logits.shape
    weights = torch.empty(tokens, spec.k, dtype=torch.float32, device=logits.device)
    ids = torch.empty(tokens, spec.k, dtype=torch.int32, device=logits.device)
    mxfp4_moe_route(logits, weights, ids, bias=balance, score=spec.score, num_groups=spec.num_groups,
                    topk_groups=spec.topk_groups, renormalize=spec.renormalize, scale=spec.scale)
    group_list = torch.empty(experts, dtype=torch.int64, device=logits.device)
    rows = torch.empty_like(ids)
    mxfp4_moe_plan(ids, group_list, rows)
    return weights, ids, group_list, rows


def _ffn(x, rows, group_list, p1, p2, b1, b2, spec, z=None, y=None):
    """The experts' two products on the dispatched rows: (activation, output)."""
    n, hidden = rows.numel(), x.shape[1]
    q = torch.empty(n, hidden, dtype=torch.uint8, device=x.device)
    s = torch.empty(n, hidden // 32, dtype=torch.uint8, device=x.device)
    mxfp4_moe_dispatch(x, rows, y=y, q=q, scales=s)
    inner = p1[0].shape[1] // (2 if spec.gated else 1)
    a = torch.empty(n, inner, dtype=x.dtype, device=x.device)
    mxfp4_grouped_matmul_act(q, s, *p1, a, group_list=group_list, act=spec.act, bias=b1, z=z)
    h = torch.empty(n, hidden, dtype=x.dtype, device=x.device)
    mxfp4_grouped_matmul_act(*_mxfp8(a), *p2, h, group_list=group_list, bias=b2)
    return a, h


class PackedExperts:
    """Experts with their weights quantized once.  Calling it takes x [tokens,
    hidden] and the router's logits [tokens, E], from one token to any number;
    ``balance`` is the router's selection bias, ``residual`` is added to the
    result (which may be written over it with ``out``)."""

    def __init__(self, w1, w2, spec: MoESpec = MoESpec(), b1=None, b2=None):
        self.spec = spec
        _check_shapes(w1.new_empty(0, w1.shape[-1], dtype=torch.bfloat16), w1.new_empty(0, w1.shape[0]), w1, w2, spec)
        self.w1, self.w2 = _pack(w1), _pack(w2)
        # copies, as the packed weights are: all of one state
        self.b1, self.b2 = (None if b is None else b.detach().clone() for b in (b1, b2))

    @torch.no_grad()
    def __call__(self, x, logits, residual=None, balance=None, out=None):
        if x.dim() != 2 or x.dtype != torch.bfloat16 or x.shape[1] != self.w2[0].shape[1]:
            raise ValueError(f"x must be a bfloat16 tensor [tokens, {self.w2[0].shape[1]}]")
        if tuple(logits.shape) != (x.shape[0], self.w1[0].shape[0]):
            raise ValueError(f"logits must be [{x.shape[0]}, {self.w1[0].shape[0]}], got {list(logits.shape)}")
        weights, _, group_list, rows = _route(logits, self.spec, balance)
        _, h = _ffn(x, rows, group_list, self.w1, self.w2, self.b1, self.b2, self.spec)
        y = torch.empty_like(x) if out is None else out
        mxfp4_moe_combine(h, rows, y, weights=weights, residual=residual)
        return y


class _MoEFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, logits, w1, w2, b1, b2, balance, spec: MoESpec):
        _check_shapes(x, logits, w1, w2, spec)
        x, logits = x.contiguous(), logits.contiguous()
        weights, ids, group_list, rows = _route(logits, spec, balance)
        n = rows.numel()
        xr = torch.empty(n, x.shape[1], dtype=x.dtype, device=x.device)
        z = torch.empty(n, w1.shape[1], dtype=x.dtype, device=x.device)
        a, h = _ffn(x, rows, group_list, _pack(w1), _pack(w2), b1, b2, spec, z=z, y=xr)
        y = torch.empty_like(x)
        mxfp4_moe_combine(h, rows, y, weights=weights)
        ctx.spec = spec
        ctx.save_for_backward(logits, w1, w2, b1, b2, weights, ids, group_list, rows, xr, z, a, h)
        return y

    @staticmethod
    @once_differentiable  # raw buffers below: a second derivative would lack this layer's part
    def backward(ctx, dy):
        spec = ctx.spec
        logits, w1, w2, b1, b2, weights, ids, group_list, rows, xr, z, a, h = ctx.saved_tensors
        need_x, need_l, need_w1, need_w2, need_b1, need_b2 = ctx.needs_input_grad[:6]
        experts, n = group_list.numel(), rows.numel()
        dy = dy.contiguous()
        dh = torch.empty_like(h)
        dweights = torch.empty_like(weights) if need_l else None
        mxfp4_moe_combine_bwd(dy, h, rows, weights, dh, dweights)
        dlogits = None
        if need_l:
            dlogits = torch.empty_like(logits)
            mxfp4_moe_route_bwd(dweights, logits, ids, dlogits, score=spec.score, renormalize=spec.renormalize,
                                scale=spec.scale)
        db1 = torch.empty(experts, w1.shape[1], dtype=torch.float32, device=dy.device) if need_b1 else None
        db2 = torch.empty(experts, w2.shape[1], dtype=torch.float32, device=dy.device) if need_b2 else None
        if need_b2:
            mxfp4_act_bwd(dh, h, dh, act="none", grad_bias=db2, group_list=group_list)

        def product(g, w):
            """g W_e of every expert's rows: both quantized along g's columns."""
            codes, scales, stride = _pack_t(w)
            out = torch.empty(n, w.shape[2], dtype=g.dtype, device=g.device)
            mxfp4_grouped_matmul(*_mxfp8(g), codes, scales, out, K=g.shape[1], group_list=group_list,
                                 b_group_stride=stride)
            return out

        def weight_grad(g, v):
            """g_e^T v_e of every expert: both quantized down the expert's rows."""
            out = torch.empty(experts, g.shape[1], v.shape[1], dtype=g.dtype, device=g.device)
            mxfp4_grouped_matmul(*_mxfp8_t(g, group_list), *_mxfp8_t(v, group_list), out, K=n, group_list=group_list,
                                 group_type=GROUP_K, b_fmt="e4m3")
            return out

        dw2 = weight_grad(dh, a).to(w2.dtype) if need_w2 else None
        dx = dw1 = None
        if need_x or need_w1 or need_b1:
            da = product(dh, w2)
            dz = torch.empty_like(z)
            mxfp4_act_bwd(da, z, dz, act=spec.act, grad_bias=db1, group_list=group_list)
            if need_w1:
                dw1 = weight_grad(dz, xr).to(w1.dtype)
            if need_x:
                dx = torch.empty_like(dy)
                mxfp4_moe_combine(product(dz, w1), rows, dx)
        return dx, dlogits, dw1, dw2, db1, db2, None, None


def moe_ffn(x, logits, w1, w2, spec: MoESpec = MoESpec(), b1=None, b2=None, balance=None):
    """Differentiable mixture-of-experts feed-forward layer: y [tokens, hidden]
    (without a residual).  The selection bias ``balance`` has no gradient;
    second derivatives are refused."""
    return _MoEFFN.apply(x, logits, w1, w2, b1, b2, balance, spec)


class MoELayer(nn.Module):
    """Router, experts and residual: y = x + moe_ffn(x, x G^T)."""

    def __init__(self, hidden: int, inner: int, experts: int, spec: MoESpec = MoESpec(), bias: bool = False, *,
                 device=None, dtype=torch.bfloat16):
        super().__init__()
        self.spec = spec
        rows = inner * (2 if spec.gated else 1)
        self.router = nn.Linear(hidden, experts, bias=False, device=device, dtype=dtype)
        self.w1 = nn.Parameter(torch.empty(experts, rows, hidden, device=device, dtype=dtype))
        self.w2 = nn.Parameter(torch.empty(experts, hidden, inner, device=device, dtype=dtype))
        self.b1 = nn.Parameter(torch.zeros(experts, rows, device=device, dtype=torch.float32)) if bias else None
        self.b2 = nn.Parameter(torch.zeros(experts, hidden, device=device, dtype=torch.float32)) if bias else None
        nn.init.normal_(self.w1, std=hidden ** -0.5)
        nn.init.normal_(self.w2, std=inner ** -0.5)

    def forward(self, x):
        flat = x.reshape(-1, x.shape[-1])
        logits = F.linear(flat.to(self.router.weight.dtype), self.router.weight)
        y = moe_ffn(flat, logits, self.w1, self.w2, self.spec, *self._biases())
        return x + y.view(x.shape)

    def packed(self) -> PackedExperts:
        """The experts' present weights, quantized for serving."""
        return PackedExperts(self.w1.detach(), self.w2.detach(), self.spec, *self._biases())

    def _biases(self):
        """As the products take them, whatever type a cast of the module gave them."""
        return (None if b is None else b.float() for b in (self.b1, self.b2))

    def extra_repr(self) -> str:
        return f"experts={self.w1.shape[0]}, spec={self.spec}"
