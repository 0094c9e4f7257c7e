"""Low-rank adapters beside quantized projections, on the library's calls.

A projection in MXFP4 stays as it is; what a task or a customer adds to it is
a pair of small matrices per adapter, y = W x + s B (A x).  One call serves the
tokens of many requests, each with its request's adapter, and training sums each
adapter's gradients over its own tokens.

- ``adapter_add``: the differentiable sum base + s (x A_i^T) B_i^T.
- ``Adapters``: a stack of adapters as a module.
- ``PackedLinear``: a projection whose MXFP4 weight is quantized once (W4A8, as
  PackedExperts does for experts); with ``backward`` it also passes gradients on to
  its input.
- ``AdapterLinear``: any projection (nn.Linear, QATLinear, PackedLinear) with
  adapters beside it:
      layer = AdapterLinear(PackedLinear.pack(linear, backward=True), adapters=4, rank=16)
      y = layer(x, ids)                       # ids int32: each token's adapter, -1 for none
      y.sum().backward()                      # gradients of x and the adapters
      clip_grad_norm_(layer.parameters(), 1.0)  # qat.clip_grad_norm_

x is [..., in] bfloat16 or float32 (PackedLinear: bfloat16; under autocast each takes x
in the projection's type), ids has x's leading shape.  Adapters kept in another type
than x's are rounded to x's for the call; their gradients, summed in float32, are
rounded to x's type once and then take the adapters' (as autocast's products do).
"""
from __future__ import annotations

import math
from typing import Optional

import torch
from torch import nn
from torch.autograd.function import once_differentiable

from . import mxfp4_adapter_bwd, mxfp4_adapter_fwd, mxfp4_grouped_matmul, mxfp4_grouped_matmul_act
from .moe import _mxfp8, _pack, _pack_t

__all__ = ["adapter_add", "Adapters", "PackedLinear", "AdapterLinear"]


def _rows(t):
    """t [..., n] as rows; a copy only where its elements are not contiguous in a row."""
    t = t.reshape(-1, t.shape[-1])
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        t = t.contiguous()
    return t


class _AdapterAdd(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, base, a, b, ids, scale):
        xr, br = _rows(x), _rows(base)
        a, b = a.contiguous(), b.contiguous()
        y = torch.empty(br.shape, dtype=base.dtype, device=base.device)
        u = None
        if ctx.needs_input_grad[3]:
            u = torch.empty(xr.shape[0], a.shape[1], dtype=torch.float32, device=x.device)
        mxfp4_adapter_fwd(xr, a, b, y, ids=ids, scale=scale, base=br, u=u)
        ctx.shape = x.shape
        ctx.save_for_backward(xr if ctx.needs_input_grad[2] else None, a, b, ids, scale, u)
        return y.view(base.shape)

    @staticmethod
    @once_differentiable  # raw buffers below: a second derivative would lack this layer's part
    def backward(ctx, gy):
        x, a, b, ids, scale, u = ctx.saved_tensors
        need_x, need_base, need_a, need_b = ctx.needs_input_grad[:4]
        gr = _rows(gy)
        gx = torch.empty(gr.shape[0], a.shape[2], dtype=gy.dtype, device=gy.device) if need_x else None
        ga = torch.empty_like(a) if need_a else None
        gb = torch.empty_like(b) if need_b else None
        if need_x or need_a or need_b:
            mxfp4_adapter_bwd(gr, a, b, x=x, u=u, ids=ids, scale=scale, grad_x=gx, grad_a=ga, grad_b=gb)
        return None if gx is None else gx.view(ctx.shape), gy if need_base else None, ga, gb, None, None


def adapter_add(x, base, a, b, ids: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None):
    """base + scale_i (x a_i^T) b_i^T with each token's adapter i = ids (int32,
    x's leading shape; None: adapter 0; outside [0, adapters): none).  base is
    [..., out] of x's type, a [adapters, rank, in], b [adapters, out, rank], scale
    float32 [adapters].  Gradients reach x, base, a and b (of up to 1024 adapters);
    second derivatives, and a scale that wants a gradient, are refused.  Under autocast
    x is taken in base's type."""
    if x.dim() < 1 or base.dim() != x.dim() or base.shape[:-1] != x.shape[:-1]:
        raise ValueError(f"base must have x's leading shape {list(x.shape[:-1])}, got {list(base.shape)}")
    if base.dtype != x.dtype and torch.is_autocast_enabled("cuda"):
        x = x.to(base.dtype)  # as the projection took it
    if base.dtype != x.dtype:
        raise ValueError(f"base must have x's type {x.dtype}, got {base.dtype}")
    if scale is not None and scale.requires_grad and torch.is_grad_enabled():
        raise ValueError("scale gets no gradient: detach it")
    if ids is not None:
        if ids.shape != x.shape[:-1]:
            raise ValueError(f"ids must be {list(x.shape[:-1])}, got {list(ids.shape)}")
        ids = ids.reshape(-1).contiguous()
    return _AdapterAdd.apply(x, base, a.to(x.dtype), b.to(x.dtype), ids, scale)


class _Float32Kept(nn.Module):
    """A module whose buffers named in ``_kept`` stay float32 when it is cast: the
    library takes them in float32."""

    _kept = ()

    def _apply(self, fn, recurse=True):
        before = {name: getattr(self, name) for name in self._kept}
        super()._apply(fn, recurse)
        for name, t in before.items():
            now = getattr(self, name)
            if now is not None and now.dtype != torch.float32:
                setattr(self, name, t.to(now.device, torch.float32))
        return self


class Adapters(_Float32Kept):
    """``adapters`` low-rank adapters of one projection.  A starts random, B at 0, so
    that a fresh adapter adds nothing; the scales alpha / rank are a buffer, float32
    through casts."""

    _kept = ("scale",)

    def __init__(self, in_features: int, out_features: int, adapters: int = 1, rank: int = 16,
                 alpha: Optional[float] = None, *, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.in_features, self.out_features, self.rank = in_features, out_features, rank
        self.a = nn.Parameter(torch.empty(adapters, rank, in_features, device=device, dtype=dtype))
        self.b = nn.Parameter(torch.zeros(adapters, out_features, rank, device=device, dtype=dtype))
        scale = (rank if alpha is None else alpha) / rank
        self.register_buffer("scale", torch.full((adapters,), float(scale), dtype=torch.float32,
                                                  device=device))
        nn.init.kaiming_uniform_(self.a.view(adapters * rank, in_features), a=math.sqrt(5))

    def forward(self, x, base, ids: Optional[torch.Tensor] = None):
        return adapter_add(x, base, self.a, self.b, ids, self.scale.float())

    def extra_repr(self) -> str:
        return f"{self.in_features}, {self.out_features}, adapters={self.a.shape[0]}, rank={self.rank}"


class _PackedProduct(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, layer):
        ctx.layer = layer
        return layer._product(x)

    @staticmethod
    @once_differentiable  # quantized products below: a second derivative would lack this layer's part
    def backward(ctx, gy):
        layer = ctx.layer
        if layer.transposed is None:
            raise RuntimeError("this PackedLinear was packed without backward=True")
        codes, scales = layer.transposed
        g = gy.reshape(-1, gy.shape[-1]).contiguous()
        gx = torch.empty(g.shape[0], layer.in_features, dtype=g.dtype, device=g.device)
        if g.shape[0]:
            mxfp4_grouped_matmul(*_mxfp8(g), codes, scales, gx, K=layer.out_features)
        return gx.view(*gy.shape[:-1], layer.in_features), None


class PackedLinear(_Float32Kept):
    """A linear layer with its weight in MXFP4 along the inputs, quantized once;
    inputs go through MXFP8 (W4A8).  The weight is not trained.  With ``backward``
    a second copy, quantized along the outputs, gives the gradient of the input as
    the mixture-of-experts layer does (gradients through MXFP8).  in and out features
    are multiples of 32; x is bfloat16.  The bias stays float32 through casts."""

    _kept = ("bias",)

    def __init__(self, weight, bias=None, backward: bool = False):
        super().__init__()
        out_features, in_features = weight.shape
        if in_features % 32 or out_features % 32:
            raise ValueError(f"in and out features must be multiples of 32, got {in_features} and {out_features}")
        self.in_features, self.out_features = in_features, out_features
        weight = weight.detach()
        codes, scales = _pack(weight)
        self.register_buffer("codes", codes)
        self.register_buffer("scales", scales)
        self.register_buffer("bias", None if bias is None else bias.detach().float().clone())
        t = _pack_t(weight.unsqueeze(0))[:2] if backward else (None, None)
        self.register_buffer("codes_t", t[0])
        self.register_buffer("scales_t", t[1])

    @classmethod
    def pack(cls, linear: nn.Linear, backward: bool = False) -> "PackedLinear":
        """``linear``'s present weight and bias, packed."""
        return cls(linear.weight, linear.bias, backward)

    @property
    def transposed(self):
        return None if self.codes_t is None else (self.codes_t, self.scales_t)

    def _product(self, x):
        rows = x.reshape(-1, self.in_features).contiguous()
        y = torch.empty(rows.shape[0], self.out_features, dtype=x.dtype, device=x.device)
        mxfp4_grouped_matmul_act(*_mxfp8(rows), self.codes, self.scales, y, bias=self.bias)
        return y.view(*x.shape[:-1], self.out_features)

    def forward(self, x):
        if torch.is_autocast_enabled("cuda") and torch.get_autocast_dtype("cuda") == torch.bfloat16:
            x = x.to(torch.bfloat16)  # as a projection in float does
        if x.dtype != torch.bfloat16 or x.shape[-1] != self.in_features:
            raise ValueError(f"x must be a bfloat16 tensor [..., {self.in_features}]")
        return _PackedProduct.apply(x, self)

    def extra_repr(self) -> str:
        return f"{self.in_features}, {self.out_features}, bias={self.bias is not None}, backward={self.codes_t is not None}"


class AdapterLinear(nn.Module):
    """A projection with adapters beside it: y = base(x) + s (x A_i^T) B_i^T.  The
    projection is left as it is (freeze its parameters to train the adapters alone)."""

    def __init__(self, base: nn.Module, adapters: int = 1, rank: int = 16, alpha: Optional[float] = None, *,
                 dtype=torch.bfloat16):
        super().__init__()
        at = next((t for t in (*base.parameters(), *base.buffers())), None)
        self.base = base
        self.adapters = Adapters(base.in_features, base.out_features, adapters, rank, alpha,
                                 device=None if at is None else at.device, dtype=dtype)

    def forward(self, x, ids: Optional[torch.Tensor] = None):
        return self.adapters(x, self.base(x), ids)
