"""Adapters beside quantized projections on the GPU, as they are used: serving,
training and clipping together.

adapter_add is checked against autograd in 64 bits on the same (rounded) values, within
the bounds of test_gpu_adapter.  PackedLinear's product is W4A8: against the float layer,
weight and input are off by about 0.1 and 0.03 of their norms, independently: 0.2 of the
result's norm, for its gradient likewise (a wrong operand is off by 1 or more)."""
import pytest
import torch
from torch import nn

import test_gpu_adapter as ta

pytestmark = pytest.mark.gpu
AD = Q = M = None
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    global AD, Q, M
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_fake_quantization_amd as mod
    from mxfp4_fake_quantization_amd import adapters, qat
    mod._load()
    AD, Q, M = adapters, qat, mod
    ta.M = mod
    yield


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [(6, 96, 160, 4, 3), (300, 200, 130, 16, 4)], ids=str)
def test_adapter_add(size, dt):
    p = ta.Problem(*size, "mixed", dt)
    leaves = [t.clone().requires_grad_() for t in (p.x, p.base, p.a, p.b)]
    y = AD.adapter_add(*leaves, p.ids, p.scale)
    want, bound, wu, _ = p.forward64(True, True)
    ta.within(y.detach(), want, bound)
    y.backward(p.gy)
    u = torch.empty(size[0], size[3], device="cuda")
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, torch.empty_like(p.base), ids=p.ids, u=u)
    refs = p.backward64(u, True, False)
    for leaf, k in zip((leaves[0], leaves[2], leaves[3]), ("grad_x", "grad_a", "grad_b")):
        ta.within(leaf.grad, *refs[k])
    assert torch.equal(leaves[1].grad, p.gy)


def test_shapes_types_and_wanted_gradients():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(3, 7, 64, generator=g, device="cuda").to(bf16)
    layer = AD.AdapterLinear(nn.Linear(64, 96, device="cuda", dtype=bf16), adapters=2, rank=8, dtype=f32)
    nn.init.normal_(layer.adapters.b, std=0.3)
    ids = torch.randint(-1, 2, (3, 7), generator=g, device="cuda", dtype=torch.int32)
    y = layer(x, ids)
    assert y.shape == (3, 7, 96) and y.dtype == bf16
    y.float().sum().backward()
    assert layer.adapters.a.grad.dtype == f32 and layer.base.weight.grad is not None
    flat = layer(x.reshape(-1, 64), ids.reshape(-1))
    assert torch.equal(flat.view_as(y), y)
    # transposed leading dimensions (the same base: nn.Linear rounds a transposed input's
    # product differently, by another library kernel)
    base = layer.base(x)
    yt = layer.adapters(x.transpose(0, 1), base.transpose(0, 1), ids.t())
    assert torch.equal(yt, y.transpose(0, 1))
    # frozen parts get no gradient, and cost none
    layer.zero_grad(set_to_none=True)
    layer.base.requires_grad_(False)
    layer.adapters.a.requires_grad_(False)
    layer(x, ids).float().sum().backward()
    assert layer.adapters.a.grad is None and layer.base.weight.grad is None and layer.adapters.b.grad is not None
    with torch.no_grad():
        assert torch.equal(layer(x, ids), y)
    # a fresh adapter adds nothing
    fresh = AD.AdapterLinear(layer.base, adapters=2, rank=8)
    assert torch.equal(fresh(x, ids), layer.base(x))


def test_second_derivative_is_refused():
    x = torch.randn(4, 32, device="cuda", requires_grad=True)
    base = torch.randn(4, 64, device="cuda", requires_grad=True)
    a, b = (torch.randn(1, 2, 32, device="cuda", requires_grad=True), torch.randn(1, 64, 2, device="cuda", requires_grad=True))
    (gx,) = torch.autograd.grad(AD.adapter_add(x, base, a, b).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()


def test_packed_linear():
    torch.manual_seed(2)
    linear = nn.Linear(256, 320, device="cuda", dtype=bf16)
    packed = AD.PackedLinear.pack(linear, backward=True)
    for shape in ((1, 256), (3, 50, 256), (700, 256), (0, 256)):
        x = torch.randn(*shape, device="cuda").to(bf16).requires_grad_()
        xf = x.detach().clone().requires_grad_()
        y, yf = packed(x), linear(xf)
        assert y.shape == yf.shape
        gy = torch.randn_like(yf)
        y.backward(gy)
        yf.backward(gy)
        for got, want in ((y.detach(), yf.detach()), (x.grad, xf.grad)):
            assert got.shape == want.shape
            if want.numel():
                assert float((got.float() - want.float()).norm() / want.float().norm()) < 0.2
    with pytest.raises(RuntimeError, match="backward=True"):
        x = torch.randn(2, 256, device="cuda").to(bf16).requires_grad_()
        AD.PackedLinear.pack(linear)(x).sum().backward()


@pytest.mark.parametrize("tokens", [5, 333])
def test_training_step_together(tokens):
    """Frozen MXFP4 projections, adapters of three tasks, one clipped step: forward, all
    gradients, the norm over them and the scaled gradients, against the same in torch on
    the layers' own outputs."""
    torch.manual_seed(tokens)
    first = AD.AdapterLinear(AD.PackedLinear.pack(nn.Linear(128, 192, device="cuda", dtype=bf16), backward=True),
                             adapters=3, rank=8)
    second = AD.AdapterLinear(AD.PackedLinear.pack(nn.Linear(192, 64, bias=False, device="cuda", dtype=bf16), backward=True),
                              adapters=3, rank=16, alpha=8.0)
    for layer in (first, second):
        nn.init.normal_(layer.adapters.b, std=0.2)
    params = [*first.parameters(), *second.parameters()]
    assert len(params) == 4
    x = torch.randn(tokens, 128, device="cuda").to(bf16)
    ids = torch.randint(-1, 3, (tokens,), device="cuda", dtype=torch.int32)
    h = torch.nn.functional.silu(first(x, ids))
    second(h, ids).float().square().sum().backward()
    # the second layer's adapter gradients by their formula
    gy = 2 * second(h.detach(), ids).detach().float()
    live = (ids >= 0).nonzero()[:, 0]
    gb = torch.zeros_like(second.adapters.b, dtype=torch.float64)
    for t in live.tolist():
        i = int(ids[t])
        u = second.adapters.a[i].double() @ h[t].detach().double()
        gb[i] += float(second.adapters.scale[i]) * torch.outer(gy[t].to(bf16).double(), u)
    got = second.adapters.b.grad.double()
    # grad_b: its bf16 rounding, gy's (2^-8) and fp32 sums: 2^-6 of the norm is above them
    assert float((got - gb).norm() / gb.norm()) < 2.0 ** -6
    grads = [p.grad.clone() for p in params]
    want = float(torch.cat([g.double().flatten() for g in grads]).norm())
    version = params[0].grad._version
    norm = Q.clip_grad_norm_(params, 0.25 * want)
    assert params[0].grad._version > version
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    coef = 0.25 * want / (want + 1e-6)
    for p, g in zip(params, grads):
        assert bool(((p.grad.double() - g.double() * coef).abs() <= g.double().abs() * coef * (2.0 ** -8 + 2.0 ** -22)
                     + 1e-38).all())


def test_clip_grad_norm():
    params = [nn.Parameter(torch.zeros(n, device="cuda", dtype=dt)) for n, dt in ((7, f32), (100, bf16), (3, f32))]
    params[0].grad = torch.full((7,), 3.0, device="cuda")
    params[1].grad = torch.full((100,), -4.0, device="cuda", dtype=bf16)
    assert params[2].grad is None
    want = (7 * 9 + 100 * 16) ** 0.5
    assert abs(float(Q.clip_grad_norm_(params, 1e9)) - want) <= 2.0 ** -23 * want
    assert float(params[0].grad[0]) == 3.0
    assert float(Q.clip_grad_norm_(params, 1.0, norm_type=float("inf"))) == 4.0
    assert abs(float(params[0].grad[0]) - 0.75) < 1e-6
    assert float(Q.clip_grad_norm_(params[2], 1.0)) == 0.0 and float(Q.clip_grad_norm_([], 1.0)) == 0.0
    params[1].grad[5] = float("nan")
    keep = params[0].grad.clone()
    with pytest.raises(RuntimeError, match="not finite"):
        Q.clip_grad_norm_(params, 1.0, error_if_nonfinite=True)
    assert torch.equal(params[0].grad, keep)


def test_serving_graph():
    """A decode step through two layers, captured and replayed with new tokens and other
    adapters, equals the eager call."""
    torch.manual_seed(9)
    layers = [AD.AdapterLinear(AD.PackedLinear.pack(nn.Linear(128, 128, device="cuda", dtype=bf16)), adapters=5, rank=8)
              for _ in range(2)]
    for layer in layers:
        nn.init.normal_(layer.adapters.b, std=0.3)
    x = torch.randn(24, 128, device="cuda").to(bf16)
    ids = torch.randint(-1, 5, (24,), device="cuda", dtype=torch.int32)

    def step():
        with torch.no_grad():
            return layers[1](layers[0](x, ids), ids)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for seed in range(3):
        torch.manual_seed(seed)
        x.copy_(torch.randn(24, 128, device="cuda"))
        ids.copy_(torch.randint(-1, 5, (24,), device="cuda"))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
