"""The adapters' modules as programs hold them: cast to another type, built under another
default type, under autocast.  On the CPU what needs no kernel, on the GPU the rest."""
import pytest
import torch
from torch import nn

import mxfp4_fake_quantization_amd as M
from mxfp4_fake_quantization_amd import adapters as AD

bf16, f32 = torch.bfloat16, torch.float32
gpu = pytest.mark.gpu


@pytest.fixture
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M._load()


@gpu
@pytest.mark.parametrize("cast", ["bfloat16", "half", "double", "to"])
def test_packed_bias_through_casts(lib, cast):
    """The bias is the float32 one before and after a cast: the same bits."""
    torch.manual_seed(3)
    layer = AD.PackedLinear.pack(nn.Linear(64, 96, device="cuda", dtype=f32), backward=True)
    x = torch.randn(5, 64, device="cuda").to(bf16)
    want, bias = layer(x), layer.bias.clone()
    same = layer.to(bf16) if cast == "to" else getattr(layer, cast)()
    assert same is layer and layer.bias.dtype == f32 and torch.equal(layer.bias, bias)
    assert torch.equal(layer(x), want)
    layer.cpu().cuda()
    assert torch.equal(layer(x), want)
    no_bias = AD.PackedLinear.pack(nn.Linear(64, 96, bias=False, device="cuda")).to(bf16)
    assert no_bias.bias is None and no_bias(x).shape == (5, 96)


@pytest.mark.parametrize("cast", ["bfloat16", "half", "double", "to"])
def test_scale_through_casts(cast):
    """alpha / rank, 4 / 3 here, stays the float32 value."""
    layer = nn.Sequential(AD.Adapters(16, 24, adapters=3, rank=12, alpha=16.0, dtype=f32))
    layer.to(bf16) if cast == "to" else getattr(layer, cast)()
    scale = layer[0].scale
    assert scale.dtype == f32 and scale.tolist() == [torch.tensor(16 / 12, dtype=f32).item()] * 3
    assert layer[0].a.dtype == {"bfloat16": bf16, "to": bf16, "half": torch.float16, "double": torch.float64}[cast]
    assert dict(layer.named_buffers())["0.scale"] is scale and "0.scale" in layer.state_dict()


@pytest.fixture(params=[bf16, torch.float64], ids=["bf16", "f64"])
def default_type(request):
    """Another default type, as programs set it while they build a model."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    yield request.param
    torch.set_default_dtype(before)


def test_scale_under_a_default_type(default_type):
    scale = AD.Adapters(16, 24, adapters=2, rank=12, alpha=16.0).scale
    assert scale.dtype == f32 and scale.tolist() == [torch.tensor(16 / 12, dtype=f32).item()] * 2


def test_no_gradients_under_a_default_type(default_type):
    from mxfp4_fake_quantization_amd import qat
    norm = qat.clip_grad_norm_([nn.Parameter(torch.zeros(3))], 1.0)
    assert norm.dtype == f32 and float(norm) == 0.0


@gpu
def test_training_under_a_default_type(lib, default_type):
    """Gradients and clipping are what they are under float32, bit for bit."""
    from mxfp4_fake_quantization_amd import qat

    def step():
        torch.manual_seed(6)
        layer = AD.AdapterLinear(nn.Linear(64, 96, device="cuda", dtype=bf16), adapters=2, rank=12, alpha=16.0)
        nn.init.normal_(layer.adapters.b, std=0.3)
        x = torch.randn(9, 64, device="cuda", dtype=f32).to(bf16)
        layer(x, torch.arange(9, device="cuda", dtype=torch.int32) % 3 - 1).float().square().sum().backward()
        norm = qat.clip_grad_norm_(layer.parameters(), 0.5)
        assert norm.dtype == f32
        return [norm, *(p.grad for p in layer.parameters())]

    got = step()
    torch.set_default_dtype(f32)
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def projection(name, n_in, n_out, dtype):
    from mxfp4_fake_quantization_amd import qat
    torch.manual_seed(4)
    linear = nn.Linear(n_in, n_out, device="cuda", dtype=dtype)
    if name == "linear":
        return linear
    return AD.PackedLinear.pack(linear, backward=True) if name == "packed" else qat.QATLinear.wrap(linear, qat.QATPolicy.w4a4())


@gpu
@pytest.mark.parametrize("name", ["linear", "qat", "packed"])
def test_autocast(lib, name):
    """Under autocast a projection makes bfloat16 of a float32 input; the adapters beside it take the input so too:
    the bits and gradients of the call on the rounded input, the input's gradient in its type."""
    layer = AD.AdapterLinear(projection(name, 64, 96, f32), adapters=2, rank=8, dtype=f32)
    nn.init.normal_(layer.adapters.b, std=0.3)
    x = torch.randn(3, 7, 64, device="cuda", requires_grad=True)
    ids = (torch.arange(21, device="cuda", dtype=torch.int32) % 3 - 1).view(3, 7)
    adapters = list(layer.adapters.parameters())
    with torch.autocast("cuda", dtype=bf16):
        y = layer(x, ids)
    assert y.dtype == bf16
    gy = torch.randn(3, 7, 96, device="cuda").to(bf16)
    grads = torch.autograd.grad(y, [x, *adapters], gy)
    assert [g.dtype for g in grads] == [f32, f32, f32]
    # by hand: the projection under autocast, the adapters on the rounded input
    v = x.detach().requires_grad_()
    with torch.autocast("cuda", dtype=bf16):
        base = layer.base(v.to(bf16) if name == "packed" else v)
    want = layer.adapters(v.to(bf16), base, ids)
    assert torch.equal(y, want)
    for a, b in zip(grads, torch.autograd.grad(want, [v, *adapters], gy)):
        assert torch.equal(a, b)
    # mixed types outside autocast are still refused
    with pytest.raises(ValueError):
        layer.adapters(v, base, ids)


@gpu
@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
def test_beside_a_fake_quantized_projection(lib, dt):
    """QATLinear as the base: its output and gradients, and the adapters' beside them."""
    layer = AD.AdapterLinear(projection("qat", 64, 96, dt), adapters=3, rank=4, dtype=dt)
    x = torch.randn(11, 64, device="cuda").to(dt).requires_grad_()
    ids = torch.arange(11, device="cuda", dtype=torch.int32) % 3
    gy = torch.randn(11, 96, device="cuda").to(dt)
    gw, gx = torch.autograd.grad(layer.base(x), [layer.base.weight, x], gy)
    y = layer(x, ids)                               # B is 0: it adds nothing
    assert torch.equal(y, layer.base(x))
    got = torch.autograd.grad(y, [layer.base.weight, x, layer.adapters.b], gy)
    assert torch.equal(got[0], gw) and torch.equal(got[1], gx) and got[2].abs().sum() > 0
