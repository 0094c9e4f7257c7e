"""The mixture-of-experts layer under another default type and after a cast, on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu
MOE = None
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    global MOE
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_fake_quantization_amd as mod
    from mxfp4_fake_quantization_amd import moe
    mod._load()
    MOE = moe
    yield


def step():
    """Forward, gradients and the packed experts of a layer with biases."""
    torch.manual_seed(8)
    layer = MOE.MoELayer(64, 96, 4, MOE.MoESpec(k=2), bias=True, device="cuda", dtype=bf16)
    assert layer.b1.dtype == layer.b2.dtype == f32
    with torch.no_grad():
        for b in (layer.b1, layer.b2):
            b.copy_(torch.randn(b.shape, device="cuda", dtype=f32))
    x = torch.randn(13, 64, device="cuda", dtype=f32).to(bf16)
    y = layer(x)
    y.float().square().sum().backward()
    logits = x @ layer.router.weight.t()
    return [y.detach(), *(p.grad for p in layer.parameters()), layer.packed()(x, logits)]


@pytest.mark.parametrize("default", [bf16, torch.float64], ids=["bf16", "f64"])
def test_under_a_default_type(default):
    """The same bits as under float32."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        got = step()
    finally:
        torch.set_default_dtype(before)
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_biases_after_a_cast():
    """A layer cast to bfloat16 is the layer of the rounded biases; their gradients are theirs, rounded."""
    torch.manual_seed(9)
    layer = MOE.MoELayer(64, 96, 4, MOE.MoESpec(k=2), bias=True, device="cuda", dtype=bf16)
    for b in (layer.b1, layer.b2):
        b.data.copy_(torch.randn(b.shape, device="cuda").to(bf16))
    x = torch.randn(13, 64, device="cuda").to(bf16)
    y = layer(x)
    y.float().square().sum().backward()
    want = [p.grad.clone() for p in layer.parameters()]
    packed = layer.packed()(x, x @ layer.router.weight.t())
    layer.zero_grad(set_to_none=True)
    layer.to(bf16)
    assert layer.b1.dtype == bf16
    again = layer(x)
    again.float().square().sum().backward()
    assert torch.equal(again, y)
    assert all(torch.equal(p.grad, g.to(bf16)) for p, g in zip(layer.parameters(), want))
    assert torch.equal(layer.packed()(x, x @ layer.router.weight.t()), packed)
