"""Second derivatives of the mixture-of-experts layer: its backward pass works on
quantized operands outside autograd, so asking for them is an error and never a
silently incomplete gradient."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_second_derivatives_are_refused():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mxfp4_fake_quantization_amd import moe
    layer = moe.MoELayer(64, 32, 4, device="cuda")
    x = torch.randn(6, 64, device="cuda").bfloat16().requires_grad_(True)
    g, = torch.autograd.grad(layer(x).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.float().square().sum().backward()
    # a first derivative with create_graph is the same as one without
    want, = torch.autograd.grad(layer(x).float().square().sum(), x)
    assert torch.equal(g.detach(), want)
