"""The mixture-of-experts layer with float32 master weights on bfloat16 tokens."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_float32_weights_train_like_their_bfloat16_values():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mxfp4_fake_quantization_amd import moe
    torch.manual_seed(3)
    spec = moe.MoESpec(k=2)
    a = moe.MoELayer(128, 64, 4, spec, bias=True, device="cuda")
    b = moe.MoELayer(128, 64, 4, spec, bias=True, device="cuda", dtype=torch.float32)
    b.load_state_dict(a.state_dict())                    # the same values, held in float32
    x = torch.randn(3, 40, 128, device="cuda").bfloat16()
    flat = x.view(-1, 128)
    logits = (flat.float() @ b.router.weight.t()).detach()
    # the same logits to both: quantized weights and all products are then equal bit for bit
    outs = []
    for layer in (a, b):
        y = moe.moe_ffn(flat, logits, layer.w1, layer.w2, spec, layer.b1, layer.b2)
        y.backward(torch.ones_like(y))
        outs.append(y.detach())
    assert torch.equal(outs[0], outs[1])
    for n in ("w1", "w2", "b1", "b2"):
        ga, gb = getattr(a, n).grad, getattr(b, n).grad
        assert gb.dtype == torch.float32 and torch.equal(ga.float(), gb), n
    y = b(x)
    y.float().square().mean().backward()
    assert y.dtype == torch.bfloat16 and torch.isfinite(y).all()
    assert b.router.weight.grad.dtype == torch.float32 and b.router.weight.grad.abs().sum() > 0
