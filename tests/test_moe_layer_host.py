"""What PackedExperts and MoELayer hold and refuse, on the CPU: the packing call
is replaced by the identity, nothing reaches the library."""
import pytest
import torch

from mxfp4_fake_quantization_amd import moe


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(moe, "_pack", lambda w: (w.detach().clone(), w.detach().clone()))


def test_packed_experts_keep_the_biases_they_were_packed_with():
    """Weights and biases of one state: a later training step changes neither."""
    layer = moe.MoELayer(64, 32, 4, moe.MoESpec(k=2), bias=True)
    experts = layer.packed()
    before = [t.clone() for t in (experts.w1[0], experts.w2[0], experts.b1, experts.b2)]
    with torch.no_grad():
        for p in layer.parameters():
            p.add_(1.0)
    for a, b in zip(before, (experts.w1[0], experts.w2[0], experts.b1, experts.b2)):
        assert torch.equal(a, b) and not b.requires_grad
    assert moe.MoELayer(64, 32, 4).packed().b1 is None


def test_packed_experts_refuse_logits_of_another_width():
    """Fewer logits than experts would route over the first experts alone."""
    w1, w2 = torch.zeros(4, 64, 64, dtype=torch.bfloat16), torch.zeros(4, 64, 32, dtype=torch.bfloat16)
    experts = moe.PackedExperts(w1, w2)
    x = torch.zeros(5, 64, dtype=torch.bfloat16)
    for shape in ((5, 3), (5, 5), (4, 4), (20,)):
        with pytest.raises(ValueError, match=r"logits must be \[5, 4\]"):
            experts(x, torch.zeros(*shape))
    with pytest.raises(ValueError, match="64"):
        experts(torch.zeros(5, 32, dtype=torch.bfloat16), torch.zeros(5, 4))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer_with_weights_of_another_type_than_x(dtype, monkeypatch):
    """float32 master weights: the router takes x to its own type."""
    layer = moe.MoELayer(64, 32, 4, dtype=dtype)
    x, seen = torch.randn(2, 5, 64).bfloat16(), {}

    def ffn(flat, logits, *a):
        seen.update(x=flat, logits=logits)
        return torch.zeros_like(flat)
    monkeypatch.setattr(moe, "moe_ffn", ffn)
    y = layer(x)
    assert y.dtype == torch.bfloat16 and torch.equal(y, x) and seen["x"].dtype == torch.bfloat16
    assert seen["logits"].dtype == dtype
    want = x.view(10, 64).to(dtype) @ layer.router.weight.t()
    assert torch.allclose(seen["logits"], want, rtol=2.0 ** -7 if dtype == torch.bfloat16 else 1e-5, atol=1e-2 if
                          dtype == torch.bfloat16 else 1e-5)
