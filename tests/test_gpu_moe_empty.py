"""The mixture-of-experts layer with nothing to do: a batch without tokens and a
batch whose tokens all go to no expert, through serving and training.  Every
result is known without rounding: empty, the residual, or zeros."""
import pytest
import torch

pytestmark = pytest.mark.gpu
M = MOE = None
NEG = float("-inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    global M, MOE
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_fake_quantization_amd as mod
    from mxfp4_fake_quantization_amd import moe
    mod._load()
    M, MOE = mod, moe
    yield


def weights(E, H, I, act):
    g = torch.Generator().manual_seed(1)
    n1 = I * (2 if act == "swiglu" else 1)
    return [(torch.randn(*s, generator=g) * 0.1).to(dt).cuda() for s, dt in
            (((E, n1, H), torch.bfloat16), ((E, H, I), torch.bfloat16), ((E, n1), torch.float32), ((E, H), torch.float32))]


@pytest.mark.parametrize("act", ["swiglu", "relu"])
@pytest.mark.parametrize("tokens", [0, 1, 70])
def test_serving(tokens, act):
    E, H, I = 3, 96, 64
    w1, w2, b1, b2 = weights(E, H, I, act)
    experts = MOE.PackedExperts(w1, w2, MOE.MoESpec(k=2, act=act), b1, b2)
    x = torch.randn(tokens, H, device="cuda").bfloat16()
    logits = torch.full((tokens, E), NEG, device="cuda")
    y = experts(x, logits, residual=x)
    assert y.shape == x.shape and torch.equal(y, x)
    assert torch.equal(experts(x, logits), torch.zeros_like(x))


@pytest.mark.parametrize("act,score,renorm", [("swiglu", "softmax", True), ("gelu", "sigmoid", False)])
@pytest.mark.parametrize("tokens", [0, 1, 70])
def test_training(tokens, act, score, renorm):
    E, H, I = 3, 96, 64
    params = [p.requires_grad_(True) for p in weights(E, H, I, act)]
    w1, w2, b1, b2 = params
    x = torch.randn(tokens, H, device="cuda").bfloat16().requires_grad_(True)
    logits = torch.full((tokens, E), NEG, device="cuda").requires_grad_(True)
    y = MOE.moe_ffn(x, logits, w1, w2, MOE.MoESpec(k=2, act=act, score=score, renormalize=renorm), b1, b2)
    assert y.shape == x.shape and (y == 0).all()
    y.backward(torch.randn(tokens, H, device="cuda").bfloat16())
    for p in (x, logits, *params):
        assert p.grad is not None and p.grad.shape == p.shape and p.grad.dtype == p.dtype and (p.grad == 0).all()


def test_layer():
    layer = MOE.MoELayer(64, 32, 4, device="cuda")
    x = torch.empty(2, 0, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = layer(x)
    assert y.shape == x.shape
    y.sum().backward()
    assert all((p.grad == 0).all() for p in layer.parameters())


def test_weight_gradient_of_no_tokens():
    """Groups that split an empty K write zeros."""
    z = torch.empty(48, 0, dtype=torch.uint8, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        c = torch.full((3, 48, 48), 5.0, dtype=dt, device="cuda")
        M.mxfp4_grouped_matmul(z, z, z, z, c, K=0, group_list=torch.zeros(3, dtype=torch.int64, device="cuda"),
                               group_type=M.GROUP_K, b_fmt="e4m3")
        assert (c == 0).all()
