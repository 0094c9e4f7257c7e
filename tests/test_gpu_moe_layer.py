"""The mixture-of-experts layer end to end on the GPU.

Serving: against the same layer in 64 bits on the decoded operands, the
activation taken through bf16 and MXFP8 as the layer does.  The two differ by
the roundings of a bf16 result (2^-9 each) and by MXFP8 codes that fall on the
other side of a rounding boundary (2^-4 of an element, a few percent of the
elements): 1 % of the norm.

Training: against float autograd of the unquantized layer.  An MXFP4 operand is
off by about 0.1 of its norm and an MXFP8 one by 0.03, independently of each
other, so a gradient through up to four such products is within 0.35 of its
norm and points its way (cosine above 0.93); a wrong operand, order or sign is
off by 1 or more."""
import pytest
import torch

pytestmark = pytest.mark.gpu
M = MOE = None


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


FP4 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def decode4(codes, scales):
    c = codes.cpu().long()
    v = torch.stack([FP4[c & 15], FP4[c >> 4]], -1).flatten(-2)
    return v * torch.exp2(scales.cpu().double() - 127).repeat_interleave(32, -1)


def through8(x):
    """bf16 -> MXFP8 -> 64-bit values, with the library's quantizer."""
    q, s = MOE._mxfp8(x.contiguous().cuda())
    return q.view(torch.float8_e4m3fn).cpu().double() * torch.exp2(s.cpu().double() - 127).repeat_interleave(32, -1)


def act64(z, name):
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        return g * torch.sigmoid(g) * u
    return z * 0.5 * torch.erfc(-z * 0.5 ** 0.5)


@pytest.mark.parametrize("tokens,act,bias", [(1, "swiglu", False), (5, "gelu", True), (64, "swiglu", True),
                                             (700, "swiglu", False)])
def test_packed_experts(tokens, act, bias):
    E, H, I, k = 6, 256, 160, 3
    spec = MOE.MoESpec(k=k, score="sigmoid", act=act, scale=1.5)
    g = torch.Generator().manual_seed(tokens)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n1 = 2 * I if act == "swiglu" else I
    w1, w2 = (rn(E, n1, H) * H ** -0.5).bfloat16(), (rn(E, H, I) * I ** -0.5).bfloat16()
    b1, b2 = (0.3 * rn(E, n1), 0.3 * rn(E, H)) if bias else (None, None)
    x, logits = rn(tokens, H).bfloat16(), rn(tokens, E)
    if tokens > 4:
        logits[3] = float("-inf")               # a token for no expert: the residual alone
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    experts = MOE.PackedExperts(cu(w1), cu(w2), spec, cu(b1), cu(b2))
    y = experts(cu(x), cu(logits), residual=cu(x)).cpu().double()
    d1, d2 = decode4(*experts.w1), decode4(*experts.w2)
    xq = through8(x)
    s = torch.sigmoid(logits.double())
    top = logits.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    want = x.double().clone()
    for t in range(tokens):
        if logits[t, 0] == float("-inf"):
            continue
        p = s[t, top[t]]
        for j in range(k):
            e = int(top[t, j])
            z = xq[t] @ d1[e].t() + (0 if b1 is None else b1[e].double())
            a = through8(act64(z, act).bfloat16()[None])[0]
            o = a @ d2[e].t() + (0 if b2 is None else b2[e].double())
            want[t] += 1.5 * p[j] / p.sum() * o.bfloat16().double()
    assert (y - want).norm() <= 0.01 * (want - x.double()).norm() + 2.0 ** -8 * want.norm()
    if tokens > 4:
        assert torch.equal(y[3], x[3].double())


@pytest.mark.parametrize("tokens", [3, 400])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_training_gradients(tokens, score, renorm):
    E, H, I, k = 5, 256, 128, 2
    spec = MOE.MoESpec(k=k, score=score, renormalize=renorm)
    g = torch.Generator().manual_seed(7 + tokens)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    base = [rn(tokens, H).bfloat16(), rn(tokens, E), (rn(E, 2 * I, H) * H ** -0.5).bfloat16(),
            (rn(E, H, I) * I ** -0.5).bfloat16(), 0.1 * rn(E, 2 * I), 0.1 * rn(E, H)]
    dy = rn(tokens, H).bfloat16()
    ours = [t.cuda().requires_grad_(True) for t in base]
    y = MOE.moe_ffn(*ours[:4], spec, *ours[4:])
    y.backward(dy.cuda())

    ref = [t.double().requires_grad_(True) for t in base]
    x, l, w1, w2, b1, b2 = ref
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, -1)
    ids = base[1].sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    if renorm:
        w = w / w.sum(-1, keepdim=True)
    out = 0
    for j in range(k):
        e = ids[:, j]
        z = torch.einsum("th,tnh->tn", x, w1[e]) + b1[e]
        a = act64(z, "swiglu")
        out = out + w[:, j:j + 1] * (torch.einsum("ti,thi->th", a, w2[e]) + b2[e])
    out.backward(dy.double())
    assert (y.detach().cpu().double() - out.detach()).norm() <= 0.25 * out.detach().norm()
    for a, b, name in zip(ours, ref, ("x", "logits", "w1", "w2", "b1", "b2")):
        got, want = a.grad.cpu().double(), b.grad
        assert got.shape == want.shape and a.grad.dtype == a.dtype, name
        assert (got - want).norm() <= 0.35 * want.norm(), name
        assert (got * want).sum() >= 0.93 * got.norm() * want.norm(), name


def test_layer_trains_and_serves():
    torch.manual_seed(0)
    layer = MOE.MoELayer(128, 64, 4, MOE.MoESpec(k=2), bias=True, device="cuda")
    x = torch.randn(2, 50, 128, device="cuda").bfloat16()
    want = torch.randn(2, 50, 128, device="cuda").bfloat16()
    opt = torch.optim.SGD(layer.parameters(), lr=0.1)
    losses = []
    for _ in range(8):
        opt.zero_grad()
        loss = (layer(x) - want).float().square().mean()
        loss.backward()
        assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in layer.parameters())
        opt.step()
        losses.append(loss.item())
    assert losses[-1] < losses[0]
    with torch.no_grad():
        y = layer(x)
    flat = x.view(-1, 128)
    served = layer.packed()(flat, torch.nn.functional.linear(flat, layer.router.weight), residual=flat)
    # the layer adds the residual to a bf16 result, serving adds it before rounding
    assert (served.view_as(y).float() - y.float()).abs().max() <= 2.0 ** -7 * y.float().abs().max()
