"""The adapters' calls as programs mix them, on the GPU: a training step with clipping in a
graph, calls under way on two streams and from two threads, and the most tokens a call takes."""
import threading

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


@pytest.mark.parametrize("tokens", [6, 300])
def test_training_graph(tokens):
    """Forward, backward and clipping of two layers captured and replayed with new inputs: the eager step's bits."""
    torch.manual_seed(tokens)
    layers = nn.ModuleList(AD.AdapterLinear(AD.PackedLinear.pack(nn.Linear(128, 128, device="cuda", dtype=bf16), backward=True),
                                            adapters=3, rank=8) for _ in range(2))
    for layer in layers:
        nn.init.normal_(layer.adapters.b, std=0.3)
    params = list(layers.parameters())
    x, gy = (torch.randn(tokens, 128, device="cuda").to(bf16) for _ in range(2))
    ids = torch.randint(-1, 3, (tokens,), device="cuda", dtype=torch.int32)

    def step():
        layers[1](layers[0](x, ids), ids).backward(gy)
        return Q.clip_grad_norm_(params, 0.5)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            layers.zero_grad(set_to_none=True)
            step()
    torch.cuda.current_stream().wait_stream(side)
    layers.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step()
    grads = [p.grad for p in params]
    for seed in range(3):
        torch.manual_seed(seed)
        x.copy_(torch.randn(tokens, 128, device="cuda"))
        gy.copy_(torch.randn(tokens, 128, device="cuda"))
        ids.copy_(torch.randint(-1, 3, (tokens,), device="cuda"))
        for p in params:
            p.grad = None
        want = [step().clone(), *(p.grad.clone() for p in params)]
        for g in grads:
            g.zero_()                 # (the capture accumulates nothing: it made the gradients)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [norm, *grads]))


def test_two_streams_and_threads():
    """Calls of different sizes under way at once give what they give alone."""
    sets = [ta.Problem(*size, "mixed", bf16, seed=i) for i, size in enumerate(
        [(40, 512, 640, 16, 5), (700, 384, 520, 40, 4), (2000, 128, 256, 8, 3), (9, 1024, 96, 100, 7)])]

    def run(p, rounds=1):
        for _ in range(rounds):
            y, u = torch.empty_like(p.base), torch.empty(p.shape[0], p.shape[3], device="cuda")
            M.mxfp4_adapter_fwd(p.x, p.a, p.b, y, ids=p.ids, scale=p.scale, base=p.base, u=u)
            out = {"grad_x": torch.empty_like(p.x), "grad_a": torch.empty_like(p.a), "grad_b": torch.empty_like(p.b)}
            M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, base=p.gbase, **out)
            norm = torch.empty(1, device="cuda")
            M.mxfp4_grad_clip([out["grad_a"], out["grad_b"]], 0.1, norm)
        return [y, u, norm, *out.values()]

    want = [run(p) for p in sets]
    torch.cuda.synchronize()
    got, errors = [None] * len(sets), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = run(sets[i], rounds=20)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (shown below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_most_tokens():
    """2^26 tokens, rows past 2^32 bytes: the first, middle and last of them against 64 bits, and the gradient of A
    from the few tokens whose grad_y is not 0."""
    tokens, n_in, n_out, rank, adapters = 1 << 26, 40, 8, 2, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(tokens, n_in, dtype=bf16, device="cuda").normal_(generator=g)
    a = torch.randn(adapters, rank, n_in, generator=g, device="cuda").to(bf16)
    b = torch.randn(adapters, n_out, rank, generator=g, device="cuda").to(bf16)
    ids = torch.randint(-1, adapters, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    y = torch.full((tokens, n_out), float("nan"), dtype=bf16, device="cuda")
    M.mxfp4_adapter_fwd(x, a, b, y, ids=ids)
    at = torch.cat([torch.arange(k, k + 500, device="cuda") for k in (0, tokens // 2 - 250, tokens - 500)])
    i = ids[at].long()
    live = (i >= 0)[:, None]
    xs, ws, vs = x[at].double(), a[i.clamp(min=0)].double(), b[i.clamp(min=0)].double()
    u = (ws @ xs[:, :, None])[:, :, 0] * live
    want = (vs @ u[:, :, None])[:, :, 0]
    size = (vs.abs() @ (ws.abs() @ xs.abs()[:, :, None]))[:, :, 0]
    ta.within(y[at], want, (n_in + 16 + 2 * rank + 4) * ta.E * size + 2.0 ** -8 * want.abs())
    assert not y.isnan().any()
    del y
    gy = torch.zeros(tokens, n_out, dtype=bf16, device="cuda")
    gy[at] = torch.randn(at.numel(), n_out, generator=g, device="cuda").to(bf16)
    ga = torch.empty_like(a)
    M.mxfp4_adapter_bwd(gy, a, b, x=x, ids=ids, grad_a=ga)
    du = (gy[at].double()[:, None, :] @ vs)[:, 0] * live
    dsize = (gy[at].double().abs()[:, None, :] @ vs.abs())[:, 0] * live
    for e in range(adapters):
        of = i == e
        want, size = du[of].t() @ xs[of], dsize[of].t() @ xs[of].abs()
        # terms that are 0 add nothing: the 1500 tokens' and du's sums
        ta.within(ga[e], want, (2 * 1500 + 64 + n_out + 16) * ta.E * size + 2.0 ** -8 * want.abs())
