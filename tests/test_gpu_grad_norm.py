"""The gradient norm and clipping on the GPU against 64 bits.

Tolerances: the sum of n terms in 64 bits is off by n 2^-53 of it at most (below
2^-30 here), its root and rounding to fp32 by 2^-24 each: 2^-23 of the norm.  The
coefficient adds an addition, a division and the norm's own error: 2^-23 + 2 * 2^-24 =
2^-22 of it; a clipped element one rounding of its type more."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
M = None
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    global M
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_fake_quantization_amd as mod
    mod._load()
    M = mod
    yield


def grads_of(sizes, dtypes, seed=0, level=1e-3):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * level * (1 + i % 5)).to(dtypes[i % len(dtypes)]).cuda()
            for i, n in enumerate(sizes)]


def norm64(grads, p):
    v = torch.cat([t.double().reshape(-1) for t in grads]).abs() if grads else torch.zeros(1)
    if p == math.inf:
        return float(v.max())
    return float(v.sum() if p == 1 else v.square().sum().sqrt())


def same_norm(got, want):
    assert abs(float(got) - want) <= 2.0 ** -23 * want, (float(got), want)


SETS = {
    "one": ([5], [f32]), "element": ([1], [bf16]), "tiny": ([2048, 64, 2048, 32], [f32]),
    "odd": ([1, 3, 1023, 1025, 4097, 8191, 8193, 70001], [bf16, f32]),
    "chunks": ([16384, 16385, 40960, 131072], [bf16]), "many": ([17 + 13 * i for i in range(700)], [bf16, f32]),
    "empty": ([0, 100, 0], [f32]), "large": ([5_000_000, 33, 12_345_677], [bf16]),
}


@pytest.mark.parametrize("p", [2.0, 1.0, math.inf])
@pytest.mark.parametrize("name", sorted(SETS))
def test_norm(name, p):
    grads = grads_of(*SETS[name])
    norm = torch.full((1,), float("nan"), device="cuda")
    M.mxfp4_grad_norm(grads, norm, norm_type=p)
    same_norm(norm, norm64(grads, p))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("ratio", [0.03, 0.999, 1.5])
@pytest.mark.parametrize("name", sorted(SETS))
def test_clip(name, ratio, in_place):
    for p in (2.0, 1.0, math.inf):
        grads = grads_of(*SETS[name])
        keep = [t.clone() for t in grads]
        want = norm64(grads, p)
        bound = ratio * want
        norm = torch.full((), float("nan"), device="cuda")
        outs = None if in_place else [torch.full_like(t, float("nan")) for t in grads]
        M.mxfp4_grad_clip(grads, bound, norm, outs=outs, norm_type=p)
        same_norm(norm, want)
        coef = min(1.0, bound / (want + 1e-6))
        for k, t, o in zip(keep, grads, grads if in_place else outs):
            off = (o.double() - k.double() * coef).abs()
            tiny = torch.finfo(t.dtype).smallest_normal  # below it a rounding is absolute
            half = torch.finfo(t.dtype).eps / 2 if coef < 1 else 0.0
            assert bool((off <= k.double().abs() * coef * (half + 2.0 ** -22) + tiny * half).all())
            if not in_place:
                assert torch.equal(t, k)
            if coef == 1.0:
                assert torch.equal(o, k)


def test_norm_given():
    """A norm from outside (several processes) is used as it is."""
    grads = grads_of([1000, 77], [bf16, f32])
    keep = [t.clone() for t in grads]
    norm = torch.tensor([50.0], device="cuda")
    M.mxfp4_grad_clip(grads, 5.0, norm, compute_norm=False)
    coef = 5.0 / (50.0 + 1e-6)
    assert float(norm) == 50.0
    for k, t in zip(keep, grads):
        assert bool(((t.double() - k.double() * coef).abs()
                     <= k.double().abs() * coef * (torch.finfo(t.dtype).eps / 2 + 2.0 ** -22) + 1e-38).all())


def test_extremes():
    """Squares beyond fp32's range neither overflow nor vanish; NaN and infinity."""
    norm = torch.empty(1, device="cuda")
    for level in (1e-30, 1e-42, 1e30):
        g = [torch.full((999,), level, device="cuda"), torch.full((3,), -level, device="cuda")]
        M.mxfp4_grad_norm(g, norm)
        want = norm64(g, 2)
        assert abs(float(norm) - want) <= 2.0 ** -23 * want + 2.0 ** -150
    big = [torch.full((100_000,), 3e38, device="cuda")]
    M.mxfp4_grad_norm(big, norm)
    assert float(norm) == math.inf                       # 9.5e40 is no fp32
    for p in (1.0, 2.0, math.inf):
        g = grads_of([3000, 20000], [bf16, f32])
        g[1][12345] = float("inf")
        M.mxfp4_grad_clip(g, 1.0, norm, norm_type=p)
        assert float(norm) == math.inf
        assert not g[0].any() and g[1][12345].isnan() and int(g[1].isnan().sum()) == 1 and not g[1][:12345].any()
        g = grads_of([3000, 20000], [bf16, f32])
        g[0][17] = float("nan")
        M.mxfp4_grad_clip(g, 1.0, norm, norm_type=p)
        assert norm.isnan().all() and all(t.isnan().all() for t in g)
    # the largest magnitude is exact, whatever its sign, and a NaN before or after it stays
    g = grads_of([50_000], [f32], level=1.0)
    g[0][49_999] = -77.25
    M.mxfp4_grad_norm(g, norm, norm_type=math.inf)
    assert float(norm) == 77.25
    for at in (0, 25_000, 49_998):
        h = [g[0].clone()]
        h[0][at] = float("nan")
        M.mxfp4_grad_norm(h, norm, norm_type=math.inf)
        assert norm.isnan().all()


def test_no_gradients():
    norm = torch.full((1,), 5.0, device="cuda")
    M.mxfp4_grad_norm([], norm)
    assert float(norm) == 0.0
    norm.fill_(5.0)
    M.mxfp4_grad_clip([torch.empty(0, device="cuda")], 1.0, norm)
    assert float(norm) == 0.0


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
def test_bucket(dt):
    """Views of a flat bucket, end to end or apart, at any element: what lies between
    them stays as it was, and end to end gives what one tensor gives."""
    g = torch.Generator().manual_seed(3)
    sizes, flat = [1000, 1, 33333, 64, 20000], (torch.randn(54400, generator=g)).to(dt).cuda()
    for gap in (0, 1, 5):
        at, views = 1, []
        for n in sizes:
            views.append((at, n))
            at += n + gap
        grads = [flat[a:a + n] for a, n in views]
        out = torch.full_like(flat, 9.0)
        norm, one = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        M.mxfp4_grad_clip(grads, 2.0, norm, outs=[out[a:a + n] for a, n in views])
        same_norm(norm, norm64(grads, 2))
        beside = torch.ones(flat.numel(), dtype=torch.bool)
        for a, n in views:
            beside[a:a + n] = False
        assert (out[beside.cuda()] == 9.0).all()
        single = [torch.empty_like(t) for t in grads]
        M.mxfp4_grad_clip(grads, 2.0, norm, outs=single)       # outputs apart: the same values
        assert all(torch.equal(out[a:a + n], s) for (a, n), s in zip(views, single))
        if gap == 0:
            M.mxfp4_grad_norm([flat[1:1 + sum(sizes)]], one)
            assert torch.equal(norm, one)


def test_past_32_bits():
    """A tensor of more than 2^32 bytes, whose last elements are what there is."""
    t = torch.zeros((1 << 31) + 77, dtype=bf16, device="cuda")
    t[-3:] = torch.tensor([3.0, -4.0, 12.0])
    t[5] = 84.0
    norm = torch.empty(1, device="cuda")
    M.mxfp4_grad_norm([t], norm)
    assert float(norm) == 85.0
    M.mxfp4_grad_clip([t], 42.5, norm)
    assert float(norm) == 85.0 and t[-3:].tolist() == [1.5, -2.0, 6.0] and float(t[5]) == 42.0
    assert int(t.count_nonzero()) == 4


def test_streams_and_graphs():
    grads = grads_of([3000, 70000, 5, 20000], [bf16, f32])
    outs = [torch.empty_like(t) for t in grads]
    norm = torch.empty(1, device="cuda")
    alone = torch.empty(1, device="cuda")

    def step():
        M.mxfp4_grad_norm(grads, alone, norm_type=1.0)
        M.mxfp4_grad_clip(grads, 0.5, norm, outs=outs)

    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in (norm, alone, *outs)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (norm, alone, *outs)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator(device="cuda").manual_seed(9)
    for _ in range(4):
        for t in grads:
            t.normal_(generator=g)
        step()
        want = [t.clone() for t in (norm, alone, *outs)]
        for t in (norm, alone, *outs):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (norm, alone, *outs)))
