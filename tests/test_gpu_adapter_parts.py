"""All 24 bits of the adapters' fp32 values (u, du) reach the bf16 products, on the GPU.

Each value is the sum of three bf16 pieces of 8 bits, p0 + p1 + p2 with p0 in [1, 2), p1 in
[2^-8, 2^-7), p2 in [2^-16, 2^-15): 24 bits, every partial sum exact in fp32.  A second
term cancels p0 + p1, so that the result is p2 times a weight.  Tolerance: two terms that are
not 0, (2 * 2 + 4) 2^-23 of their magnitudes as in test_gpu_adapter, and the result's
rounding: 2^-18 of the weight beside 2^-16 to 2^-15.  (Two parts of 16 bits in all give 0 or
2^-15 for p2.)"""
import pytest
import torch

from test_gpu_adapter import E, half, within

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


def pieces(n, g):
    """[3, n]: pieces of one sign, 8 bits each."""
    m = 1 + torch.randint(0, 128, (3, n), generator=g).double() / 128
    return m * torch.tensor([1.0, 2.0 ** -8, 2.0 ** -16]).double()[:, None] * (1 - 2 * torch.randint(0, 2, (n,), generator=g))


SIZES = [  # tokens, in, out, rank, adapters: few rows, then many
    (1, 64, 128, 16, 2), (6, 96, 80, 3, 2), (40, 64, 96, 16, 5), (30, 72, 130, 24, 4), (33, 65, 97, 45, 3), (20, 128, 64, 128, 2),
    (70, 70, 140, 2, 1), (300, 200, 130, 16, 3), (300, 64, 520, 24, 2), (150, 129, 66, 40, 3), (200, 96, 192, 128, 2)]


def weights(tokens, cols, rank, adapters, g):
    """v [tokens, cols] and w [adapters, rank, cols]: v w^T is the three pieces' sum at one rank and the
    first two's at another, 0 at the rest; c [adapters, rank, n] weights of both, of opposite signs."""
    at = [torch.randperm(cols, generator=g)[:3] for _ in range(adapters)]
    ranks = [torch.randperm(rank, generator=g)[:2] for _ in range(adapters)]
    ids = torch.randint(0, adapters, (tokens,), generator=g)
    v = torch.randn(tokens, cols, generator=g).double()
    w = torch.zeros(adapters, rank, cols).double()
    p = pieces(tokens, g)
    for i in range(adapters):
        w[i, ranks[i][0], at[i]] = 1
        w[i, ranks[i][1], at[i][:2]] = 1
        for t in (ids == i).nonzero()[:, 0].tolist():
            v[t, at[i]] = p[:, t]
    return v, w, p, ids, ranks


def cancelling(adapters, n, rank, ranks, g):
    """[adapters, n, rank] weights c of the first rank, -c of the second."""
    c = torch.zeros(adapters, n, rank).double()
    val = torch.randint(64, 128, (adapters, n), generator=g).double() / 64
    for i in range(adapters):
        c[i, :, ranks[i][0]], c[i, :, ranks[i][1]] = val[i], -val[i]
    return c, val


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_products(size, dt):
    """y, and grad_x by the same product with the weights' parts exchanged."""
    tokens, n_in, n_out, rank, adapters = size
    g = torch.Generator().manual_seed(tokens + rank)
    for forward in (True, False):
        cols, n = (n_in, n_out) if forward else (n_out, n_in)
        v, w, p, ids, ranks = weights(tokens, cols, rank, adapters, g)
        c, val = cancelling(adapters, n, rank, ranks, g)
        want = p[2][:, None] * val[ids]
        size_of = 2 * p.sum(0).abs()[:, None] * val[ids]
        v, ids = v.to(dt).cuda(), ids.to(torch.int32).cuda()
        got = torch.empty(tokens, n, dtype=dt, device="cuda")
        if forward:
            M.mxfp4_adapter_fwd(v, w.to(dt).cuda(), c.to(dt).cuda(), got, ids=ids)
        else:
            M.mxfp4_adapter_bwd(v, c.transpose(1, 2).contiguous().to(dt).cuda(), w.transpose(1, 2).contiguous().to(dt).cuda(),
                                ids=ids, grad_x=got)
        want, size_of = want.cuda(), size_of.cuda()
        within(got, want, 8 * E * size_of + half(dt) * want.abs())


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [s for s in SIZES if s[0] >= 2 * s[4]], ids=str)
def test_weight_gradients(size, dt):
    """Two tokens of each adapter have a part in one rank, with opposite rows."""
    tokens, n_in, n_out, rank, adapters = size
    g = torch.Generator().manual_seed(tokens + 7 * rank)
    v, w, p, ids, ranks = weights(tokens, n_out, rank, adapters, g)
    x = torch.randint(-128, 129, (tokens, n_in), generator=g).double() / 64
    pairs = torch.randperm(tokens, generator=g)[:2 * adapters].view(adapters, 2)
    gy, u = torch.zeros_like(v), torch.zeros(tokens, rank).double()
    rows = torch.randint(-128, 129, (tokens, n_out), generator=g).double() / 64
    want_a, size_a = torch.zeros(adapters, rank, n_in).double(), torch.zeros(adapters, rank, n_in).double()
    want_b, size_b = torch.zeros(adapters, n_out, rank).double(), torch.zeros(adapters, n_out, rank).double()
    gy_u = torch.zeros_like(gy)  # grad_y of the second call, whose u has the pieces
    for i, (s, t) in enumerate(pairs.tolist()):
        ids[s] = ids[t] = i
        r = int(ranks[i][0])
        at = w[i, r].nonzero()[:, 0]
        low = w[i, ranks[i][1]].nonzero()[:, 0]
        q = pieces(1, g)[:, 0]
        order = [k for k in at.tolist() if k in low.tolist()] + [k for k in at.tolist() if k not in low.tolist()]
        gy[s, order] = q
        gy[t, order[:2]] = q[:2]
        w[i, ranks[i][1]] = 0
        x[t] = -x[s]
        want_a[i, r], size_a[i, r] = q[2] * x[s], 2 * q.sum().abs() * x[s].abs()
        u[s, r], u[t, r] = q.sum(), q[:2].sum()
        gy_u[s], gy_u[t] = rows[s], -rows[s]
        want_b[i, :, r], size_b[i, :, r] = q[2] * rows[s], 2 * q.sum().abs() * rows[s].abs()
    dev = lambda m: m.to(dt).cuda()  # noqa: E731
    a, b, ids = torch.zeros(adapters, rank, n_in, dtype=dt, device="cuda"), dev(w.transpose(1, 2).contiguous()), ids.to(torch.int32).cuda()
    ga, gb = torch.empty_like(a), torch.empty_like(b)
    M.mxfp4_adapter_bwd(dev(gy), a, b, x=dev(x), ids=ids, grad_a=ga)
    want, bound = want_a.cuda(), size_a.cuda()
    within(ga, want, 8 * E * bound + half(dt) * want.abs())
    M.mxfp4_adapter_bwd(dev(gy_u), a, b, u=u.float().cuda(), ids=ids, grad_b=gb)
    want, bound = want_b.cuda(), size_b.cuda()
    within(gb, want, 8 * E * bound + half(dt) * want.abs())


def as_formula(got, terms, base=0.0):
    """The infinities and NaN of the sum of the last dimension's terms (in 64 bits), and its finite values
    within 2^-8 of a bf16 result and (6 m + 64) 2^-23 of the m terms' magnitudes: three products a term,
    each an addition and its rounding, and the waves' parts."""
    want = base + terms.sum(-1)
    got, m = got.double().cpu(), terms.shape[-1]
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.isinf(), want.isinf()) and torch.equal(got[want.isinf()], want[want.isinf()])
    ok = want.isfinite()
    bound = 2.0 ** -8 * want.abs() + (6 * m + 64) * E * (abs(base) + terms.abs().sum(-1))
    assert bool(((got - want).abs()[ok] <= bound[ok]).all())


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [(5, 64, 72, 16, 2), (40, 136, 65, 7, 3), (30, 72, 130, 24, 4), (50, 128, 128, 100, 4),
                                  (300, 64, 130, 16, 3), (300, 96, 136, 24, 2), (150, 130, 66, 40, 3), (200, 192, 96, 96, 2)], ids=str)
def test_infinite_operands(size, dt):
    """Infinities in weights and rows beside values of few bits, whose lower parts are 0 if nothing is
    borrowed: y, grad_x, grad_a and grad_b are what the formula gives."""
    tokens, n_in, n_out, rank, adapters = size
    g = torch.Generator().manual_seed(tokens + rank)
    ids = torch.randint(0, adapters, (tokens,), generator=g)
    dev = lambda m: m.to(dt).cuda()  # noqa: E731

    def few_bits(*shape):
        return torch.tensor([0.0, 1.0, -2.0, 0.5, 3.0, 1.0, -1.0, 0.125])[torch.randint(0, 8, shape, generator=g)].double()

    def with_infinities(*shape, rate):
        v = few_bits(*shape)
        at = torch.rand(*shape, generator=g)
        v[at < rate] = float("inf")
        v[at > 1 - rate] = -float("inf")
        return v

    def ones(cols):  # [adapters, rank, cols]: rank r takes column r (from the first again past the last)
        w = torch.zeros(adapters, rank, cols).double()
        w[:, torch.arange(rank), torch.arange(rank) % cols] = 1
        return w

    def picked(v):   # v times ones() of the same columns
        return v[:, torch.arange(rank) % v.shape[1]]

    rate = 0.6 / rank
    i = ids.to(torch.int32).cuda()
    x, base, b = few_bits(tokens, n_in), few_bits(tokens, n_out), with_infinities(adapters, n_out, rank, rate=rate)
    y = torch.empty(tokens, n_out, dtype=dt, device="cuda")
    M.mxfp4_adapter_fwd(dev(x), dev(ones(n_in)), dev(b), y, ids=i, base=dev(base))
    as_formula(y, picked(x)[:, None, :] * b[ids], base)
    gy, a = few_bits(tokens, n_out), with_infinities(adapters, rank, n_in, rate=rate)
    one = ones(n_out).transpose(1, 2).contiguous()
    gx = torch.empty(tokens, n_in, dtype=dt, device="cuda")
    M.mxfp4_adapter_bwd(dev(gy), dev(a), dev(one), ids=i, grad_x=gx)
    as_formula(gx, picked(gy)[:, None, :] * a[ids].transpose(1, 2))
    # a weight gradient's infinities: values that are not 0, that they stay infinities
    v = few_bits(tokens, n_out)
    v[v == 0] = 1
    rows = with_infinities(tokens, n_in, rate=0.3 / tokens)
    ga = torch.empty(adapters, rank, n_in, dtype=dt, device="cuda")
    M.mxfp4_adapter_bwd(dev(v), dev(a), dev(one), x=dev(rows), ids=i, grad_a=ga)
    u = few_bits(tokens, rank)
    u[u == 0] = 1
    gr = with_infinities(tokens, n_out, rate=0.3 / tokens)
    gb = torch.empty(adapters, n_out, rank, dtype=dt, device="cuda")
    M.mxfp4_adapter_bwd(dev(gr), dev(a), dev(one), u=u.float().cuda(), ids=i, grad_b=gb)
    for e in range(adapters):
        at = ids == e
        as_formula(ga[e], (picked(v)[at][:, :, None] * rows[at][:, None, :]).movedim(0, -1))
        as_formula(gb[e], (gr[at][:, :, None] * u[at][:, None, :]).movedim(0, -1))
    assert ga.isinf().any() and gb.isinf().any() and y.isinf().any() and gx.isinf().any()
