"""The low-rank adapters on the GPU against their formulas in 64 bits.

Tolerances, derived from the arithmetic (E: 2^-23 per fp32 addition or product,
which covers a matrix core that truncates; H: 2^-8 of a bf16 result, 2^-24 of an
fp32 one; S: 2^-16 for an fp32 value that goes into a bf16 product as two halves, 0
in fp32; bf16 products are exact in fp32, fp32 ones count within E):
  u          (K + 16) E sum|x||a|                      (the waves' parts included)
  y          |s| |b| err(u) + (S + (2 r + 4) E) |s| |u| |b| before its rounding, H |y| for it
  grad_x     the same with du for u, a for b
  grad_a     err(du) |x| + (S + (2 n + 64) E) |du| |x|, H |grad_a|  (n: the adapter's rows)
  grad_b     the same with s u and grad_y, u being an input."""
import pytest
import torch

pytestmark = pytest.mark.gpu
M = None
E = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def lib():
    global M
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_fake_quantization_amd as mod
    mod._load()
    M = mod
    yield


bf16, f32 = torch.bfloat16, torch.float32


def half(dt):
    return torch.finfo(dt).eps / 2


def split(dt):
    return 2.0 ** -16 if dt == bf16 else 0.0


def ids_of(pattern, tokens, adapters, g):
    """None, or the adapter of each token."""
    if pattern == "null":
        return None
    if pattern == "runs":       # requests one after the other
        cuts = torch.rand(tokens, generator=g) < 6.0 / max(tokens, 6)
        order = torch.randint(0, adapters, (tokens + 1,), generator=g)
        ids = order[cuts.long().cumsum(0)]
    elif pattern == "mixed":    # any order, some without an adapter, some numbers out of range
        ids = torch.randint(-1, adapters, (tokens,), generator=g)
        ids[torch.rand(tokens, generator=g) < 0.1] = adapters + 7
    elif pattern == "none":
        ids = torch.full((tokens,), -1)
    else:                       # all tokens the last adapter
        ids = torch.full((tokens,), adapters - 1)
    return ids.to(torch.int32).cuda()


class Problem:
    def __init__(self, tokens, n_in, n_out, rank, adapters, pattern, dt, seed=0):
        g = torch.Generator().manual_seed(seed + 1000 * tokens + rank)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.dt, self.shape = dt, (tokens, n_in, n_out, rank, adapters)
        self.x = r(tokens, n_in).to(dt).cuda()
        self.a = (r(adapters, rank, n_in) * n_in ** -0.5).to(dt).cuda()
        self.b = (r(adapters, n_out, rank) * 0.3).to(dt).cuda()
        self.scale = (0.5 + torch.rand(adapters, generator=g)).cuda()
        self.base = r(tokens, n_out).to(dt).cuda()
        self.gy = r(tokens, n_out).to(dt).cuda()
        self.gbase = r(tokens, n_in).to(dt).cuda()
        self.ids = ids_of(pattern, tokens, adapters, g)

    def rows(self):
        """(adapter, its rows) of all adapters."""
        tokens, adapters = self.shape[0], self.shape[4]
        ids = torch.zeros(tokens, dtype=torch.int64) if self.ids is None else self.ids.cpu().long()
        return [(i, (ids == i).nonzero()[:, 0].cuda()) for i in range(adapters)]

    def forward64(self, scale, base):
        """(y, its bound, u, its bound)."""
        tokens, n_in, n_out, rank, _ = self.shape
        u = torch.zeros(tokens, rank, dtype=torch.float64, device="cuda")
        ub = torch.zeros_like(u)
        y = self.base.double() if base else torch.zeros(tokens, n_out, dtype=torch.float64, device="cuda")
        e = torch.zeros_like(y)
        for i, at in self.rows():
            if at.numel():
                x, a, b = self.x[at].double(), self.a[i].double(), self.b[i].double()
                s = float(self.scale[i]) if scale else 1.0
                u[at] = x @ a.t()
                ub[at] = (n_in + 16) * E * (x.abs() @ a.abs().t())
                y[at] += s * (u[at] @ b.t())
                e[at] += s * (ub[at] @ b.abs().t()) + (split(self.dt) + (2 * rank + 4) * E) * s * (u[at].abs() @ b.abs().t())
        return y, e + half(self.dt) * (y.abs() + e) + E * y.abs(), u, ub

    def backward64(self, u, scale, base):
        """name -> (value, bound)."""
        tokens, n_in, n_out, rank, adapters = self.shape
        gx = self.gbase.double() if base else torch.zeros(tokens, n_in, dtype=torch.float64, device="cuda")
        ex = torch.zeros_like(gx)
        ga, gb = torch.zeros_like(self.a, dtype=torch.float64), torch.zeros_like(self.b, dtype=torch.float64)
        ea, eb = torch.zeros_like(ga), torch.zeros_like(gb)
        h, sp = half(self.dt), split(self.dt)
        for i, at in self.rows():
            n = at.numel()
            if n:
                x, a, b, gy = self.x[at].double(), self.a[i].double(), self.b[i].double(), self.gy[at].double()
                s = float(self.scale[i]) if scale else 1.0
                du = s * (gy @ b)
                de = (n_out + 16) * E * s * (gy.abs() @ b.abs())
                gx[at] += du @ a
                ex[at] += de @ a.abs() + (sp + (2 * rank + 4) * E) * (du.abs() @ a.abs())
                ga[i] = du.t() @ x
                ea[i] = de.t() @ x.abs() + (sp + (2 * n + 64) * E) * (du.abs().t() @ x.abs())
                ui = u[at].double()
                gb[i] = s * (gy.t() @ ui)
                eb[i] = s * (sp + (2 * n + 64) * E) * (gy.abs().t() @ ui.abs())
        out = {"grad_x": (gx, ex), "grad_a": (ga, ea), "grad_b": (gb, eb)}
        return {k: (v, e + h * (v.abs() + e) + E * v.abs()) for k, (v, e) in out.items()}


def within(got, want, bound):
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"off by up to {float((off / bound.clamp(min=1e-300)).max()):.3g} bounds"


SIZES = [
    # tokens, in, out, rank, adapters
    (1, 64, 64, 1, 1), (1, 4096, 1000, 16, 5), (2, 33, 31, 3, 2), (3, 1025, 515, 5, 4), (7, 256, 130, 8, 3),
    (16, 512, 512, 16, 16), (17, 97, 1031, 12, 6), (63, 640, 257, 24, 9), (64, 128, 384, 32, 64), (65, 700, 129, 33, 3),
    (130, 511, 513, 64, 4), (257, 2048, 96, 7, 20), (300, 90, 2050, 100, 2), (1000, 1024, 640, 128, 3),
    (2111, 320, 448, 16, 40), (5000, 96, 64, 4, 7)]


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pattern", ["mixed", "runs"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, pattern, dt):
    p = Problem(*size, pattern, dt)
    y = torch.full_like(p.base, float("nan"))
    u = torch.full((size[0], size[3]), float("nan"), device="cuda")
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, y, ids=p.ids, scale=p.scale, base=p.base, u=u)
    want, bound, wu, bu = p.forward64(True, True)
    within(u, wu, bu)
    within(y, want, bound)
    # without u, scale and base
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, y, ids=p.ids)
    want, bound, _, _ = p.forward64(False, False)
    within(y, want, bound)


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pattern", ["mixed", "runs"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, pattern, dt):
    p = Problem(*size, pattern, dt)
    u = p.forward64(True, True)[2].float()
    out = {"grad_x": torch.full_like(p.x, float("nan")), "grad_a": torch.full_like(p.a, float("nan")),
           "grad_b": torch.full_like(p.b, float("nan"))}
    M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, base=p.gbase, **out)
    for k, (want, bound) in p.backward64(u, True, True).items():
        within(out[k], want, bound)
    # each gradient alone, without scale and base, gives the same as together
    for t in out.values():
        t.fill_(float("nan"))
    M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, **out)
    for k, (want, bound) in p.backward64(u, False, False).items():
        within(out[k], want, bound)
        alone = torch.full_like(out[k], float("nan"))
        M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, **{k: alone})
        assert torch.equal(alone, out[k])


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pattern", ["null", "last", "runs"])
@pytest.mark.parametrize("size", [(200, 256, 208, 8, 30), (256, 160, 96, 24, 16), (190, 129, 131, 50, 64), (61, 520, 72, 128, 5)],
                         ids=str)
def test_few_rows_of_one(size, pattern, dt):
    """Few rows to many adapters, of which one has all or most of them: several tiles of rows a workgroup."""
    p = Problem(*size, pattern, dt)
    y, u = torch.empty_like(p.base), torch.empty(size[0], size[3], device="cuda")
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, y, ids=p.ids, scale=p.scale, base=p.base, u=u)
    wy, ey, wu, eu = p.forward64(True, True)
    within(y, wy, ey)
    within(u, wu, eu)
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, p.base, ids=p.ids, scale=p.scale, base=p.base)
    assert torch.equal(p.base, y)                     # in place


# rows of x, W or u shorter than 16 bytes, the other dimension whole blocks of the kernels
SHORT = [(200, 4, 128, 2, 3), (300, 6, 512, 3, 2), (70, 3, 64, 1, 2), (40, 512, 3, 5, 2), (500, 1, 1, 7, 3), (1, 2, 256, 1, 1)]


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SHORT, ids=str)
def test_short_rows(size, dt):
    p = Problem(*size, "mixed" if size[0] > 1 else "null", dt)
    y, u = torch.empty_like(p.base), torch.empty(size[0], size[3], device="cuda")
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, y, ids=p.ids, scale=p.scale, base=p.base, u=u)
    wy, ey, wu, eu = p.forward64(True, True)
    within(y, wy, ey)
    within(u, wu, eu)
    out = {"grad_x": torch.empty_like(p.x), "grad_a": torch.empty_like(p.a), "grad_b": torch.empty_like(p.b)}
    M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, base=p.gbase, **out)
    for k, (want, bound) in p.backward64(u, True, True).items():
        within(out[k], want, bound)


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pattern", ["null", "none", "last"])
@pytest.mark.parametrize("size", [(5, 200, 70, 8, 3), (150, 384, 520, 20, 3)], ids=str)
def test_id_patterns(size, pattern, dt):
    p = Problem(*size, pattern, dt)
    y, u = torch.empty_like(p.base), torch.empty(size[0], size[3], device="cuda")
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, y, ids=p.ids, scale=p.scale, base=p.base, u=u)
    want, bound, wu, bu = p.forward64(True, True)
    within(u, wu, bu)
    within(y, want, bound)
    out = {"grad_x": torch.empty_like(p.x), "grad_a": torch.empty_like(p.a), "grad_b": torch.empty_like(p.b)}
    M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, base=p.gbase, **out)
    for k, (want, bound) in p.backward64(u, True, True).items():
        within(out[k], want, bound)
    if pattern == "none":
        assert torch.equal(y, p.base) and not u.any() and torch.equal(out["grad_x"], p.gbase)
        assert not out["grad_a"].any() and not out["grad_b"].any()


def test_rows_are_their_own():
    """NaN and infinity in one row, and in the weights of an adapter that no row
    has, touch nothing else; -0 and NaN of the base pass where there is no adapter."""
    for size in [(40, 300, 200, 16, 4), (200, 300, 200, 40, 4)]:
        for dt in (bf16, f32):
            p = Problem(*size, "mixed", dt)
            p.ids[p.ids == 3] = 1
            p.ids[7], p.ids[8], p.ids[9] = 0, 2, -1
            clean = torch.empty_like(p.base)
            M.mxfp4_adapter_fwd(p.x, p.a, p.b, clean, ids=p.ids, scale=p.scale, base=p.base)
            x, a, b, base = p.x.clone(), p.a.clone(), p.b.clone(), p.base.clone()
            x[7], x[8, 5], x[9] = float("nan"), float("inf"), float("nan")
            a[3], b[3] = float("nan"), float("inf")
            base[9, 0], base[9, 1] = -0.0, float("nan")
            y = torch.empty_like(p.base)
            M.mxfp4_adapter_fwd(x, a, b, y, ids=p.ids, scale=p.scale, base=base)
            rest = torch.ones(size[0], dtype=torch.bool)
            rest[[7, 8, 9]] = False
            rest = rest.cuda()
            assert torch.equal(y[rest], clean[rest])
            assert y[7].isnan().all() and not y[8].isfinite().any()
            as_int = torch.int16 if dt == bf16 else torch.int32
            assert torch.equal(y[9].view(as_int), base[9].view(as_int))
            # backward: the poisoned rows stay out of the other adapters' gradients
            u = torch.empty(size[0], size[3], device="cuda")
            M.mxfp4_adapter_fwd(p.x, p.a, p.b, clean, ids=p.ids, u=u)
            gy = p.gy.clone()
            gy[7], x[8] = float("nan"), p.x[8]
            got, want = ({"grad_x": torch.empty_like(p.x), "grad_a": torch.empty_like(p.a), "grad_b": torch.empty_like(p.b)}
                         for _ in range(2))
            M.mxfp4_adapter_bwd(gy, a, b, x=x, u=u, ids=p.ids, scale=p.scale, **got)
            M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, **want)
            keep = torch.arange(size[0], device="cuda") != 7
            assert torch.equal(got["grad_x"][keep], want["grad_x"][keep]) and got["grad_x"][7].isnan().all()
            for k in ("grad_a", "grad_b"):
                assert torch.equal(got[k][1:], want[k][1:]) and got[k][0].isnan().any()


def test_infinite_u():
    """An infinite u keeps its sign through the two halves."""
    for dt in (bf16, f32):
        for tokens in (3, 100):
            x = torch.ones(tokens, 64, dtype=dt, device="cuda")
            a = torch.zeros(1, 2, 64, dtype=dt, device="cuda")
            a[0, 0, 3], a[0, 1, 5] = float("inf"), 1.0
            b = torch.zeros(1, 40, 2, dtype=dt, device="cuda")
            b[0, :, 0] = torch.where(torch.arange(40, device="cuda") % 2 == 0, 2.0, -2.0).to(dt)
            b[0, :, 1] = 1.0
            y = torch.empty(tokens, 40, dtype=dt, device="cuda")
            M.mxfp4_adapter_fwd(x, a, b, y)
            assert (y[:, ::2] == float("inf")).all() and (y[:, 1::2] == -float("inf")).all()


@pytest.mark.parametrize("dt", [bf16, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 9, 140])
def test_strided_rows_and_alignment(tokens, dt):
    """x, base, y and the gradients as columns of wider matrices, starting at any
    element; what lies beside them stays as it was."""
    n_in, n_out, rank, adapters = 130, 260, 9, 3
    p = Problem(tokens, n_in, n_out, rank, adapters, "mixed", dt)

    def wide(t, left, right):
        w = torch.full((t.shape[0] + 2, left + t.shape[1] + right), 7.0, dtype=t.dtype, device="cuda")
        v = w[1:-1, left:left + t.shape[1]]
        v.copy_(t)
        return w, v

    def beside(w, v_shape, left):
        w = w.clone()
        w[1:-1, left:left + v_shape[1]] = 7.0
        return bool((w == 7.0).all())

    y0, u = torch.empty_like(p.base), torch.empty(tokens, rank, device="cuda")
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, y0, ids=p.ids, scale=p.scale, base=p.base, u=u)
    a1 = torch.empty(p.a.numel() + 1, dtype=dt, device="cuda")[1:].view_as(p.a).copy_(p.a)
    b1 = torch.empty(p.b.numel() + 3, dtype=dt, device="cuda")[3:].view_as(p.b).copy_(p.b)
    _, x = wide(p.x, 3, 2)
    _, base = wide(p.base, 1, 0)
    wy, y = wide(torch.zeros_like(p.base), 5, 4)
    M.mxfp4_adapter_fwd(x, a1, b1, y, ids=p.ids, scale=p.scale, base=base)
    assert torch.equal(y, y0) and beside(wy, y.shape, 5)
    # in place over base
    wb, base = wide(p.base, 1, 6)
    M.mxfp4_adapter_fwd(x, a1, b1, base, ids=p.ids, scale=p.scale, base=base)
    assert torch.equal(base, y0) and beside(wb, base.shape, 1)

    want = {"grad_x": torch.empty_like(p.x), "grad_a": torch.empty_like(p.a), "grad_b": torch.empty_like(p.b)}
    M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, base=p.gbase, **want)
    _, gy = wide(p.gy, 2, 5)
    wg, gx = wide(p.gbase, 7, 1)
    ga = torch.empty(p.a.numel() + 1, dtype=dt, device="cuda")[1:].view_as(p.a)
    gb = torch.empty(p.b.numel() + 1, dtype=dt, device="cuda")[1:].view_as(p.b)
    M.mxfp4_adapter_bwd(gy, a1, b1, x=x, u=u, ids=p.ids, scale=p.scale, base=gx, grad_x=gx, grad_a=ga, grad_b=gb)
    assert torch.equal(gx, want["grad_x"]) and beside(wg, gx.shape, 7)
    assert torch.equal(ga, want["grad_a"]) and torch.equal(gb, want["grad_b"])


def test_no_tokens():
    p = Problem(0, 64, 96, 4, 3, "mixed", bf16)
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, torch.empty_like(p.base), ids=p.ids)
    ga, gb = torch.full_like(p.a, 3.0), torch.full_like(p.b, 3.0)
    u = torch.empty(0, 4, device="cuda")
    M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, grad_x=torch.empty_like(p.x), grad_a=ga, grad_b=gb)
    assert not ga.any() and not gb.any()
    M.mxfp4_adapter_bwd(p.gy, p.a, p.b, ids=p.ids, grad_x=torch.empty_like(p.x))


def test_against_differences():
    """The gradients against central differences of the forward formula in fp32."""
    p = Problem(21, 48, 36, 5, 3, "mixed", f32)
    g = torch.Generator().manual_seed(5)

    def loss(x, a, b):
        y = torch.empty_like(p.base)
        M.mxfp4_adapter_fwd(x, a, b, y, ids=p.ids, scale=p.scale, base=p.base)
        return float((y.double() * p.gy.double()).sum())

    y, u = torch.empty_like(p.base), torch.empty(21, 5, device="cuda")
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, y, ids=p.ids, scale=p.scale, base=p.base, u=u)
    out = {"grad_x": torch.empty_like(p.x), "grad_a": torch.empty_like(p.a), "grad_b": torch.empty_like(p.b)}
    M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, **out)
    size = float((y.double().abs() * p.gy.double().abs()).sum())
    for k, i in (("grad_x", 0), ("grad_a", 1), ("grad_b", 2)):
        v = [p.x, p.a, p.b]
        d = torch.randn(v[i].shape, generator=g).cuda()
        h = 2.0 ** -6   # the loss is linear in each argument: only rounding is left
        lo, hi = list(v), list(v)
        lo[i], hi[i] = v[i] - h * d, v[i] + h * d
        slope = (loss(*hi) - loss(*lo)) / (2 * h)
        want = float((out[k].double() * d.double()).sum())
        # each fp32 y is off by (K + 2 r + 20) 2^-23 of its terms' magnitudes at most; `size` stands for them within 4
        assert abs(slope - want) <= 2 * 4 * size * (48 + 30) * E / (2 * h)


def test_many_adapters():
    """The backward pass at its limit of adapters, and more of them forward."""
    p = Problem(700, 40, 24, 2, 1024, "mixed", bf16)
    u = p.forward64(True, True)[2].float()
    out = {"grad_a": torch.empty_like(p.a), "grad_b": torch.empty_like(p.b)}
    M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, **out)
    want = p.backward64(u, True, True)
    for k in out:
        within(out[k], *want[k])
    p = Problem(90, 40, 24, 2, 3000, "mixed", bf16)
    y = torch.empty_like(p.base)
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, y, ids=p.ids, scale=p.scale, base=p.base)
    within(y, *p.forward64(True, True)[:2])


def test_long_training_batch():
    """Several pieces an adapter, in both orders of tokens."""
    for pattern in ("runs", "mixed"):
        p = Problem(9000, 160, 224, 16, 3, pattern, bf16)
        u = p.forward64(True, True)[2].float()
        out = {"grad_x": torch.empty_like(p.x), "grad_a": torch.empty_like(p.a), "grad_b": torch.empty_like(p.b)}
        M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, base=p.gbase, **out)
        for k, (want, bound) in p.backward64(u, True, True).items():
            within(out[k], want, bound)
        again = {k: torch.empty_like(t) for k, t in out.items()}
        M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, base=p.gbase, **again)
        assert all(torch.equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("tokens,ld", [(70, 1 << 25), (300, 1 << 23)])
def test_rows_far_apart(tokens, ld):
    """Columns of matrices whose rows lie more than 2^32 bytes from the first: the bits of the same rows together."""
    p = Problem(tokens, 64, 96, 8, 3, "mixed", bf16)
    far = torch.empty(tokens, ld, dtype=bf16, device="cuda")
    x, y, gy, gx = (far[:, 128 * k:128 * k + n] for k, n in enumerate((64, 96, 96, 64)))
    x.copy_(p.x)
    gy.copy_(p.gy)
    want, u = torch.empty_like(p.base), torch.empty(tokens, 8, device="cuda")
    wx, wa, wb = torch.empty_like(p.x), torch.empty_like(p.a), torch.empty_like(p.b)
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, want, ids=p.ids, base=p.base, u=u)
    M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, grad_x=wx, grad_a=wa, grad_b=wb)
    v, ga, gb = torch.empty_like(u), torch.empty_like(p.a), torch.empty_like(p.b)
    M.mxfp4_adapter_fwd(x, p.a, p.b, y, ids=p.ids, base=p.base, u=v)
    M.mxfp4_adapter_bwd(gy, p.a, p.b, x=x, u=u, ids=p.ids, grad_x=gx, grad_a=ga, grad_b=gb)
    for a, b in ((y, want), (v, u), (gx, wx), (ga, wa), (gb, wb)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [3, 300])
def test_weights_past_32_bits(tokens):
    """The last of adapters that together hold more than 2^32 bytes."""
    p = Problem(tokens, 8192, 1024, 128, 2, "mixed", bf16)
    a = torch.empty(2100, 128, 8192, dtype=bf16, device="cuda")
    b = torch.empty(2100, 1024, 128, dtype=bf16, device="cuda")
    a[[0, 2099]] = p.a
    b[[0, 2099]] = p.b
    ids = torch.where(p.ids == 1, 2099, torch.where(p.ids == 0, 0, -1)).to(torch.int32)
    want, y = torch.empty_like(p.base), torch.empty_like(p.base)
    M.mxfp4_adapter_fwd(p.x, p.a, p.b, want, ids=p.ids, base=p.base)
    M.mxfp4_adapter_fwd(p.x, a, b, y, ids=ids, base=p.base)
    # (how the long dimension is cut hangs on the number of adapters: two sums in fp32, rounded once each)
    bound = p.forward64(False, True)[1]
    within(y, want.double(), 2 * bound)


@pytest.mark.parametrize("tokens,adapters", [(4, 3), (300, 5)])
def test_streams_and_graphs(tokens, adapters):
    """On another stream and in replayed graphs with new inputs, the same bits."""
    p = Problem(tokens, 256, 320, 16, adapters, "mixed", bf16)
    y, u = torch.empty_like(p.base), torch.empty(tokens, 16, device="cuda")
    out = {"grad_x": torch.empty_like(p.x), "grad_a": torch.empty_like(p.a), "grad_b": torch.empty_like(p.b)}
    outs = [y, u, *out.values()]

    def step():
        M.mxfp4_adapter_fwd(p.x, p.a, p.b, y, ids=p.ids, scale=p.scale, base=p.base, u=u)
        M.mxfp4_adapter_bwd(p.gy, p.a, p.b, x=p.x, u=u, ids=p.ids, scale=p.scale, base=p.gbase, **out)

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (p.x, p.gy, p.base, p.gbase):
            t.normal_(generator=g)
        p.ids.random_(-1, adapters, generator=g)

    fill(0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    step()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(1, 5):
        fill(seed)
        step()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
        assert not all(torch.equal(a, b) for a, b in zip(first, outs))
