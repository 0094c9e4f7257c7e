"""The grouped MX product with its epilogue, and the epilogue's backward, on
the GPU against 64-bit formulas.

The operands of the exact cases are small multiples of powers of two, so that
every partial sum is exact in the matrix cores and in fp32: z must be equal
(fp32) or equal after rounding (bf16).  An activation's error, for an argument
x: the hardware exponential's argument is rounded by |x| 2^-24, its result, the
reciprocal and the products by a few 2^-23, the normal distribution function
is within 1.5e-7 / 2 (+ a few 2^-24); so |act error| <= |x| ((|x| + 8) 2^-23 +
1.5e-7) =: act_tol(x), and as much, without the factor |x|, for the slope times
(1 + |x|).  bf16 outputs add 2^-8 of their value."""
import numpy as np
import pytest
import torch

from gpu_util import Guarded
from mx_tolerance import mx_matmul_bound

pytestmark = pytest.mark.gpu
M = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global M
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_fake_quantization_amd as mod
    mod._load()
    M = mod
    yield


FP4 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def act_tol(x):
    return x.abs() * ((x.abs() + 8) * 2.0 ** -23 + 1.5e-7)


def act64(x, name):
    if name == "relu":
        return x.clamp(min=0), (x > 0).double()
    if name in ("silu", "swiglu"):
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    if name in ("gelu", "geglu"):
        cdf = 0.5 * torch.erfc(-x * 0.5 ** 0.5)
        return x * cdf, cdf + x * torch.exp(-x * x / 2) / (2 * np.pi) ** 0.5
    return x, torch.ones_like(x)


def mx_codes(g, rows, K, fmt, block, exact, ld):
    """(codes [rows, ld], scales, values [rows, K] in 64 bits); ld bytes a row."""
    nb = -(-K // block)
    sc = torch.randint(126, 129, (rows, nb), generator=g) if exact else torch.randint(118, 124, (rows, nb), generator=g)
    if fmt == "e2m1":
        code = torch.randint(16, (rows, K), generator=g)
        v = FP4[code]
        data = code[:, 0::2] | (code[:, 1::2] << 4)
    else:
        t8 = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
        x = torch.randint(-2, 3, (rows, K), generator=g).float() if exact else 4 * torch.randn(rows, K, generator=g)
        q = x.to(t8)
        v, data = q.double(), q.view(torch.uint8).long()
    v = v * torch.ldexp(torch.ones(rows, nb, dtype=torch.float64), sc - 127).repeat_interleave(block, 1)[:, :K]
    out = torch.full((rows, ld), 0xA5, dtype=torch.uint8)
    out[:, :data.shape[1]] = data.to(torch.uint8)
    return out, sc.to(torch.uint8).contiguous(), v


def case(seed, counts, rows, K, N, act, a_fmt="e4m3", b_fmt="e2m1", a_block=32, b_block=32, bias=None, res=False,
         keep_z=False, dtype="f32", exact=True, list_type=1):
    """Runs one product and checks everything it writes."""
    g = torch.Generator().manual_seed(seed)
    gated = act in ("swiglu", "geglu")
    nb, G = (2 * N if gated else N), max(1, len(counts or [1]))
    lda = -(-K // 16) * 16 + 16
    kb = K // 2 if b_fmt == "e2m1" else K
    ldb = -(-kb // 16) * 16
    a, asc, av = mx_codes(g, rows, K, a_fmt, a_block, exact, lda)
    bs = [mx_codes(g, nb, K, b_fmt, b_block, exact, ldb) for _ in range(G)]
    b, bsc = torch.stack([t[0] for t in bs]), torch.stack([t[1] for t in bs])
    dt = DT[dtype]
    bias_t = None
    if bias == "groups":
        bias_t = torch.randint(-8, 9, (G, nb), generator=g).float() / 4
    elif bias == "one":
        bias_t = torch.randint(-8, 9, (nb,), generator=g).float() / 4
    res_t = torch.randn(rows, N, generator=g).to(dt) if res else None
    ends = [rows] if counts is None else list(np.cumsum(counts))
    starts = [0] + ends[:-1]
    total = ends[-1]
    c, z = Guarded((rows, N), dt), Guarded((rows, nb), dt) if keep_z else None
    old = c.t.clone()
    gl = None
    if counts is not None:
        gl = torch.tensor(counts if list_type == 1 else ends, dtype=torch.int64, device="cuda")
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    M.mxfp4_grouped_matmul_act(cu(a), cu(asc), cu(b), cu(bsc), c.t, group_list=gl, act=act, bias=cu(bias_t),
                               residual=cu(res_t), z=z.t if z else None, K=K, group_list_type=list_type, a_fmt=a_fmt,
                               b_fmt=b_fmt, a_block=a_block, b_block=b_block)
    torch.cuda.synchronize()
    c.check_tail()
    if z:
        z.check_tail()
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    got = c.t.cpu().double()
    assert torch.equal(c.t[total:].view(torch.uint8), old[total:].view(torch.uint8))      # rows of no group
    for e in range(G):
        lo, hi = starts[e], ends[e]
        if lo == hi:
            continue
        w = bs[e][2]
        zz = av[lo:hi] @ w.t()
        bound = torch.zeros_like(zz) if exact else torch.from_numpy(
            mx_matmul_bound(av[lo:hi].numpy(), w.numpy()))
        if bias_t is not None:
            zz = zz + (bias_t[e] if bias_t.dim() == 2 else bias_t).double()
        if z:
            zg = z.t[lo:hi].cpu()
            if exact:
                assert torch.equal(zg, zz.float().to(dt))
            else:
                assert ((zg.double() - zz).abs() <= bound + half * zz.abs()).all()
        x = zz[:, :N]
        want, slope = act64(x, act)
        err = (act_tol(x) if act not in ("none", "relu") else 0) + bound[:, :N] * 1.2
        if gated:
            up = zz[:, N:]
            err = err * up.abs() + bound[:, N:] * (want.abs() + bound[:, :N])
            want = want * up
        if res:
            want = want + res_t[lo:hi].double()
        assert ((got[lo:hi] - want).abs() <= err + half * want.abs() + 2.0 ** -22 * x.abs()).all(), (e, lo, hi)
    if res:                                                  # c over the residual
        c2 = cu(res_t)
        M.mxfp4_grouped_matmul_act(cu(a), cu(asc), cu(b), cu(bsc), c2, group_list=gl, act=act, bias=cu(bias_t),
                                   residual=c2, K=K, group_list_type=list_type, a_fmt=a_fmt, b_fmt=b_fmt,
                                   a_block=a_block, b_block=b_block)
        assert torch.equal(c2[:total], c.t[:total])


# few rows: the forms for 16, 32 and 64 rows a tile
FEW = [
    (None, 1, 32, 16), (None, 1, 7168, 33), (None, 5, 96, 1), (None, 16, 128, 64), (None, 17, 256, 47),
    (None, 64, 288, 40), (None, 33, 2048, 96), ([1, 0, 1, 1], 3, 512, 48), ([0, 8, 0, 0, 3], 11, 1056, 50),
    ([0, 0], 4, 64, 32), ([16, 1, 17, 30], 66, 544, 35), ([64, 65, 1, 0, 40], 170, 224, 72),
    ([2] * 70 + [0] * 10, 150, 160, 20), ([7, 9], 20, 768, 130)]


@pytest.mark.parametrize("n", range(len(FEW)))
@pytest.mark.parametrize("act", ["none", "swiglu", "silu"])
def test_few_rows_exact(n, act):
    counts, rows, K, N = FEW[n]
    case(10 + n, counts, rows, K, N, act, bias="groups" if n % 2 else "one", res=n % 3 == 0, keep_z=n % 3 != 1,
         dtype="bf16" if n % 4 == 1 else "f32")


# few rows, so many columns that a wave takes the whole K of its own: 16, 32 and
# 64 rows a workgroup, one slab of K and several, the last one partial, odd
# columns, rows past the total
WIDE16, WIDE32, WIDE64 = [17, 0, 33, 16, 1, 40], [40, 0, 64, 33, 1, 70, 65], [64, 65, 1, 0, 120]


@pytest.mark.parametrize("counts,rows,K,N,act,b_fmt,b_block", [
    (WIDE16, 107, 1312, 11001, "none", "e2m1", 32), (WIDE16, 108, 288, 5471, "swiglu", "e2m1", 32),
    (WIDE16, 107, 32, 11001, "relu", "e2m1", 32), (WIDE16, 107, 288, 11001, "none", "e4m3", 32),
    (WIDE16, 107, 1184, 5471, "swiglu", "e2m1", 128), (WIDE32, 276, 608, 8777, "gelu", "e2m1", 32),
    (WIDE32, 273, 288, 4390, "geglu", "e4m3", 32), (WIDE64, 250, 608, 16390, "none", "e2m1", 32),
    (WIDE64, 253, 1056, 8210, "swiglu", "e2m1", 32)])
def test_few_rows_of_many_columns_exact(counts, rows, K, N, act, b_fmt, b_block):
    case(rows + K, counts, rows, K, N, act, b_fmt=b_fmt, b_block=b_block, bias="groups", res=K == 1312, keep_z=True,
         dtype="bf16" if N % 2 else "f32")


# many rows: whole and ragged tiles, the tail launch, odd columns
MANY = [
    (None, 257, 256, 256, "relu"), (None, 300, 128, 100, "none"), (None, 600, 416, 257, "gelu"),
    ([300, 0, 212], 512, 384, 129, "swiglu"), ([256, 256], 512, 512, 128, "swiglu"), ([130, 1, 400], 540, 160, 64, "geglu"),
    ([0, 700, 3], 703, 96, 515, "silu"), (None, 2000, 32, 31, "swiglu"), ([1000, 500], 1500, 1024, 2100, "none"),
    ([200, 90, 310], 600, 288, 300, "geglu")]


@pytest.mark.parametrize("n", range(len(MANY)))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_exact(n, dtype):
    counts, rows, K, N, act = MANY[n]
    case(50 + n, counts, rows, K, N, act, bias=(None, "one", "groups")[n % 3], res=n % 2 == 0, keep_z=n % 3 != 2,
         dtype=dtype)


# as many rows, and columns enough for the tiles
TILES = [
    (None, 257, 256, 2100, "relu"), (None, 600, 416, 1025, "gelu"), ([300, 0, 212], 512, 384, 1030, "swiglu"),
    ([130, 1, 400], 540, 160, 1060, "geglu"), ([0, 700, 3], 703, 96, 1315, "silu"), (None, 2000, 32, 331, "swiglu"),
    ([200, 90, 310], 603, 288, 900, "geglu")]


@pytest.mark.parametrize("n", range(len(TILES)))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tiles_exact(n, dtype):
    counts, rows, K, N, act = TILES[n]
    case(150 + n, counts, rows, K, N, act, bias=(None, "one", "groups")[n % 3], res=n % 2 == 0, keep_z=n % 3 != 2,
         dtype=dtype)


@pytest.mark.parametrize("rows,counts,list_type", [(257, [257], 1), (300, [299], 1), (320, [250], 0), (290, [0], 1),
                                                   (528, [513], 0)])
@pytest.mark.parametrize("act,N", [("none", 2111), ("geglu", 1063)])
def test_tiles_of_one_group_with_few_last_rows(rows, counts, list_type, act, N):
    case(rows + 1, counts, rows, 320, N, act, bias="groups", res=True, keep_z=True, dtype="bf16", list_type=list_type)


@pytest.mark.parametrize("a_fmt,b_fmt,a_block,b_block", [
    ("e5m2", "e2m1", 32, 32), ("e4m3", "e4m3", 32, 32), ("e4m3", "e2m1", 128, 128), ("e5m2", "e4m3", 128, 32),
    ("e4m3", "e4m3", 32, 128)])
@pytest.mark.parametrize("K,act", [(96, "swiglu"), (640, "none"), (416, "gelu")])
def test_tiles_of_formats_and_blocks(a_fmt, b_fmt, a_block, b_block, K, act):
    case(K, [200, 130], 330, K, 1510, act, a_fmt, b_fmt, a_block, b_block, bias="groups", keep_z=True, dtype="f32",
         list_type=K // 96 % 2)


@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tiles_of_realistic_operands(act, dtype):
    case(4, [260, 140], 400, 512, 1200, act, bias="one", res=True, keep_z=True, dtype=dtype, exact=False)


# one group whose last rows have a launch of their own, and a list that ends
# before, inside and after them
@pytest.mark.parametrize("rows,counts,list_type", [
    (257, [257], 1), (300, [300], 0), (300, [299], 1), (320, [256], 1), (320, [250], 0), (272, [260], 1), (290, [0], 1),
    (528, [513], 0)])
@pytest.mark.parametrize("act", ["none", "geglu"])
def test_one_group_with_few_last_rows(rows, counts, list_type, act):
    case(rows, counts, rows, 320, 67, act, bias="groups", res=True, keep_z=True, dtype="bf16", list_type=list_type)


@pytest.mark.parametrize("rows,counts", [(6, [2, 0, 4]), (70, [30, 40]), (330, [200, 130])])
@pytest.mark.parametrize("a_fmt,b_fmt,a_block,b_block", [
    ("e5m2", "e2m1", 32, 32), ("e4m3", "e4m3", 32, 32), ("e4m3", "e2m1", 128, 128), ("e5m2", "e4m3", 128, 32),
    ("e4m3", "e4m3", 32, 128)])
def test_formats_and_blocks(rows, counts, a_fmt, b_fmt, a_block, b_block):
    for K, act in ((96, "swiglu"), (640, "none"), (416, "gelu")):
        case(rows + K, counts, rows, K, 70, act, a_fmt, b_fmt, a_block, b_block, bias="groups", keep_z=True,
             dtype="f32", list_type=K // 96 % 2)


@pytest.mark.parametrize("rows,counts", [(9, [4, 5]), (90, [50, 40]), (400, [260, 140])])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_realistic_operands(rows, counts, act, dtype):
    case(3, counts, rows, 512, 96, act, bias="one", res=True, keep_z=True, dtype=dtype, exact=False)


def test_same_bits_as_the_plain_product():
    """Without an epilogue, in tiles (many rows and columns): the plain
    product's result, bit for bit."""
    g = torch.Generator().manual_seed(2)
    a, asc, _ = mx_codes(g, 900, 512, "e4m3", 32, False, 512)
    b, bsc, _ = mx_codes(g, 2 * 1100, 512, "e2m1", 32, False, 256)
    gl = torch.tensor([500, 400], device="cuda")
    args = [a.cuda(), asc.cuda(), b.view(2, 1100, -1).cuda(), bsc.view(2, 1100, -1).cuda()]
    for dt in (torch.bfloat16, torch.float32):
        c0, c1 = (torch.zeros(900, 1100, dtype=dt, device="cuda") for _ in range(2))
        M.mxfp4_grouped_matmul(*args, c0, group_list=gl)
        M.mxfp4_grouped_matmul_act(*args, c1, group_list=gl)
        assert torch.equal(c0, c1)


def test_extreme_arguments():
    """Large |z|: silu and gelu reach 0 and z without NaN."""
    v = torch.tensor([0.0, 6.0, 96.0, 384.0, 1e4, -6.0, -96.0, -384.0, -1e4], dtype=torch.float32)
    a = torch.zeros(v.numel(), 32, dtype=torch.uint8, device="cuda")
    sc = torch.full((v.numel(), 1), 127, dtype=torch.uint8, device="cuda")
    b = torch.zeros(v.numel(), 16, dtype=torch.uint8, device="cuda")
    for act in ("silu", "gelu", "relu"):
        c = torch.empty(v.numel(), v.numel(), device="cuda")
        M.mxfp4_grouped_matmul_act(a, sc, b, sc, c, act=act, bias=v.cuda())
        want = act64(v.double(), act)[0]
        assert ((c[0].cpu().double() - want).abs() <= act_tol(v.double())).all()
        dz = torch.empty_like(c)
        M.mxfp4_act_bwd(torch.ones_like(c), v.cuda().expand_as(c).contiguous(), dz, act=act)
        slope = act64(v.double(), act)[1]
        tol = (1 + v.double().abs()) * ((v.double().abs() + 8) * 2.0 ** -23 + 1.5e-7)
        assert ((dz[0].cpu().double() - slope).abs() <= tol).all()


# ---- the epilogue's backward --------------------------------------------------------

BWD = [(None, 1, 1), (None, 3, 7), (None, 64, 32), ([3, 0, 61, 1], 65, 33), ([64, 65, 0, 130], 260, 100),
       ([0, 0, 5], 9, 2049), (None, 129, 4096), ([500, 12], 512, 8), ([10] * 40, 400, 72)]


@pytest.mark.parametrize("n", range(len(BWD)))
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_act_backward(n, act, dtype):
    counts, rows, cols = BWD[n]
    dt = DT[dtype]
    g = torch.Generator().manual_seed(n)
    gated = act in ("swiglu", "geglu")
    zc = cols * (2 if gated else 1)
    z, dc = (2 * torch.randn(rows, zc, generator=g)).to(dt), torch.randn(rows, cols, generator=g).to(dt)
    G = 1 if counts is None else len(counts)
    ends = [rows] if counts is None else list(np.cumsum(counts))
    dz, db = Guarded((rows, zc), dt), Guarded((G, zc), torch.float32)
    old = dz.t.clone()
    gl = None if counts is None else torch.tensor(counts, device="cuda")
    M.mxfp4_act_bwd(dc.cuda(), z.cuda(), dz.t, act=act, grad_bias=db.t, group_list=gl)
    torch.cuda.synchronize()
    dz.check_tail()
    db.check_tail()
    x, d = z.double()[:, :cols], dc.double()
    f, slope = act64(x, act)
    tol = (1 + x.abs()) * ((x.abs() + 8) * 2.0 ** -23 + 1.5e-7) * d.abs()
    if gated:
        up = z.double()[:, cols:]
        want = torch.cat([d * up * slope, d * f], -1)
        tol = torch.cat([tol * up.abs(), tol], -1)
    else:
        want = d * slope
    if act in ("none", "relu"):
        tol = torch.zeros_like(tol)
    tol = tol + 2.0 ** -22 * want.abs()
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    total = ends[-1]
    assert ((dz.t.cpu().double() - want).abs() <= tol + half * want.abs())[:total].all()
    assert torch.equal(dz.t[total:].view(torch.uint8), old[total:].view(torch.uint8))
    for e, (lo, hi) in enumerate(zip([0] + ends[:-1], ends)):
        s, size = want[lo:hi].sum(0), want[lo:hi].abs().sum(0)
        assert ((db.t[e].cpu().double() - s).abs() <= tol[lo:hi].sum(0) + (hi - lo + 8) * 2.0 ** -23 * size).all()
    # without the bias gradient; in place without a gate; twice the same bits
    dz2, db2 = torch.zeros(rows, zc, dtype=dt, device="cuda"), torch.zeros(G, zc, device="cuda")
    M.mxfp4_act_bwd(dc.cuda(), z.cuda(), dz2, act=act, group_list=gl)
    assert torch.equal(dz2[:total], dz.t[:total])
    if not gated:
        z2 = z.cuda()
        M.mxfp4_act_bwd(dc.cuda(), z2, z2, act=act, group_list=gl)
        assert torch.equal(z2[:total], dz.t[:total])
    M.mxfp4_act_bwd(dc.cuda(), z.cuda(), dz2, act=act, grad_bias=db2, group_list=gl)
    assert torch.equal(db2, db.t)


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
def test_act_backward_against_differences(act):
    """Central differences of the 64-bit activation."""
    g = torch.Generator().manual_seed(1)
    gated = act in ("swiglu", "geglu")
    z, dc = torch.randn(6, 20 if gated else 10, generator=g), torch.randn(6, 10, generator=g)
    dz = torch.empty_like(z, device="cuda")
    M.mxfp4_act_bwd(dc.cuda(), z.cuda(), dz, act=act)

    def out(zz):
        return act64(zz[:, :10], act)[0] * (zz[:, 10:] if gated else 1.0)

    eps = 1e-5
    for j in range(z.shape[1]):
        a, b = z.double(), z.double()
        a[:, j] += eps
        b[:, j] -= eps
        d = ((out(a) - out(b)) * dc.double()).sum(1) / (2 * eps)
        # third derivatives of order 1 times |dc up| <= 16, 64-bit rounding / eps, and the slope's own error
        assert ((dz[:, j].cpu().double() - d).abs() <= 16 * (eps ** 2 + 12 * 2.0 ** -23 + 3e-7)).all()


def test_empty_products():
    e = lambda *s, dtype=torch.uint8: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    c = e(0, 32, dtype=torch.bfloat16)
    M.mxfp4_grouped_matmul_act(e(0, 64), e(0, 2), e(32, 32), e(32, 2), c)
    db = torch.ones(3, 16, device="cuda")
    z = e(0, 16, dtype=torch.float32)
    M.mxfp4_act_bwd(z, z, torch.empty_like(z), grad_bias=db, group_list=torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert (db == 0).all()
