"""The grouped MX product with its epilogue where the 256 x 256 tiles run: alone,
with a tail of 128 x 128 tiles behind full rounds, and in bands for wide rows.
Operands, formulas and bounds are those of test_gpu_moe_product.

``form`` repeats the launcher's choice on the host, and every case says which
form it is meant for: a change of the choice fails here instead of leaving the
large tiles untested."""
import pytest
import torch

import test_gpu_moe_product as product

pytestmark = pytest.mark.gpu
M = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global M
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_fake_quantization_amd as mod
    mod._load()
    M = product.M = mod
    yield


def form(rows, counts, N, gated):
    """(form, 256 x 256 tiles, tail tiles' 256 x 256 units) of a call."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    G = len(counts) if counts else 1
    up = lambda a, b: -(-a // b)  # noqa: E731
    pieces = (rows // 64 + (G if counts else (rows % 64 > 0))) * up(N, 16 if gated else 32)
    if up(rows, min(G, rows)) <= 64 or pieces <= cus:
        return "rows", 0, 0
    rest = rows % 256
    if G == 1 and 0 < rest <= 64 and rows > 256 and rows // 256 * up(N, 256) <= 1024:
        rows, counts = rows - rest, None                     # the last rows have a launch of their own
    tiles_n = up(N, 128 if gated else 256)
    real = sum(up(c, 256) for c in (counts or [rows])) * tiles_n
    if tiles_n > 32:
        return "bands", real, 0
    tail = real % cus
    tail = tail if 2 * tail <= cus else 0
    return ("tiles + tail" if tail and real > tail else "tail" if tail else "tiles"), real - tail, tail


MIXED = [256, 70, 0, 300, 65, 255, 1, 512, 66, 130, 90, 257]      # 2002 rows in 14 M-tiles
HALVES = [300, 220]                                               # 520 rows in 3
ENDS = [256, 256, 600, 900, 1500, 1500, 2040]                     # cumulative, an empty group among them; 9 M-tiles


CASES = [
    # form, rows, counts, K, N, act, weights, output; scale rows are dword-aligned for K = 128, 256, 512
    ("tiles", 2002, MIXED, 96, 2500, "none", "e2m1", "bf16"),
    ("tiles", 2010, MIXED, 512, 2497, "gelu", "e2m1", "f32"),
    ("tiles", 2002, MIXED, 416, 2500, "relu", "e4m3", "bf16"),
    ("tiles", 2002, MIXED, 256, 2305, "silu", "e4m3", "f32"),
    ("tiles", 2002, MIXED, 96, 1250, "swiglu", "e2m1", "f32"),
    ("tiles", 2010, MIXED, 544, 1249, "geglu", "e2m1", "bf16"),
    ("tiles", 2002, MIXED, 160, 1280, "swiglu", "e4m3", "bf16"),
    ("tiles", 2002, MIXED, 512, 1250, "geglu", "e4m3", "f32"),
    ("tiles", 2600, None, 128, 4000, "silu", "e2m1", "bf16"),      # 40 last rows in a launch of their own
    ("tiles", 2600, [2600], 96, 2000, "swiglu", "e2m1", "f32"),
    ("tiles + tail", 2002, MIXED, 320, 4900, "silu", "e2m1", "bf16"),
    ("tiles + tail", 2002, MIXED, 96, 4900, "none", "e4m3", "f32"),
    ("tiles + tail", 2002, MIXED, 128, 2450, "swiglu", "e2m1", "bf16"),
    ("tiles + tail", 2002, MIXED, 96, 2450, "geglu", "e4m3", "bf16"),
    ("bands", 530, HALVES, 288, 8300, "gelu", "e2m1", "bf16"),
    ("bands", 520, HALVES, 96, 8300, "none", "e4m3", "f32"),
    ("bands", 530, HALVES, 128, 4201, "geglu", "e2m1", "f32"),
    ("bands", 520, HALVES, 352, 4200, "swiglu", "e4m3", "bf16"),
    ("bands", 530, None, 64, 8201, "silu", "e2m1", "bf16"),
]


@pytest.mark.parametrize("n", range(len(CASES)))
def test_exact(n):
    want, rows, counts, K, N, act, b_fmt, dtype = CASES[n]
    assert form(rows, counts, N, act in ("swiglu", "geglu"))[0] == want
    # all parts of the epilogue at once in most cases, each left out in some
    product.case(300 + n, counts, rows, K, N, act, b_fmt=b_fmt, bias=("groups", "one", None)[n % 3], res=n % 4 != 1,
                 keep_z=n % 5 != 3, dtype=dtype)


@pytest.mark.parametrize("act,N,a_block,b_block,a_fmt", [("silu", 4100, 128, 32, "e4m3"), ("geglu", 2050, 32, 128, "e5m2")])
def test_exact_with_cumulative_ends(act, N, a_block, b_block, a_fmt):
    counts = [b - a for a, b in zip([0] + ENDS, ENDS)]
    assert form(2050, counts, N, act == "geglu")[0] == "tiles"
    product.case(400 + N, counts, 2050, 256, N, act, a_fmt=a_fmt, a_block=a_block, b_block=b_block, bias="groups", res=True,
                 keep_z=True, dtype="bf16", list_type=0)


@pytest.mark.parametrize("act,N,dtype", [("gelu", 2500, "bf16"), ("swiglu", 1250, "f32"), ("swiglu", 1250, "bf16")])
def test_realistic_operands(act, N, dtype):
    assert form(2002, MIXED, N, act == "swiglu")[0] == "tiles"
    product.case(6, MIXED, 2002, 160, N, act, bias="groups", res=True, keep_z=True, dtype=dtype, exact=False)


@pytest.mark.parametrize("b_fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("N,want", [(2500, "tiles"), (4900, "tiles + tail"), (8300, "bands")])
def test_same_bits_as_the_plain_product(N, want, b_fmt):
    """Without an epilogue: the plain product's result, bit for bit."""
    rows, K = 2002, 544
    assert form(rows, MIXED, N, False)[0] == want
    G, g = len(MIXED), torch.Generator().manual_seed(N)
    a, asc, _ = product.mx_codes(g, rows, K, "e4m3", 32, False, K)
    kb = K // 2 if b_fmt == "e2m1" else K
    b, bsc, _ = product.mx_codes(g, G * N, K, b_fmt, 32, False, kb)
    gl = torch.tensor(MIXED, device="cuda")
    args = [a.cuda(), asc.cuda(), b.view(G, N, -1).cuda(), bsc.view(G, N, -1).cuda()]
    for dt in (torch.bfloat16, torch.float32):
        c0, c1 = (torch.zeros(rows, N, dtype=dt, device="cuda") for _ in range(2))
        M.mxfp4_grouped_matmul(*args, c0, group_list=gl, b_fmt=b_fmt)
        M.mxfp4_grouped_matmul_act(*args, c1, group_list=gl, b_fmt=b_fmt)
        assert torch.equal(c0, c1)
