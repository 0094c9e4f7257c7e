"""gelu and its slope in fp32 to the accuracy of fp32, tails included.

Bound, with u = 2^-24: Phi(-|x|) = exp(-x^2 / 2) Q(|x|).  The exponent's argument
carries up to 4 roundings and its factor log2 e 0.2 u, so |x|^2 / 2 * 4.4 u in the
result; the hardware's 2^x and reciprocal 2 u each, the polynomial's fit 0.2 u, its
rounding and the products 5 u.  So the tail is known to TAIL = (2.2 x^2 + 9.2) u
of itself, 1 - tail to u more, and the product with x to u of the result."""
import numpy as np
import pytest
import torch
from scipy.special import erfc

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_fake_quantization_amd as mod
    mod._load()
    return mod


def arguments():
    g = torch.Generator().manual_seed(4)
    x = torch.cat([torch.linspace(-9, 9, 3000), 3 * torch.randn(1000, generator=g), torch.tensor(
        [0.0, -0.0, 1e-30, -1e-30, 2.0 ** -24, -2.0 ** -24, 40.0, -40.0])])
    return x[:4000].float() if x.numel() < 4000 else x.float()


def exact(x):
    """Phi, gelu and slope in 64 bits, and the bounds of the computed gelu and slope."""
    x = x.double().numpy()
    phi = np.exp(-x * x / 2) / (2 * np.pi) ** 0.5
    cdf = 0.5 * erfc(-x * 0.5 ** 0.5)
    rel = (2.2 * x * x + 9.2) * U
    # below 2^-126 the exponential may be flushed to zero
    tail = np.where(x > 0, 0.5 * erfc(np.abs(x) * 0.5 ** 0.5), cdf)
    dcdf = tail * rel + np.where(x > 0, U, 0.0) + 2.0 ** -126
    value, slope = x * cdf, cdf + x * phi
    dvalue = np.abs(x) * dcdf + 2 * U * np.abs(value) + 2.0 ** -149
    dslope = dcdf + np.abs(x) * (phi * rel + 2.0 ** -126) + 2 * U * np.abs(slope)
    return value, slope, dvalue, dslope


def run(M, x):
    """gelu(x) as a product's epilogue (zero products, x as the bias), and its slope."""
    n = x.numel()
    zero = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    c = torch.empty(1, n, device="cuda")
    M.mxfp4_grouped_matmul_act(zero(1, 32), zero(1, 1) + 127, zero(n, 16), zero(n, 1) + 127, c, act="gelu", bias=x.cuda())
    d = torch.empty(1, n, device="cuda")
    M.mxfp4_act_bwd(torch.ones(1, n, device="cuda"), x.cuda()[None], d, act="gelu")
    return c[0].cpu().double().numpy(), d[0].cpu().double().numpy()


def test_gelu_and_its_slope(M):
    x = arguments()
    got, slope_got = run(M, x)
    value, slope, dvalue, dslope = exact(x)
    assert (np.abs(got - value) <= dvalue).all(), x[np.abs(got - value) > dvalue][:9]
    assert (np.abs(slope_got - slope) <= dslope).all(), x[np.abs(slope_got - slope) > dslope][:9]


def test_mean_error_over_normal_arguments(M):
    """The whole vector's error against the plain formula's in fp32."""
    x = torch.randn(200000, generator=torch.Generator().manual_seed(1))
    got, slope_got = run(M, x)
    value, slope, _, _ = exact(x)
    plain = (x * 0.5 * (1 + torch.erf(x * 0.5 ** 0.5))).double().numpy()
    rms = lambda e, v: np.sqrt((e ** 2).sum() / (v ** 2).sum())  # noqa: E731
    mine, theirs = rms(got - value, value), rms(plain - value, value)
    print(f"gelu: {mine:.2e}, plain {theirs:.2e}; slope: {rms(slope_got - slope, slope):.2e}")
    # an exponential, a reciprocal, a polynomial and two products, u / sqrt 3 each at most
    assert mine <= U and rms(slope_got - slope, slope) <= U


def test_infinite_arguments(M):
    inf = float("inf")
    got, _ = run(M, torch.tensor([inf, float("nan"), 3.0e38, -3.0e38, 1e20, -1e20]))
    assert got[0] == inf and np.isnan(got[1]) and got[2] == np.float32(3.0e38) and got[3] == 0
    assert got[4] == np.float32(1e20) and got[5] == 0
