"""The gated product and its gradient where gate's sigmoid is near or below fp32's smallest normal number and up, or the gradient,
is near its largest: finite operands, results that bf16 can hold.

sigmoid(g) is then off by a few of its last places, which are 2^-149 there (exp's result, a product: 4 2^-149 covers them),
beside the relative bounds of expert_util."""
import pytest
import torch

import expert_util as xu
from expert_util import BF16

pytestmark = pytest.mark.gpu
LAST = 4 * 2.0 ** -149


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    return lm


def gates(R):
    """From where sigmoid is 0 in fp32 to where it is 1."""
    return torch.linspace(-110, 110, R, device="cuda").to(BF16)


def ups(N):
    sign = torch.where(torch.arange(N, device="cuda") % 2 == 0, 1.0, -1.0)
    return (torch.logspace(28, 38.4, N, device="cuda", dtype=torch.float64) * sign).to(BF16)


def compare(got, want, tol):
    fits = want.abs() < 3e38
    off = (got.double() - want).abs()
    bad = fits & ~(off <= tol)
    assert bool(fits.any()) and not bool(bad.any()), f"{int(bad.sum())} of {int(fits.sum())}, at {bad.nonzero()[0].tolist()}: " \
        f"{float(got[bad][0])} for {float(want[bad][0])}"


# tiles of few rows, of 128 rows, pairs of CTAs
SIZES = [(120, 64), (300, 1280), (3000, 4096)]


@pytest.mark.parametrize("R,N", SIZES)
def test_gated_ffn(lm, R, N):
    x, wg, wu = (torch.zeros(n, 8, dtype=BF16, device="cuda") for n in (R, N, N))
    x[:, 0], x[:, 1], wg[:, 0], wu[:, 1] = gates(R), 1, 1, ups(N)
    h = torch.zeros(R, N, dtype=BF16, device="cuda")
    lm.lmoe_gated_ffn(x, wg, wu, h)
    # (each sum is one product, exact)
    g, u = gates(R).double()[:, None], ups(N).double()[None]
    s = torch.sigmoid(g)
    want = g * s * u
    tol = xu.rounded(want, 2.0 ** -19 * (1 + g.abs()) * want.abs() + (g * u).abs() * LAST, BF16)
    compare(h, want, tol)


@pytest.mark.parametrize("R,N", SIZES)
@pytest.mark.parametrize("size", [2.0 ** -20, 1.0, 2.0 ** 20], ids=["small", "one", "large"])
def test_gated_ffn_grad(lm, R, N, size):
    dy, wd = torch.zeros(R, 8, dtype=BF16, device="cuda"), torch.zeros(8, N, dtype=BF16, device="cuda")
    dy[:, 3], wd[3] = size, 1.5
    g, u = gates(R)[:, None].expand(R, N).contiguous(), ups(N)[None].expand(R, N).contiguous()
    dg, du = torch.zeros_like(g), torch.zeros_like(u)
    lm.lmoe_gated_ffn_grad(dy, wd, g, u, dg, du)
    G, U, dh = g.double(), u.double(), 1.5 * size
    s = torch.sigmoid(G)
    f = s + G * s * torch.sigmoid(-G)
    eg = 2.0 ** -19 * (1 + G.abs()) ** 2 * s + (1 + G.abs()) * LAST
    compare(dg, dh * U * f, xu.rounded(dh * U * f, dh * U.abs() * eg, BF16))
    eu = 2.0 ** -19 * (1 + G.abs()) * (G * s).abs() + G.abs() * LAST
    compare(du, dh * G * s, xu.rounded(dh * G * s, dh * eu, BF16))
