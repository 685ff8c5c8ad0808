"""How exact the bf16 experts' sums are, by their length and by each way they are taken: tiles of 32 and 128 rows, pairs of
CTAs, reductions shared by a cluster, two pairs of operands, results that are added to.  The bounds of expert_util allow any order
of fp32 additions; these hold what the operators promise beyond that.

An MMA adds 16 products to a running sum, and cuts the 17 terms at the sum's last bit: at most 17 2^-23 of it.  For products of one sign
the running sum grows evenly, so a chunk of 48 MMAs loses at most 17 2^-23 (1 + .. + 48) / 48 = 5e-5 of itself (CUT), and so does the
result, whatever its length; each of the n chunks is added with a rounding of at most 2^-24 of the sum so far, n 2^-25 in all.
In the 2-norm over many results the cuts are spread evenly over a last place (1 / sqrt 3 of it in the mean square), which is 0.74
2^-23 of a value in the mean square.  Random signs: the running sum is sqrt(j / 48) of the chunk's after j MMAs, and
0.58 0.74 2^-23 times the sum of these, 32.4, is 1.7e-6; chunks are independent.  One sign: 24.5 in place of 32.4, 1.3e-6.  NORM is above
both.  A sum that does not end leaves 4.4e-6 after 4096 products already."""
import pytest
import torch

import expert_util as xu
from expert_util import BF16

pytestmark = pytest.mark.gpu
F32 = torch.float32
CUT = 17 * 2.0 ** -23 * 24.5
NORM = 2.0 ** -19
SAME = pytest.mark.parametrize("same", [False, True], ids=["random", "one_sign"])


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    return lm


def values(shape, seed, same, std=1.0):
    t = torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * std
    return (t.abs() if same else t).to(BF16)


def mm(a, w, transposed=False):
    """a w^T, or a w, in 64 bits, a piece of the reduction at a time."""
    out, step = 0, 1 << 15
    for k in range(0, a.shape[1], step):
        m = w[k:k + step].double() if transposed else w[:, k:k + step].double().t()
        out = out + a[:, k:k + step].double() @ m
    return out


def dwx(dy, x):
    out, step = 0, 1 << 19
    for r in range(0, dy.shape[0], step):
        out = out + dy[r:r + step].double().t() @ x[r:r + step].double()
    return out


def off(y, want):
    return float((y.double() - want).norm() / want.norm())


def half_place(v):
    """Half of bf16's last place of each value."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -120))) - 8)


def within(y, want, tol, what=""):
    """y (bf16) is the rounding of something within tol of want."""
    d = (y.double() - want).abs() - half_place(want) - tol - tol.clamp_min(0) * 2.0 ** -7
    assert float(d.max()) <= 0, f"{what}: {float(d.max()):.3g} past the bound, {int((d > 0).sum())} of {d.numel()}, " \
                                f"mean {float(((y.double() - want) / want).mean()):.3g} of the result"


def lost(want, products):
    """The bound of a sum of one sign's products: cuts and additions of its chunks."""
    return want.abs() * (CUT + (products / 768 + 1) * 2.0 ** -25)


# (rows, N): tiles of 32 rows by a cluster and alone, of 128 rows by a cluster and alone, pairs of CTAs
TILES = [(8, 256), (16, 16384), (200, 1024), (512, 4096), (512, 8192)]


@SAME
@pytest.mark.parametrize("K", [768, 4096, 65536])
@pytest.mark.parametrize("R,N", TILES)
@pytest.mark.parametrize("transposed", [False, True], ids=["nt", "nn"])
def test_fp32_products(lm, R, N, K, transposed, same):
    a, w = values((R, K), 1, same), values((K, N) if transposed else (N, K), 2, same)
    y = torch.zeros(R, N, device="cuda")
    lm.lmoe_matmul_bf16(a, w, y, transposed=transposed)
    assert off(y, mm(a, w, transposed)) <= NORM


@SAME
@pytest.mark.parametrize("N", [392, 2048])
def test_fp32_products_of_uneven_experts(lm, N, same):
    K, c = 4096, [300, 0, 5, 412, 128, 700, 129]
    o = xu.offsets_of(c)
    a, w, w2 = values((sum(c), K), 1, same), values((len(c), N, K), 2, same), values((len(c), N, K), 3, same)
    y = torch.zeros(sum(c), N, device="cuda")
    lm.lmoe_matmul_bf16(a, w, y, offsets=o, a2=a, w2=w2)
    for e, (lo, hi) in enumerate(xu.groups(o, sum(c), len(c))):
        if hi > lo:
            assert off(y[lo:hi], mm(a[lo:hi], w[e]) + mm(a[lo:hi], w2[e])) <= NORM, e


@SAME
@pytest.mark.parametrize("R", [700, 4096, 1 << 18])
@pytest.mark.parametrize("N,K", [(256, 256), (1024, 1024), (2048, 2048)])   # a cluster (long ones), one CTA or pairs
@pytest.mark.parametrize("accumulate", [False, True], ids=["new", "added"])
def test_fp32_weight_gradients(lm, R, N, K, accumulate, same):
    dy, x, dw = values((R, N), 1, same), values((R, K), 2, same), values((N, K), 3, same).float()
    start = dw.double() if accumulate else 0
    lm.lmoe_matmul_bf16_wgrad(dy, x, dw, accumulate=accumulate)
    assert off(dw, dwx(dy, x) + start) <= NORM


# ------------------------------------------------------------------ long reductions to bf16, products of one sign
@pytest.mark.parametrize("R,N", TILES)
@pytest.mark.parametrize("transposed", [False, True], ids=["nt", "nn"])
def test_long_products(lm, R, N, transposed):
    K = (1 << 20) - 8 if N <= 1024 else (1 << 18) + 8
    a, w = values((R, K), 1, True), values((K, N) if transposed else (N, K), 2, True)
    y = torch.zeros(R, N, dtype=BF16, device="cuda")
    lm.lmoe_matmul_bf16(a, w, y, transposed=transposed)
    want = mm(a, w, transposed)
    within(y, want, lost(want, K))


@pytest.mark.parametrize("R,N", TILES[:4])
def test_long_products_of_two_pairs_and_experts(lm, R, N):
    K, E = 1 << 18, 2
    c = [R // 2 + 1, R - R // 2 - 1]
    o, N = xu.offsets_of(c), min(N, 2048)
    a, w, w2 = values((R, K), 1, True), values((E, N, K), 2, True), values((E, N, K), 3, True)
    y = torch.zeros(R, N, dtype=BF16, device="cuda")
    lm.lmoe_matmul_bf16(a, w, y, offsets=o, a2=a, w2=w2)
    for e, (lo, hi) in enumerate(xu.groups(o, R, E)):
        want = mm(a[lo:hi], w[e]) + mm(a[lo:hi], w2[e])
        within(y[lo:hi], want, lost(want, 2 * K))


def test_products_just_below_the_length_that_ends_sums(lm):
    """16384 products in one sum: 1024 MMAs, 17 2^-23 512 of the result at most."""
    for R, N in TILES:
        a, w = values((R, 16384), 1, True), values((N, 16384), 2, True)
        y = torch.zeros(R, N, dtype=BF16, device="cuda")
        lm.lmoe_matmul_bf16(a, w, y)
        want = mm(a, w)
        within(y, want, 17 * 2.0 ** -23 * 512.5 * want.abs())


@pytest.mark.parametrize("R,N,K,c", [((1 << 22) + 13, 64, 72, None), ((1 << 20) + 5, 264, 136, [1 << 19, 0, 37, (1 << 19) - 32]),
                                     ((1 << 18) + 77, 2048, 2056, None), ((1 << 18), 2048, 1032, [200000, 100, 1 << 15, 29276])])
@pytest.mark.parametrize("accumulate", [False, True], ids=["new", "added"])
def test_long_weight_gradients(lm, R, N, K, c, accumulate):
    o, E = (None, 1) if c is None else (xu.offsets_of(c), len(c))
    dy, x = values((R, N), 1, True), values((R, K), 2, True)
    start = values((E, N, K), 3, True, 1000)
    dw = [start.clone(), start.clone()]
    lm.lmoe_matmul_bf16_wgrad(dy, x, dw[0], offsets=o, dy2=dy, dw2=dw[1], accumulate=accumulate)
    assert torch.equal(dw[0], dw[1])
    for e, (lo, hi) in enumerate(xu.groups(o, R, E)):
        want = dwx(dy[lo:hi], x[lo:hi]) if hi > lo else torch.zeros(N, K, dtype=torch.float64, device="cuda")
        tol = lost(want, hi - lo)
        if accumulate:
            want = want + start[e].double()
            tol = tol + 2.0 ** -24 * want
        if float(want.max()) > 0:
            within(dw[0][e], want, tol, f"expert {e}")
        else:
            assert not bool(dw[0][e].any())


GATED = [(8, 256), (16, 10240), (200, 512), (1900, 1032)]


@pytest.mark.parametrize("R,N", GATED)
def test_long_gated_products(lm, R, N):
    K = (1 << 18) + 8 if N > 8192 else (1 << 20) - 8
    std = 1.5 * K ** -0.5
    x, wg, wu = values((R, K), 1, True, std), values((N, K), 2, True, std), values((N, K), 3, True, std)
    h, g, u = (torch.zeros(R, N, dtype=BF16, device="cuda") for _ in range(3))
    lm.lmoe_gated_ffn(x, wg, wu, h, g, u)
    G, U = mm(x, wg), mm(x, wu)
    tg, tu = lost(G, K), lost(U, K)
    within(g, G, tg, "gate")
    within(u, U, tu, "up")
    s = G * torch.sigmoid(G)
    within(h, s * U, 1.1 * tg * (U + tu) + s * tu + 2.0 ** -19 * (1 + G) * s * U, "h")
    h2 = torch.zeros_like(h)
    lm.lmoe_gated_ffn(x, wg, wu, h2)
    assert torch.equal(h, h2)


@pytest.mark.parametrize("R,N", [GATED[0], GATED[1], GATED[2], (1900, 2056)])
@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
def test_long_gradients_of_the_gated_product(lm, R, N, in_place):
    K = (1 << 18) + 8 if N > 8192 else (1 << 20) - 8
    dy, wd = values((R, K), 1, True, K ** -0.5), values((K, N), 2, True, K ** -0.5)
    g, u = values((R, N), 3, True), values((R, N), 4, True)
    dh = mm(dy, wd, True)
    t, G, U = lost(dh, K), g.double(), u.double()
    s = torch.sigmoid(G)
    fg, fu = U * (s + G * s * torch.sigmoid(-G)), G * s
    dg, du = (g, u) if in_place else (torch.zeros_like(g), torch.zeros_like(u))
    lm.lmoe_gated_ffn_grad(dy, wd, g, u, dg, du)
    eg, eu = 2.0 ** -19 * (1 + G) ** 2 * s * U, 2.0 ** -19 * (1 + G) * fu
    within(dg, dh * fg, t * (fg + eg) + dh * eg, "dgate")
    within(du, dh * fu, t * (fu + eu) + dh * eu, "dup")
