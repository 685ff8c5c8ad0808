"""8-bit products whose scales lie far from one: an operand's scale may be as small as the quantisers'
floor 2^-126 or large, so that the product of two scales, or of a block's sum with one of them, leaves
fp32's range while the result is well inside it.

Codes are small multiples of a power of two and scales are powers of two, so that every sum here is exact
and results are compared exactly; with scales of any mantissa the bound of train_util.product holds, plus
one smallest step of fp32 per block for what falls below the normal range."""
import pytest
import torch

import train_util as tu
from train_util import E4M3, E5M2, assert_close

pytestmark = pytest.mark.gpu
OUT = pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
# 16 columns a tile, the same with the reduction split, 64 columns, the same split, rows as lanes
SIZES = [(6, 256, 256), (6, 256, 2048), (100, 640, 400), (100, 640, 2048), (600, 5000, 256)]
SIZE = pytest.mark.parametrize("R,N,K", SIZES)


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    return lm


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def integers(shape, fmt, seed):
    return torch.randint(-4, 5, shape, generator=gen(seed), device="cuda").float().to(fmt)


def two_to(e):
    """2^e as fp32, exactly (e: a tensor of whole numbers from -149 to 127)."""
    return torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e.cpu().double()).float().cuda()


def operands(R, N, K, seed=0, fmt=E4M3):
    return integers((R, K), fmt, seed + 1), integers((N, K), E4M3, seed + 2)


def matmul(lm, a, a_s, w, w_s, out):
    y = torch.full((a.shape[0], w.shape[0]), 7.25, dtype=out, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lm.lmoe_matmul_fp8(a, a_s, w, w_s, y, status=status)
    assert int(status) == 0
    return y


# sums of up to 2048 products of at most 16: below 2^15, so 2^15 times the scales' product is the largest
@SIZE
@OUT
@pytest.mark.parametrize("ea,ew", [(-126, -14), (-126, -20), (-20, -110), (-70, -60), (-126, 100), (100, -126), (-140, 30),
                                   (60, 50), (127, -100)])
def test_far_scales(lm, R, N, K, ea, ew, out):
    a, w = operands(R, N, K)
    kb, nb = -(-K // 128), -(-N // 128)
    a_s, w_s = two_to(torch.full((kb, R), ea)), two_to(torch.full((nb, kb), ew))
    want = (a.double() @ w.double().t()) * 2.0 ** (ea + ew)
    assert float(want.abs().max()) < 2.0 ** 127
    # (a sum is a whole number of steps 2^(ea + ew) from 2^-146 on: nothing is lost below the normal range)
    assert torch.equal(matmul(lm, a, a_s, w, w_s, out), want.float().to(out))


# large codes: the scales' product is below the smallest number fp32 has, the result a normal one
@SIZE
@OUT
@pytest.mark.parametrize("ea,ew", [(-126, -24), (-110, -50), (-126, -40)])
def test_sums_that_bring_far_scales_back(lm, R, N, K, ea, ew, out):
    a = (integers((R, K), E5M2, 1).float() * 2.0 ** 13).to(E5M2)
    w = (integers((N, K), E4M3, 2).float() * 2.0 ** 6).to(E4M3)
    kb, nb = -(-K // 128), -(-N // 128)
    want = (a.double() @ w.double().t()) * 2.0 ** (ea + ew)      # multiples of 2^(19 + ea + ew): 2^-147 at least
    got = matmul(lm, a, two_to(torch.full((kb, R), ea)), w, two_to(torch.full((nb, kb), ew)), out)
    assert torch.equal(got, want.float().to(out))


@SIZE
@OUT
def test_far_and_near_scales_beside_each_other(lm, R, N, K, out):
    # every row and every 128 columns have their own: only some lanes of a block are far
    a, w = operands(R, N, K, 3)
    kb, nb = -(-K // 128), -(-N // 128)
    ea = torch.randint(0, 8, (R,), generator=gen(5), device="cuda").cpu()
    ea = torch.tensor([-126, -110, 0, 1, -3, 40, 90, 2])[ea]
    ew = torch.tensor([-20, 0, 5, -14, 20, -1])[torch.arange(nb) % 6]
    a_s, w_s = two_to(ea.expand(kb, R).contiguous()), two_to(ew[:, None].expand(nb, kb).contiguous())
    y = a.double() @ w.double().t()
    e = ea[:, None] + ew.repeat_interleave(128)[:N][None]
    want = y * torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e.double()).cuda()
    assert torch.equal(matmul(lm, a, a_s, w, w_s, out), want.float().to(out))


@SIZE
def test_overflow_only_where_the_result_overflows(lm, R, N, K):
    a, w = operands(R, N, K, 6)
    kb, nb = -(-K // 128), -(-N // 128)
    a.view(torch.uint8)[:R // 2] = 0      # sums of zero: zero, whatever the scales
    y = matmul(lm, a, two_to(torch.full((kb, R), 127)), w, two_to(torch.full((nb, kb), 120)), torch.float32)
    assert bool((y[:R // 2] == 0).all())
    one = a.double()[R // 2:, :128] @ w.double()[:, :128].t()   # (several blocks may be infinities of both signs)
    if kb == 1:
        assert torch.equal(y[R // 2:], torch.where(one == 0, 0.0, one.sign() * float("inf")).float())
    assert not bool(torch.isfinite(y[R // 2:]).all())


@SIZE
def test_far_scales_of_any_mantissa(lm, R, N, K):
    a, w = operands(R, N, K, 9, E5M2)
    kb, nb = -(-K // 128), -(-N // 128)
    for lo, hi, wlo, whi in ((-126, -100, -30, -10), (-80, -60, -70, -40), (80, 110, -126, -90), (0, 60, 0, 50)):
        rnd = lambda shape, b, t, s: ((1 + torch.rand(shape, generator=gen(s), device="cuda")).double() * torch.exp2(
            torch.randint(b, t, shape, generator=gen(s + 1), device="cuda").double())).float()
        a_s, w_s = rnd((kb, R), lo, hi, 11), rnd((nb, kb), wlo, whi, 13)
        want, tol = tu.product(tu.values(a, a_s, False), tu.values(w, w_s, True))
        assert_close(matmul(lm, a, a_s, w, w_s, torch.float32), want, tol + 2.0 ** -149 * (kb + 1), f"{lo} {wlo}")


@SIZE
def test_gradient_rows_near_the_smallest_scale(lm, R, N, K):
    # from the quantisers themselves: gradients of about 2^-118 with weights of about 2^-5
    g = gen(20)
    dy = torch.randn(R, K, generator=g, device="cuda") * 2.0 ** -118
    w = torch.randn(N, K, generator=g, device="cuda") * 2.0 ** -5
    kb, nb = -(-K // 128), -(-N // 128)
    q, s = torch.zeros(R, K, dtype=torch.uint8, device="cuda").view(E5M2), torch.zeros(kb, R, device="cuda")
    wq, ws = torch.zeros(N, K, dtype=torch.uint8, device="cuda").view(E4M3), torch.zeros(nb, kb, device="cuda")
    lm.lmoe_quantize_fp8_rows(dy, q, s)
    lm.lmoe_quantize_fp8_weight(w, wq, ws)
    want, tol = tu.product(tu.values(q, s, False), tu.values(wq, ws, True))
    assert_close(matmul(lm, q, s, wq, ws, torch.float32), want, tol + 2.0 ** -149 * (kb + 1))


# ------------------------------------------------------------------ weight gradients
def wgrad(lm, dy, ds, x, xs, out=torch.float32):
    dw = torch.full((dy.shape[0], x.shape[0]), 7.25, dtype=out, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lm.lmoe_matmul_fp8_wgrad(dy, ds, x, xs, dw, status=status)
    assert int(status) == 0
    return dw


# (exponents of dy's and x's codes, of their scales): a block's sum times one scale alone falls below the
# normal range, or passes its end
@OUT
@pytest.mark.parametrize("cy,cx,ey,ex", [(-14, -6, 60, -126), (-14, -6, -126, 60), (8, 4, -60, 119), (8, 4, 119, -60),
                                         (0, 0, -126, 20), (-14, -6, 110, -140), (-14, -6, 119, -100), (0, 0, -60, -60)])
@pytest.mark.parametrize("N,K,P", [(130, 200, 128), (256, 144, 384)])
def test_far_scales_in_weight_gradients(lm, N, K, P, cy, cx, ey, ex, out):
    dy = (torch.randint(-3, 4, (N, P), generator=gen(1), device="cuda").float() * 2.0 ** cy).to(E5M2)
    x = (torch.randint(-4, 5, (K, P), generator=gen(2), device="cuda").float() * 2.0 ** cx).to(E4M3)
    want = (dy.double() @ x.double().t()) * 2.0 ** (ey + ex)
    got = wgrad(lm, dy, two_to(torch.full((P // 128, N), ey)), x, two_to(torch.full((P // 128, K), ex)), out)
    assert torch.equal(got, want.float().to(out))


@pytest.mark.parametrize("N,K,P", [(130, 200, 128), (300, 400, 640)])
def test_far_and_near_scales_in_weight_gradients(lm, N, K, P):
    dy = (torch.randn(N, P, generator=gen(1), device="cuda") * 60).to(E5M2)
    x = (torch.randn(K, P, generator=gen(2), device="cuda") * 60).to(E4M3)
    pick = lambda es, n, s: two_to(torch.tensor(es)[torch.randint(0, len(es), (P // 128, n), generator=gen(s), device="cuda").cpu()]) \
        * (1 + torch.rand(P // 128, n, generator=gen(s + 5), device="cuda"))
    for ey, ex in (([-126, -100, 0, 3], [-126, -20, 0, 90]), ([-120, -100], [90, 100, 110]), ([90, 100], [-126, -100])):
        ds, xs = pick(ey, N, 3), pick(ex, K, 4)
        want, tol = tu.product(tu.values(dy, ds, False), tu.values(x, xs, False))
        assert_close(wgrad(lm, dy, ds, x, xs), want, tol + 2.0 ** -149 * (P // 128 + 1), f"{ey} {ex}")
