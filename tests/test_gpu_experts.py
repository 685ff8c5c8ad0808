"""The bf16 experts' operators against plain forms in 64 bits.

With operands that are small integers every sum is exact in fp32 (below 2^24), whatever its order, so layouts and
edges are compared exactly; with random operands the error is bounded as expert_util derives it."""
import ctypes

import pytest
import torch

import expert_util as xu
from expert_util import BF16, close

pytestmark = pytest.mark.gpu
F32 = torch.float32
OUT = pytest.mark.parametrize("out", [F32, BF16], ids=["f32", "bf16"])
WAITS = 0x1 | 0x2 | 0x4 | 0x10   # the error word's bits of waits that gave up


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


def ints(shape, seed, most=3):
    return torch.randint(-most, most + 1, shape, generator=gen(seed), device="cuda").to(BF16)


def normal(shape, seed, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).to(BF16)


def buffer(rows, N, dtype, fill=7.25):
    """[rows, N] and four rows more, which have to stay as they are."""
    t = torch.full((rows + 4, N), fill, dtype=dtype, device="cuda")
    return t, t[:rows]


def counts(name, R):
    """Rows of each expert."""
    return {"one": [R], "even": [R // 4, R // 4, R // 4, R - 3 * (R // 4)],
            "skewed": [0, 1, R - 1 - R // 5, 0, 0, R // 5, 0],
            "many": [i % 3 for i in range(40)] + [R - 39]}[name] if R >= 40 or name != "many" else [R] + [0] * 40


# (rows, N, K): single rows, tiles of few rows, whole and ragged tiles, reductions that are shared by a cluster
SHAPES = [(1, 8, 8), (1, 256, 2048), (3, 136, 72), (17, 64, 1032), (16, 264, 520), (33, 72, 136), (64, 128, 64),
          (100, 520, 4104), (127, 1000, 192), (128, 256, 256), (129, 136, 264), (257, 392, 72), (300, 640, 1096),
          (1000, 264, 512), (2050, 520, 136)]
SPLITS = ["one", "even", "skewed", "many"]


def weights(E, N, K, seed, transposed, make=ints):
    w = make((E, N, K), seed)
    return w.transpose(1, 2).contiguous() if transposed else w


# ------------------------------------------------------------------ products
@pytest.mark.parametrize("R,N,K", SHAPES)
@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("transposed", [False, True], ids=["nt", "nn"])
def test_matmul_is_exact_on_integers(lm, R, N, K, split, transposed):
    c = counts(split, R)
    E, off = len(c), xu.offsets_of(c) if len(c) > 1 else None
    a, w = ints((R, K), 1), weights(E, N, K, 2, transposed)
    whole, y = buffer(R, N, F32)
    lm.lmoe_matmul_bf16(a, w, y, offsets=off, transposed=transposed)
    want = xu.product(a, w, off, transposed)[0]
    assert torch.equal(y.double(), want)
    assert bool((whole[R:] == 7.25).all())
    a2, w2 = ints((R, K), 3), weights(E, N, K, 4, transposed)
    whole, y = buffer(R, N, BF16)
    lm.lmoe_matmul_bf16(a, w, y, offsets=off, a2=a2, w2=w2, transposed=transposed)
    want = want + xu.product(a2, w2, off, transposed)[0]
    assert torch.equal(y, want.float().to(BF16))
    assert bool((whole[R:] == 7.25).all())
    assert lm.lmoe_bf16_check_status() == (0, 0)


@pytest.mark.parametrize("R,N,K,E", [(5, 512, 4096, 1), (60, 512, 1024, 9), (700, 392, 2056, 3), (1500, 1024, 512, 2)])
@pytest.mark.parametrize("transposed", [False, True], ids=["nt", "nn"])
@OUT
def test_matmul_of_random_operands(lm, R, N, K, E, transposed, out):
    off = xu.offsets_of([R // E] * (E - 1) + [R - R // E * (E - 1)])
    a, w = normal((R, K), 1), weights(E, N, K, 2, transposed, normal)
    y = torch.zeros(R, N, dtype=out, device="cuda")
    lm.lmoe_matmul_bf16(a, w, y, offsets=off, transposed=transposed)
    want, tol = xu.product(a, w, off, transposed)
    close(y, want, xu.rounded(want, tol, out))


def test_no_rows(lm):
    N, K, E = 64, 128, 3
    e = lambda n: torch.empty(0, n, dtype=BF16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    w, wt = ints((E, N, K), 1), ints((E, K, N), 2)
    n0 = lm.lmoe_kernel_launches()
    lm.lmoe_gated_ffn(e(K), w, w, e(N), e(N), e(N), offsets=off)
    lm.lmoe_gated_ffn_grad(e(K), wt, e(N), e(N), e(N), e(N), offsets=off)
    lm.lmoe_matmul_bf16(e(K), w, e(N), offsets=off)
    lm.lmoe_matmul_bf16(e(K), wt, e(N), offsets=off, a2=e(K), w2=wt, transposed=True)
    for dtype in (F32, BF16):
        dw, dw2 = (torch.full((E, N, K), 3.0, dtype=dtype, device="cuda") for _ in range(2))
        lm.lmoe_matmul_bf16_wgrad(e(N), e(K), dw, offsets=off, dy2=e(N), dw2=dw2, accumulate=True)
        assert bool((dw == 3).all()) and bool((dw2 == 3).all())
        lm.lmoe_matmul_bf16_wgrad(e(N), e(K), dw, offsets=off, dy2=e(N), dw2=dw2)
        assert bool((dw == 0).all()) and bool((dw2 == 0).all())
    assert lm.lmoe_kernel_launches() == n0
    # rows, but none of an expert
    a, y, dw = ints((50, K), 3), torch.full((50, N), 7.25, device="cuda"), torch.full((E, N, K), 3.0, device="cuda")
    lm.lmoe_matmul_bf16(a, w, y, offsets=off)
    lm.lmoe_matmul_bf16_wgrad(ints((50, N), 4), a, dw, offsets=off)
    assert bool((y == 7.25).all()) and bool((dw == 0).all())


def test_rows_of_no_expert_and_wild_offsets(lm):
    R, N, K = 300, 136, 264
    a, w = ints((R, K), 1), ints((3, N, K), 2)
    a[:20], a[250:] = float("nan"), float("inf")
    for off in ([20, 100, 100, 250], [20, 20, 20, 250], [20, 250, 250, 250]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        whole, y = buffer(R, N, F32)
        lm.lmoe_matmul_bf16(a, w, y, offsets=off)
        want = xu.product(a, w, off)[0]
        assert torch.equal(y[20:250].double(), want[20:250])
        assert bool((y[:20] == 7.25).all()) and bool((whole[250:] == 7.25).all())
    # out of range, falling: clamped, and nothing behind the result is written
    for off in ([-5, 100, 400, 1 << 30], [200, 100, 50, 0], [-(1 << 31), 1 << 30, 7, 300], [0, 300, 0, 300]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        for shape in ((R, N), (R, N)):
            whole, y = buffer(*shape, F32)
            lm.lmoe_matmul_bf16(a, w, y, offsets=off)
            assert bool((whole[R:] == 7.25).all())
            h, g, u = (buffer(R, N, BF16) for _ in range(3))
            lm.lmoe_gated_ffn(a, w, w, h[1], g[1], u[1], offsets=off)
            for b in (h, g, u):
                assert bool((b[0][R:] == 7.25).all())
            dw = torch.full((3 * N * K + 64,), 7.25, device="cuda")
            lm.lmoe_matmul_bf16_wgrad(ints((R, N), 5), a, dw[:-64].view(3, N, K), offsets=off)
            assert bool((dw[-64:] == 7.25).all())
    assert lm.lmoe_bf16_check_status() == (0, 0)


@pytest.mark.parametrize("R,E", [(8, 64), (40, 9), (400, 3), (1200, 4)])
def test_a_bad_row_stays_its_own(lm, R, E):
    N, K = 264, 320
    off = xu.offsets_of([R // E] * (E - 1) + [R - R // E * (E - 1)])
    a, w = normal((R, K), 1), normal((E, N, K), 2)
    bad = list(range(0, R, 7))
    a[bad[0::2]], a[bad[1::2], 5] = float("nan"), float("inf")
    y = torch.zeros(R, N, device="cuda")
    lm.lmoe_matmul_bf16(a, w, y, offsets=off)
    good = torch.ones(R, dtype=torch.bool, device="cuda")
    good[bad] = False
    want, tol = xu.product(a, w, off)
    close(y[good], want[good], tol[good])
    assert not bool(torch.isfinite(y[~good]).any())


# ------------------------------------------------------------------ the gated block
@pytest.mark.parametrize("R,N,K", SHAPES)
@pytest.mark.parametrize("split", SPLITS)
def test_gated_ffn(lm, R, N, K, split):
    c = counts(split, R)
    E, off = len(c), xu.offsets_of(c) if len(c) > 1 else None
    x, wg, wu = normal((R, K), 1), normal((E, N, K), 2, 2 * K ** -0.5), normal((E, N, K), 3, K ** -0.5)
    bufs = [buffer(R, N, BF16) for _ in range(3)]
    lm.lmoe_gated_ffn(x, wg, wu, *[b[1] for b in bufs], offsets=off)
    for (whole, got), (want, tol), name in zip(bufs, xu.gated(x, wg, wu, off), "hgu"):
        close(got, want, tol, name)
        assert bool((whole[R:] == 7.25).all())
    h2 = torch.zeros(R, N, dtype=BF16, device="cuda")
    lm.lmoe_gated_ffn(x, wg, wu, h2, offsets=off)
    assert torch.equal(h2, bufs[0][1])      # with nothing saved: the same
    # integers: gate and up exactly
    x, wg, wu = ints((R, K), 4), ints((E, N, K), 5), ints((E, N, K), 6)
    lm.lmoe_gated_ffn(x, wg, wu, *[b[1] for b in bufs], offsets=off)
    assert torch.equal(bufs[1][1], xu.product(x, wg, off)[0].float().to(BF16))
    assert torch.equal(bufs[2][1], xu.product(x, wu, off)[0].float().to(BF16))
    assert lm.lmoe_bf16_check_status() == (0, 0)


def test_gated_ffn_of_large_and_small_values(lm):
    """exp(-g) over its whole range: g from -200 to 200, and infinities."""
    K, N = 8, 64
    g = torch.linspace(-200, 200, 128, device="cuda").to(BF16)
    x = torch.zeros(128, K, dtype=BF16, device="cuda")
    x[:, 0], x[:, 1] = g, 1
    wg, wu = torch.zeros(N, K, dtype=BF16, device="cuda"), torch.zeros(N, K, dtype=BF16, device="cuda")
    wg[:, 0] = 1
    wu[:, 1] = torch.linspace(-3, 3, N, device="cuda").to(BF16)
    h, a, b = (torch.zeros(128, N, dtype=BF16, device="cuda") for _ in range(3))
    lm.lmoe_gated_ffn(x, wg, wu, h, a, b)
    for got, (want, tol) in zip((h, a, b), xu.gated(x, wg, wu)):
        close(got, want, tol)
    x[5, 0], x[6, 0], x[7, 0] = float("inf"), -float("inf"), float("nan")
    wg[:, 0] = 2
    lm.lmoe_gated_ffn(x, wg, wu, h)
    assert bool(torch.isnan(h[5:8]).all())   # (an infinity of x meets a zero of w_up: u is NaN in those rows)
    assert bool(torch.isfinite(h[:5]).all()) and bool(torch.isfinite(h[8:]).all())


def test_gated_ffn_where_gate_overflows(lm):
    """Finite operands whose products leave fp32's range: silu(inf) = inf, silu(-inf) = -inf 0 is NaN."""
    x, wg, wu = torch.zeros(4, 8, dtype=BF16, device="cuda"), torch.zeros(32, 8, dtype=BF16, device="cuda"), \
        torch.ones(32, 8, dtype=BF16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0], x[:, 1] = 3e38, -3e38, 1, 2
    wg[:, 0], wu[:, 0] = 2, 0
    h = torch.zeros(4, 32, dtype=BF16, device="cuda")
    lm.lmoe_gated_ffn(x, wg, wu, h)
    assert bool((h[0] == float("inf")).all()) and bool(torch.isnan(h[1]).all()) and bool(torch.isfinite(h[2:]).all())


@pytest.mark.parametrize("R,N,K", SHAPES)
@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
def test_gated_ffn_grad(lm, R, N, K, split, in_place):
    c = counts(split, R)
    E, off = len(c), xu.offsets_of(c) if len(c) > 1 else None
    dy, wd, g, u = normal((R, K), 1, 1e-2), normal((E, K, N), 2, N ** -0.5), normal((R, N), 3, 3), normal((R, N), 4)
    want = xu.gated_grad(dy, wd, g, u, off)
    bufs = [buffer(R, N, BF16) for _ in range(2)]
    if in_place:
        for b, src in zip(bufs, (g, u)):
            b[1].copy_(src)
        lm.lmoe_gated_ffn_grad(dy, wd, bufs[0][1], bufs[1][1], bufs[0][1], bufs[1][1], offsets=off)
    else:
        lm.lmoe_gated_ffn_grad(dy, wd, g, u, bufs[0][1], bufs[1][1], offsets=off)
    for (whole, got), (v, tol), name in zip(bufs, want, ("dgate", "dup")):
        close(got, v, tol, name)
        assert bool((whole[R:] == 7.25).all())
    assert lm.lmoe_bf16_check_status() == (0, 0)


def test_gated_ffn_grad_of_full_tiles_many_times(lm):
    """Large tiles, where the tensor cores keep shared memory busy: the same bits each time, and the right ones."""
    R, N, K, E = 8192, 2048, 2048, 8
    off = xu.offsets_of([1300, 700, 1024, 100, 2000, 1024, 1500, 544])
    dy, wd, g, u = normal((R, K), 1, 1e-2), normal((E, K, N), 2, N ** -0.5), normal((R, N), 3, 2), normal((R, N), 4)
    (dg, tg), (du, tu) = xu.gated_grad(dy, wd, g, u, off)
    for _ in range(25):
        a, b = torch.zeros_like(g), torch.zeros_like(u)
        lm.lmoe_gated_ffn_grad(dy, wd, g, u, a, b, offsets=off)
        close(a, dg, tg, "dgate")
        close(b, du, tu, "dup")


def test_gated_ffn_of_full_tiles_many_times(lm):
    R, N, K, E = 8192, 2048, 2048, 8
    off = xu.offsets_of([1300, 700, 1024, 100, 2000, 1024, 1500, 544])
    x, wg, wu = normal((R, K), 1), normal((E, N, K), 2, K ** -0.5), normal((E, N, K), 3, K ** -0.5)
    want = xu.gated(x, wg, wu, off)
    for _ in range(25):
        bufs = [torch.zeros(R, N, dtype=BF16, device="cuda") for _ in range(3)]
        lm.lmoe_gated_ffn(x, wg, wu, *bufs, offsets=off)
        for got, (v, tol), name in zip(bufs, want, "hgu"):
            close(got, v, tol, name)


def test_products_of_full_tiles_many_times(lm):
    R, N, K, E = 8192, 2048, 2048, 8
    off = xu.offsets_of([1300, 700, 1024, 100, 2000, 1024, 1500, 544])
    a, w, dy = ints((R, K), 1), ints((E, N, K), 2), ints((R, N), 3)
    want, dw = xu.product(a, w, off)[0], xu.wgrad(dy, a, E, off)[0]
    for out in (F32, BF16):
        for _ in range(25):
            y, d = torch.zeros(R, N, dtype=out, device="cuda"), torch.zeros(E, N, K, dtype=out, device="cuda")
            lm.lmoe_matmul_bf16(a, w, y, offsets=off)
            lm.lmoe_matmul_bf16_wgrad(dy, a, d, offsets=off)
            assert torch.equal(y, want.float().to(out)) and torch.equal(d, dw.float().to(out))


def test_gradient_is_that_of_the_block(lm):
    """dgate, dup against differences of the loss sum(dy . y) with the down projection behind the gated product."""
    R, N, K, h = 12, 24, 40, 2.0 ** -10
    dy, wd, g, u = normal((R, K), 1), normal((K, N), 2), normal((R, N), 3), normal((R, N), 4)
    dg, du = torch.zeros_like(g), torch.zeros_like(u)
    lm.lmoe_gated_ffn_grad(dy, wd, g, u, dg, du)

    def loss(g, u):   # of each (r, n) alone: the loss is a sum over them
        return (dy.double() @ wd.double()) * (g * torch.sigmoid(g) * u)
    G, U = g.double(), u.double()
    # the second difference's error is h^2/6 times a third derivative of silu, which is below 1
    dh = (dy.double() @ wd.double()).abs()
    tol = h * h * dh * (1 + U.abs()) + 2.0 ** -30
    for got, d in ((dg, (loss(G + h, U) - loss(G - h, U)) / (2 * h)), (du, (loss(G, U + h) - loss(G, U - h)) / (2 * h))):
        close(got, d, tol + 1.5 * 2.0 ** -8 * d.abs() + 2.0 ** -15 * dh * (1 + U.abs()))


# ------------------------------------------------------------------ weight gradients
WSHAPES = [(1, 8, 8), (5, 64, 64), (16, 136, 72), (17, 128, 128), (63, 264, 8), (64, 8, 264), (100, 200, 136),
           (130, 72, 520), (1000, 264, 392), (2049, 136, 256)]


@pytest.mark.parametrize("R,N,K", WSHAPES)
@pytest.mark.parametrize("split", SPLITS)
@OUT
@pytest.mark.parametrize("accumulate", [False, True], ids=["new", "added"])
def test_wgrad_is_exact_on_integers(lm, R, N, K, split, out, accumulate):
    c = counts(split, R)
    E, off = len(c), xu.offsets_of(c) if len(c) > 1 else None
    dy, dy2, x = ints((R, N), 1), ints((R, N), 2), ints((R, K), 3)
    bufs = []
    for _ in range(2):
        b = torch.full((E * N * K + 64,), 0.0, dtype=out, device="cuda")
        b[:-64] = ints((E * N * K,), 4).to(out)
        b[-64:] = 7.25
        bufs.append(b)
    start = [b[:-64].view(E, N, K).clone() for b in bufs]
    dw, dw2 = (b[:-64].view(E, N, K) for b in bufs)
    lm.lmoe_matmul_bf16_wgrad(dy, x, dw, offsets=off, dy2=dy2, dw2=dw2, accumulate=accumulate)
    for got, d, s in ((dw, dy, start[0]), (dw2, dy2, start[1])):
        want = xu.wgrad(d, x, E, off)[0] + (s.double() if accumulate else 0)
        assert torch.equal(got, want.float().to(out))
    if accumulate:   # an expert without rows is left as it was
        for e, (lo, hi) in enumerate(xu.groups(off, R, E)):
            if lo == hi:
                assert torch.equal(dw[e], start[0][e])
    single = start[0].clone()
    lm.lmoe_matmul_bf16_wgrad(dy, x, single, offsets=off, accumulate=accumulate)
    assert torch.equal(single, dw)
    assert bool((bufs[0][-64:] == 7.25).all()) and bool((bufs[1][-64:] == 7.25).all())
    assert lm.lmoe_bf16_check_status() == (0, 0)


@OUT
def test_wgrad_of_random_operands(lm, out):
    for R, N, K, c in ((700, 264, 520, [300, 0, 400]), (37, 512, 256, [1, 36]), (4096, 256, 256, [4096])):
        off = xu.offsets_of(c)
        dy, x = normal((R, N), 1, 1e-3), normal((R, K), 2)
        dw = torch.zeros(len(c), N, K, dtype=out, device="cuda")
        lm.lmoe_matmul_bf16_wgrad(dy, x, dw, offsets=off)
        want, tol = xu.wgrad(dy, x, len(c), off)
        close(dw, want, xu.rounded(want, tol, out))
        start = normal((len(c), N, K), 3, 1e-2).to(out)
        dw = start.clone()
        lm.lmoe_matmul_bf16_wgrad(dy, x, dw, offsets=off, accumulate=True)
        want, tol = xu.wgrad(dy, x, len(c), off, start)
        close(dw, want, xu.rounded(want, tol, out))


@pytest.mark.parametrize("c", [[3, 5, 1, 200, 64, 16, 79], [1] * 40, [65, 15, 17, 130], [70, 0, 0, 31]])
def test_other_experts_rows_do_not_count(lm, c):
    """An expert's neighbours hold infinities and NaN, rows of no expert too."""
    N, K = 136, 200
    R = sum(c) + 60
    off = (torch.tensor([0] + c).cumsum(0) + 20).to(torch.int32).cuda()
    clean_dy, clean_x = ints((R, N), 1), ints((R, K), 2)
    bounds = off.tolist()
    for e in range(len(c)):
        dy, x = clean_dy.clone(), clean_x.clone()
        mine = torch.zeros(R, dtype=torch.bool, device="cuda")
        mine[bounds[e]:bounds[e + 1]] = True
        dy[~mine], x[~mine] = float("nan"), float("inf")
        dw = torch.zeros(len(c), N, K, device="cuda")
        lm.lmoe_matmul_bf16_wgrad(dy, x, dw, offsets=off)
        d, v = clean_dy[mine].double(), clean_x[mine].double()
        assert torch.equal(dw[e].double(), d.t() @ v), e
        if e >= 6:
            break


# ------------------------------------------------------------------ status, streams, graphs
def raw(lm, name, dims, out, budget, status, *args):
    from latent_mixture_experts_router_gb300 import _lib
    R, N, K, E, transposed, accumulate = dims
    shape = _lib.lmoe_bf16_matmul(R, N, K, E, 0 if out == F32 else 1, transposed, accumulate, budget)
    st = getattr(_lib._lib(), name)(ctypes.byref(shape), *[t if t is None else t.data_ptr() for t in args],
                                    status.data_ptr() if status is not None else None,
                                    torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    return int(status.item()) & 0xffffffff if status is not None else None


@pytest.mark.parametrize("R,E,N,K", [(6, 1, 256, 256), (6, 1, 256, 2048), (100, 1, 640, 400), (100, 3, 640, 2048),
                                     (600, 1, 5000, 256), (40, 9, 520, 512), (3000, 6, 1000, 1024), (700, 2, 2048, 64)])
def test_waits_that_give_up(lm, R, E, N, K):
    off = (torch.arange(E + 1, device="cuda") * R // E).int()
    a, w, g, u = ints((R, K), 1), ints((E, N, K), 2), ints((R, N), 3), ints((R, N), 4)
    wt = w.transpose(1, 2).contiguous()
    b = [buffer(R, N, BF16) for _ in range(3)]
    y = buffer(R, N, F32)
    dw = torch.full((E * N * K + 64,), 7.25, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = [
        lambda n: raw(lm, "lmoe_gated_ffn", (R, N, K, E, 0, 0), BF16, n, status, a, w, w, off, b[0][1], b[1][1], b[2][1]),
        lambda n: raw(lm, "lmoe_gated_ffn_grad", (R, N, K, E, 0, 0), BF16, n, status, a, wt, g, u, off, b[0][1], b[1][1]),
        lambda n: raw(lm, "lmoe_matmul_bf16", (R, N, K, E, 0, 0), F32, n, status, a, w, None, None, off, y[1]),
        lambda n: raw(lm, "lmoe_matmul_bf16", (R, N, K, E, 1, 0), F32, n, status, a, wt, a, wt, off, y[1]),
        lambda n: raw(lm, "lmoe_matmul_bf16_wgrad", (R, N, K, E, 0, 0), F32, n, status, g, a, None, off, dw, None),
    ]
    for call in calls:
        for _ in range(2):
            assert call(1) & ~WAITS == 0
        status.zero_()
        assert call(0) == 0
    for whole, _ in b + [y]:
        assert bool((whole[R:] == 7.25).all())
    assert bool((dw[-64:] == 7.25).all())
    assert torch.equal(y[1].double(), 2 * xu.product(a, w, off)[0])
    assert torch.equal(dw[:-64].view(E, N, K).double(), xu.wgrad(g, a, E, off)[0])


def test_calls_without_a_status_word_report_too(lm):
    assert lm.lmoe_bf16_check_status()[0] in (0, -6)
    s = torch.cuda.Stream()
    lm.lmoe_bf16_wait_selftest(100_000, stream=s)
    st, word = lm.lmoe_bf16_check_status(stream=s)
    assert st == -6 and word & WAITS and word & ~WAITS == 0
    assert lm.lmoe_bf16_check_status() == (0, 0)
    # a wait gives up after 20 us at the earliest: tiles of 1024 blocks, 256 cycles each at least, take 100
    a, w = ints((300, 65536), 1), ints((5000, 65536), 2)
    y = torch.zeros(300, 5000, device="cuda")
    for _ in range(3):
        raw(lm, "lmoe_matmul_bf16", (300, 5000, 65536, 1, 0, 0), F32, 1, None, a, w, None, None, None, y)
    assert lm.lmoe_bf16_check_status()[0] == -6
    lm.lmoe_matmul_bf16(a, w, y)
    assert lm.lmoe_bf16_check_status() == (0, 0)
    assert torch.equal(y.double(), a.double() @ w.double().t())


def test_long_calls_are_no_timeouts(lm):
    """Calls of tens of milliseconds: no wait of theirs may take the whole for its own."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    assert lm.lmoe_bf16_check_status()[0] in (0, -6)
    a, w = normal((1 << 18, 8192), 1), normal((8192, 8192), 2)
    y = torch.zeros(1 << 18, 8192, dtype=BF16, device="cuda")
    dw = torch.zeros(8192, 8192, device="cuda")
    lm.lmoe_matmul_bf16(a, w, y)
    lm.lmoe_matmul_bf16_wgrad(a, a, dw)
    assert lm.lmoe_bf16_check_status() == (0, 0)
    rows = torch.tensor([0, 77777, (1 << 18) - 1], device="cuda")
    want, tol = xu.product(a[rows], w)
    close(y[rows], want, xu.rounded(want, tol, BF16))
    d = a[:, :16].double()
    want, tol = d.t() @ a[:, :64].double(), (d.abs().t() @ a[:, :64].double().abs()) * 2.0 ** -23 * 768
    close(dw[:16, :64], want, tol)


def test_two_streams_at_once(lm):
    """Calls on two streams share nothing: each gives what it gives alone."""
    made = []
    for i, (R, N, K, E) in enumerate(((900, 1024, 512, 3), (20, 2048, 1024, 8))):
        off = xu.offsets_of([R // E] * (E - 1) + [R - R // E * (E - 1)])
        made.append((ints((R, K), i), ints((E, N, K), i + 5), off, torch.zeros(R, N, device="cuda"),
                     torch.zeros(E, N, K, device="cuda"), ints((R, N), i + 9)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(10):
        for s, (a, w, off, y, dw, dy) in zip(streams, made):
            lm.lmoe_matmul_bf16(a, w, y, offsets=off, stream=s)
            lm.lmoe_matmul_bf16_wgrad(dy, a, dw, offsets=off, stream=s)
    torch.cuda.synchronize()
    for a, w, off, y, dw, dy in made:
        assert torch.equal(y.double(), xu.product(a, w, off)[0])
        assert torch.equal(dw.double(), xu.wgrad(dy, a, w.shape[0], off)[0])
    assert lm.lmoe_bf16_check_status() == (0, 0)


@pytest.mark.parametrize("R,E", [(8, 16), (500, 4)])
def test_captured_calls_follow_their_inputs(lm, R, E):
    """A graph of the calls, replayed with other rows, weights and offsets in the same buffers."""
    N, K = 256, 512
    x, wg, wd = ints((R, K), 1), ints((E, N, K), 2), ints((E, K, N), 3)
    off = xu.offsets_of([R // E] * (E - 1) + [R - R // E * (E - 1)])
    h, g, u, dg, du = (torch.zeros(R, N, dtype=BF16, device="cuda") for _ in range(5))
    y, dw = torch.zeros(R, K, device="cuda"), torch.zeros(E, N, K, device="cuda")

    def step():
        lm.lmoe_gated_ffn(x, wg, wg, h, g, u, offsets=off)
        lm.lmoe_matmul_bf16(h, wd, y, offsets=off)
        lm.lmoe_gated_ffn_grad(x, wd, g, u, dg, du, offsets=off)
        lm.lmoe_matmul_bf16_wgrad(dg, x, dw, offsets=off)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (10, 20):
        x.copy_(ints((R, K), seed))
        wg.copy_(ints((E, N, K), seed + 1))
        c = torch.bincount(torch.randint(0, E, (R,), generator=gen(seed), device="cuda"), minlength=E)
        off.copy_(xu.offsets_of(c.tolist()))
        graph.replay()
        got = [t.clone() for t in (h, g, u, y, dg, du, dw)]
        for t in (h, g, u, y, dg, du, dw):
            t.zero_()
        step()
        for a, b in zip(got, (h, g, u, y, dg, du, dw)):
            assert torch.equal(a, b)
        assert torch.equal(g, xu.product(x, wg, off)[0].float().to(BF16))


def test_the_same_inputs_give_the_same_bits(lm):
    R, N, K, E = 700, 520, 1032, 5
    off = xu.offsets_of([100, 0, 300, 7, 293])
    a, w, dy = normal((R, K), 1), normal((E, N, K), 2), normal((R, N), 3)
    first = None
    for _ in range(3):
        y, dw = torch.zeros(R, N, device="cuda"), torch.zeros(E, N, K, device="cuda")
        lm.lmoe_matmul_bf16(a, w, y, offsets=off)
        lm.lmoe_matmul_bf16_wgrad(dy, a, dw, offsets=off)
        if first is None:
            first = (y, dw)
        assert torch.equal(y, first[0]) and torch.equal(dw, first[1])


def test_more_than_32_bits_of_elements(lm):
    """Weights of more than 2^32 elements, rows far into them: addresses beyond 32 bits."""
    E, N, K = 130, 4096, 8192
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("not enough memory")
    w = torch.zeros(E, N, K, dtype=BF16, device="cuda")
    for e in (0, 63, 64, 127, 128, 129):
        w[e] = ints((N, K), e, 2)
    c = [0] * E
    c[63], c[64], c[127], c[128], c[129] = 3, 1, 2, 40, 5
    off = xu.offsets_of(c)
    a = ints((51, K), 7, 2)
    y = torch.zeros(51, N, device="cuda")
    lm.lmoe_matmul_bf16(a, w, y, offsets=off)
    for e in (63, 64, 127, 128, 129):
        lo, hi = int(off[e]), int(off[e + 1])
        assert torch.equal(y[lo:hi].double(), a[lo:hi].double() @ w[e].double().t())
    dw, dy = w, ints((51, N), 8, 2)       # written over
    lm.lmoe_matmul_bf16_wgrad(dy, a, dw, offsets=off)
    for e in (0, 63, 64, 127, 128, 129):
        lo, hi = int(off[e]), int(off[e + 1])
        assert torch.equal(dw[e].double(), dy[lo:hi].double().t() @ a[lo:hi].double()), e
