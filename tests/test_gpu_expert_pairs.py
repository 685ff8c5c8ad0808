"""Pairs of CTAs at sizes that are no multiples of anything: widths and reductions that end inside a box, experts of a row more than
a tile, of one row and of none, one matrix of fewer rows than a box is high.  Sizes are such that the rules take pairs.
Operands are small integers, so sums are exact; the gated calls are bounded as expert_util derives it."""
import pytest
import torch

import expert_util as xu
from expert_util import BF16, close

pytestmark = pytest.mark.gpu
F32 = torch.float32
OUT = pytest.mark.parametrize("out", [F32, BF16], ids=["f32", "bf16"])


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    return lm


def ints(shape, seed):
    return torch.randint(-3, 4, shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)


def normal(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * std).to(BF16)


def buffer(rows, N, dtype):
    t = torch.full((rows + 4, N), 7.25, dtype=dtype, device="cuda")
    return t, t[:rows]


# rows of each expert (one: a matrix), N, K
SIZES = [([17], 40000, 1032), ([40], 40008, 1096), ([63], 39992, 1032), ([130], 40000, 1032), ([257], 40072, 200),
         ([257, 1, 442], 3000, 200), ([255, 0, 256, 513], 3016, 72), ([129, 127, 128, 385], 2824, 1000),
         ([383, 641], 5000, 8), ([100, 150, 90], 6600, 264)]
IDS = ["-".join(map(str, c)) + f"_{n}x{k}" for c, n, k in SIZES]


@pytest.mark.parametrize("c,N,K", SIZES, ids=IDS)
@pytest.mark.parametrize("transposed", [False, True], ids=["nt", "nn"])
@OUT
def test_products(lm, c, N, K, transposed, out):
    R, E, off = sum(c), len(c), xu.offsets_of(c) if len(c) > 1 else None
    shape = (E, K, N) if transposed else (E, N, K)
    a, a2, w, w2 = ints((R, K), 1), ints((R, K), 2), ints(shape, 3), ints(shape, 4)
    for pair in ({}, dict(a2=a2, w2=w2)):
        whole, y = buffer(R, N, out)
        lm.lmoe_matmul_bf16(a, w, y, offsets=off, transposed=transposed, **pair)
        want = xu.product(a, w, off, transposed)[0]
        if pair:
            want = want + xu.product(a2, w2, off, transposed)[0]
        assert torch.equal(y, want.float().to(out))
        assert bool((whole[R:] == 7.25).all())
    assert lm.lmoe_bf16_check_status() == (0, 0)


@pytest.mark.parametrize("c,N,K", SIZES, ids=IDS)
def test_gated_ffn(lm, c, N, K):
    N = N // 16 * 8 if len(c) > 1 else N // 4 // 8 * 8      # (a tile has half as many columns)
    R, E, off = sum(c), len(c), xu.offsets_of(c) if len(c) > 1 else None
    x, wg, wu = normal((R, K), 1), normal((E, N, K), 2, 2 * K ** -0.5), normal((E, N, K), 3, K ** -0.5)
    bufs = [buffer(R, N, BF16) for _ in range(3)]
    lm.lmoe_gated_ffn(x, wg, wu, *[b[1] for b in bufs], offsets=off)
    for (whole, got), (want, tol), name in zip(bufs, xu.gated(x, wg, wu, off), "hgu"):
        close(got, want, tol, name)
        assert bool((whole[R:] == 7.25).all())
    assert lm.lmoe_bf16_check_status() == (0, 0)


@pytest.mark.parametrize("c,N,K", SIZES, ids=IDS)
@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
def test_gated_ffn_grad(lm, c, N, K, in_place):
    R, E, off = sum(c), len(c), xu.offsets_of(c) if len(c) > 1 else None
    dy, wd, g, u = normal((R, K), 1, 1e-2), normal((E, K, N), 2, N ** -0.5), normal((R, N), 3, 3), normal((R, N), 4)
    want = xu.gated_grad(dy, wd, g, u, off)
    bufs = [buffer(R, N, BF16) for _ in range(2)]
    if in_place:
        for b, src in zip(bufs, (g, u)):
            b[1].copy_(src)
        g, u = bufs[0][1], bufs[1][1]
    lm.lmoe_gated_ffn_grad(dy, wd, g, u, bufs[0][1], bufs[1][1], offsets=off)
    for (whole, got), (v, tol), name in zip(bufs, want, ("dgate", "dup")):
        close(got, v, tol, name)
        assert bool((whole[R:] == 7.25).all())
    assert lm.lmoe_bf16_check_status() == (0, 0)


@pytest.mark.parametrize("c,N,K", [([257, 0, 443], 3000, 1000), ([1], 5000, 4104), ([15, 1, 16, 17], 2824, 1032), ([1000], 4104, 5000),
                                   ([63, 65, 64, 200], 2568, 1288)])
@OUT
@pytest.mark.parametrize("accumulate", [False, True], ids=["new", "added"])
def test_weight_gradients(lm, c, N, K, out, accumulate):
    R, E, off = sum(c), len(c), xu.offsets_of(c) if len(c) > 1 else None
    dy, dy2, x, start = ints((R, N), 1), ints((R, N), 2), ints((R, K), 3), ints((E, N, K), 4)
    bufs = [torch.cat([start.flatten().to(out), torch.full((64,), 7.25, dtype=out, device="cuda")]) for _ in range(2)]
    dw, dw2 = (b[:-64].view(E, N, K) for b in bufs)
    lm.lmoe_matmul_bf16_wgrad(dy, x, dw, offsets=off, dy2=dy2, dw2=dw2, accumulate=accumulate)
    for got, d in ((dw, dy), (dw2, dy2)):
        want = xu.wgrad(d, x, E, off)[0] + (start.double() if accumulate else 0)
        assert torch.equal(got, want.float().to(out))
    assert all(bool((b[-64:] == 7.25).all()) for b in bufs)
    assert lm.lmoe_bf16_check_status() == (0, 0)
