"""8-bit quantisers and products against plain forms in 64 bits.

Quantisers: the rule has one outcome, so scales and codes are compared exactly.  Products: fed with
codes that are small integers and scales that are powers of two, every sum is exact in fp32 (below
2^24 steps), whatever its order, so layouts and edges are compared exactly (bf16: one rounding); with
random operands the error is bounded by that of an fp32 sum in any order (train_util.product)."""
import pytest
import torch

import train_util as tu
from train_util import E4M3, E5M2, assert_close

pytestmark = pytest.mark.gpu
FMT = pytest.mark.parametrize("fmt", [E4M3, E5M2], ids=["e4m3", "e5m2"])
TYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


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


def source(rows, K, dtype, seed=0, pad=0, base=0):
    """[rows, K] of widely spread magnitudes, some zeros, rows of K + pad from element ``base`` on."""
    g = gen(seed * 100003 + rows * 31 + K)
    buf = torch.full((base + rows * (K + pad) + 16,), float("nan"), device="cuda", dtype=dtype)
    x = buf[base:base + rows * (K + pad)].view(rows, K + pad)[:, :K]
    v = torch.randn(rows, K, generator=g, device="cuda") * torch.exp(3 * torch.randn(rows, K, generator=g, device="cuda"))
    v[torch.rand(rows, K, generator=g, device="cuda") < 0.1] = 0
    x.copy_(v)
    return x


def bytes_(fmt, *shape, fill=0x5a):
    return torch.full(shape, fill, dtype=torch.uint8, device="cuda").view(fmt)


def same_codes(got, want, what=""):
    assert torch.equal(got.double() + 0.0, want + 0.0), what   # (-0 and 0 are the same value)


# ------------------------------------------------------------------ rows
def check_rows(lm, src, fmt, index=None, pow2=False):
    x = tu.gathered(src, index)
    R, K = x.shape
    codes, scales = bytes_(fmt, R, K), torch.full((-(-K // 128), R), -1.0, device="cuda")
    lm.lmoe_quantize_fp8_rows(src, codes, scales, index, pow2)
    q, s = tu.quantize_rows(x, fmt, pow2)
    assert torch.equal(scales.double(), s), "scales"
    same_codes(codes, q, "codes")
    # a value is off by at most half a step, or half the smallest step of its block
    tol = tu.HALF[fmt] * x.abs() + s.t().repeat_interleave(128, 1)[:, :K] * (2.0 ** -10 if fmt == E4M3 else 2.0 ** -17)
    assert_close(tu.values(codes, scales, False), x, tol * (1 + 1e-6), "values")


@FMT
@TYPES
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 4096), (3, 128), (16, 144), (17, 272), (100, 2048), (129, 1040), (8, 7168)])
def test_rows(lm, rows, K, dtype, fmt):
    check_rows(lm, source(rows, K, dtype), fmt)
    check_rows(lm, source(rows, K, dtype, 1), fmt, pow2=True)


@TYPES
@pytest.mark.parametrize("pad,base", [(0, 1), (8, 0), (4, 0), (1, 0), (2, 2), (0, 4)])
def test_rows_strided_and_unaligned(lm, pad, base, dtype):
    check_rows(lm, source(37, 400, dtype, pad=pad, base=base), E4M3)


@TYPES
def test_rows_gathered(lm, dtype):
    src = source(50, 528, dtype)
    idx = torch.randint(0, 50, (333,), generator=gen(1), device="cuda").int()
    check_rows(lm, src, E4M3, idx)
    idx[::7], idx[3::11] = -1, 50            # outside: rows of zeros
    idx[-1] = 2 ** 31 - 1
    check_rows(lm, src, E5M2, idx)
    check_rows(lm, source(60, 528, dtype)[:5], E4M3)                      # more rows in memory than asked for
    check_rows(lm, src[:0], E4M3, torch.zeros(9, dtype=torch.int32, device="cuda"))   # nothing to gather from
    check_rows(lm, src, E4M3, idx[:0])


@FMT
@TYPES
def test_rows_special_values(lm, dtype, fmt):
    src = source(12, 384, dtype)
    src[0] = 0                                            # a block of zeros: the smallest scale
    src[1, 128:256] = 2.0 ** -130                          # below it
    src[2] = torch.finfo(dtype).max
    src[3] = -torch.finfo(dtype).max
    src[4, 5] = 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149
    src[5, ::2] = torch.finfo(dtype).tiny
    for pow2 in (False, True):
        check_rows(lm, src, fmt, pow2=pow2)
    src[6, 0], src[7, 200], src[8, 383] = float("inf"), float("nan"), -float("inf")
    codes, scales = bytes_(fmt, 12, 384), torch.zeros(3, 12, device="cuda")
    for pow2 in (False, True):
        lm.lmoe_quantize_fp8_rows(src, codes, scales, None, pow2)
        bad = torch.zeros(3, 12, dtype=torch.bool, device="cuda")
        bad[0, 6] = bad[1, 7] = bad[2, 8] = True
        assert torch.equal(~torch.isfinite(scales), bad)   # those blocks and no others
        clean = torch.where(torch.isfinite(src), src, 0.0)
        q, s = tu.quantize_rows(clean.double(), fmt, pow2)
        assert torch.equal(torch.where(bad, s.float(), scales).double(), s)
        keep = (~bad).t().repeat_interleave(128, 1)
        assert torch.equal(torch.where(keep, codes.double(), 0.0), torch.where(keep, q, 0.0))


# ------------------------------------------------------------------ weights
@FMT
@TYPES
@pytest.mark.parametrize("E,N,K", [(1, 16, 16), (1, 128, 128), (3, 144, 400), (2, 1000, 272), (1, 1, 2048), (5, 130, 128)])
def test_weight(lm, E, N, K, dtype, fmt):
    src = source(E * N, K, dtype).view(E, N, K)
    for pow2 in (False, True):
        both = N % 16 == 0
        codes, scales = bytes_(fmt, E, N, K), torch.full((E, -(-N // 128), -(-K // 128)), -1.0, device="cuda")
        ct, st = bytes_(fmt, E, K, N), torch.full((E, -(-K // 128), -(-N // 128)), -1.0, device="cuda")
        lm.lmoe_quantize_fp8_weight(src, codes, scales, ct if both else None, st if both else None, pow2)
        for e in range(E):
            q, s = tu.quantize_weight(src[e].double(), fmt, pow2)
            assert torch.equal(scales[e].double(), s)
            same_codes(codes[e], q)
        if both:
            assert torch.equal(ct.view(torch.uint8), codes.view(torch.uint8).transpose(1, 2))
            assert torch.equal(st, scales.transpose(1, 2))


@TYPES
def test_weight_two_dimensional_and_unaligned(lm, dtype):
    buf = source(1, 96 * 160 + 8, dtype)[0]
    for base in (0, 1, 2):
        src = buf[base:base + 96 * 160].view(96, 160)
        codes, scales, ct, st = bytes_(E4M3, 96, 160), torch.zeros(1, 2, device="cuda"), bytes_(E4M3, 160, 96), \
            torch.zeros(2, 1, device="cuda")
        lm.lmoe_quantize_fp8_weight(src, codes, scales, ct, st)
        q, s = tu.quantize_weight(src.double(), E4M3)
        assert torch.equal(scales.double(), s)
        same_codes(codes, q)
        same_codes(ct, q.t())


def test_weight_many_matrices(lm):
    src = source(1500 * 16, 16, torch.float32).view(1500, 16, 16)
    codes, scales = bytes_(E4M3, 1500, 16, 16), torch.zeros(1500, 1, 1, device="cuda")
    lm.lmoe_quantize_fp8_weight(src, codes, scales)
    q, s = tu.rule(src.double(), (1, 2), E4M3)
    assert torch.equal(scales.double(), s)
    same_codes(codes, q)


# ------------------------------------------------------------------ columns
def split(R, E, seed, empty=0.3):
    """offsets [E + 1] of an uneven split, some experts without rows."""
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(E, generator=g) * (torch.rand(E, generator=g) > empty)
    w[int(torch.randint(0, E, (1,), generator=g))] += 0.5
    c = torch.bincount(torch.multinomial(w, max(R, 1), replacement=True, generator=g), minlength=E) if R else torch.zeros(E)
    return torch.cat([torch.zeros(1), c.cumsum(0)]).int().cuda()


def check_cols(lm, src, fmt, offsets, index=None, pow2=False):
    x = tu.gathered(src, index)
    (R, K), E = x.shape, 1 if offsets is None else len(offsets) - 1
    Rp = lm.lmoe_fp8_padded_rows(R, E)
    codes, scales = bytes_(fmt, K, Rp), torch.full((Rp // 128, K), -1.0, device="cuda")
    lm.lmoe_quantize_fp8_cols(src, codes, scales, offsets, index, pow2)
    q, s = tu.quantize_cols(x, offsets, fmt, pow2)
    n = q.shape[1]
    assert torch.equal(scales[:n // 128].double(), s)
    same_codes(codes[:, :n], q)
    # behind the last expert's blocks: as they were
    assert bool((codes[:, n:].view(torch.uint8) == 0x5a).all()) and bool((scales[n // 128:] == -1).all())


@FMT
@TYPES
@pytest.mark.parametrize("R,E,K", [(1, 1, 16), (1, 9, 128), (127, 1, 144), (128, 1, 272), (129, 2, 400), (1000, 7, 528),
                                   (60, 200, 64), (900, 1024, 32), (300, 3, 2048)])
def test_cols(lm, R, E, K, dtype, fmt):
    check_cols(lm, source(R, K, dtype), fmt, split(R, E, R + E))
    check_cols(lm, source(R, K, dtype), fmt, split(R, E, R + E + 1), pow2=True)


@TYPES
def test_cols_one_group_strided_gathered(lm, dtype):
    check_cols(lm, source(300, 176, dtype), E5M2, None)
    for pad, base in ((4, 0), (1, 0), (0, 1), (2, 2)):
        check_cols(lm, source(200, 176, dtype, pad=pad, base=base), E4M3, split(200, 4, 3))
    idx = torch.randint(-3, 44, (500,), generator=gen(3), device="cuda").int()   # some outside [0, 40)
    check_cols(lm, source(40, 176, dtype), E5M2, split(500, 6, 5), idx)


def test_cols_bad_offsets_are_clamped(lm):
    # offsets below zero, past the rows, and decreasing: clamped, nothing behind the padded rows is touched
    src = source(100, 64, torch.float32)
    for offs in ([0, 40, 1000], [-50, 60, 100], [50, 20, 100], [100, 100, 100], [0, 2 ** 31 - 1, -2 ** 31]):
        check_cols(lm, src, E4M3, torch.tensor(offs, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ products
def integers(shape, fmt, seed, lo=-4, hi=4):
    return torch.randint(lo, hi + 1, shape, generator=gen(seed), device="cuda").float().to(fmt)


def powers(shape, seed):
    return torch.exp2(torch.randint(-2, 3, shape, generator=gen(seed), device="cuda").float())


def matmul_case(R, E, N, K, af, wf, seed=0, exact=True):
    kb, nb = -(-K // 128), -(-N // 128)
    if exact:
        # terms are multiples of 2^-4 below 2^8, so that sums of up to 4096 stay below 2^24 steps
        a, w = integers((R, K), af, seed + 1), integers((E, N, K), wf, seed + 2)
        return a, powers((kb, R), seed + 3), w, powers((E, nb, kb), seed + 4)
    a = (torch.randn(R, K, generator=gen(seed + 1), device="cuda") * 60).to(af)
    w = (torch.randn(E, N, K, generator=gen(seed + 2), device="cuda") * 60).to(wf)
    return a, torch.rand(kb, R, generator=gen(seed + 3), device="cuda") + 0.1, w, \
        torch.rand(E, nb, kb, generator=gen(seed + 4), device="cuda") + 0.1


def check_matmul(lm, a, a_s, w, w_s, offsets, out_dtype, exact, out=None, stream=None):
    R, (E, N, _) = a.shape[0], w.shape
    y = out if out is not None else torch.full((R, N), 7.25, dtype=out_dtype, device="cuda")
    y.fill_(7.25)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w1, s1 = (w, w_s) if offsets is not None else (w[0], w_s[0])
    lm.lmoe_matmul_fp8(a, a_s, w1, s1, y, offsets=offsets, status=status, stream=stream)
    torch.cuda.synchronize()
    assert int(status) == 0
    done = torch.zeros(R, dtype=torch.bool, device="cuda")
    av = tu.values(a, a_s, False)
    for e, (lo, hi) in enumerate(tu.groups(offsets, R)):
        if hi <= lo:
            continue
        done[lo:hi] = True
        want, tol = tu.product(av[lo:hi], tu.values(w[e], w_s[e], True))
        if exact:
            assert torch.equal(y[lo:hi], want.to(torch.float32).to(out_dtype)), (e, lo, hi)
        else:
            assert_close(y[lo:hi], want, tol + tu.HALF[out_dtype] * (want.abs() + tol), f"expert {e}")
    assert bool((y[~done] == 7.25).all())   # rows of no expert: as they were
    return y


# every kind of tile: one row to 16, few rows split along K, few rows per expert, many; ragged ends in
# rows (below, at and behind a tile), columns (odd N: scattered stores) and K (short blocks)
DENSE = [(1, 1, 16), (1, 128, 128), (1, 4096, 2048), (8, 200, 144), (16, 129, 1040), (17, 64, 256), (33, 1000, 4096),
         (63, 2048, 2064), (65, 256, 512), (127, 513, 400), (128, 8192, 256), (129, 5000, 272), (1000, 5001, 144), (700, 4096, 1024)]


@pytest.mark.parametrize("R,N,K", DENSE)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_matmul_dense(lm, R, N, K, out):
    check_matmul(lm, *matmul_case(R, 1, N, K, E4M3, E4M3), None, out, True)
    check_matmul(lm, *matmul_case(R, 1, N, K, E5M2, E4M3, 7, exact=False), None, out, False)


GROUPED = [(1, 4, 256, 128), (8, 64, 512, 256), (16, 3, 200, 400), (40, 200, 144, 256), (200, 2, 4100, 2048), (300, 5, 1003, 528),
           (900, 7, 5120, 144), (2000, 9, 600, 272), (700, 1024, 48, 64), (3000, 3, 5000, 144)]


@pytest.mark.parametrize("R,E,N,K", GROUPED)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_matmul_grouped(lm, R, E, N, K, out):
    check_matmul(lm, *matmul_case(R, E, N, K, E5M2, E5M2), split(R, E, R), out, True)
    check_matmul(lm, *matmul_case(R, E, N, K, E4M3, E5M2, 5, exact=False), split(R, E, R + 1), out, False)


@pytest.mark.parametrize("R,N", [(5, 640), (90, 1100), (1500, 5000)])
def test_rows_of_no_expert_are_left(lm, R, N):
    a = matmul_case(R, 3, N, 272, E4M3, E4M3)
    for offs in ([R // 3, R // 2, R // 2, R - 1], [0, 0, 0, 0], [R, R, R, R], [-9, 2, 2, R + 50], [1, 1, 2, 3]):
        check_matmul(lm, *a, torch.tensor(offs, dtype=torch.int32, device="cuda"), torch.bfloat16, True)


@pytest.mark.parametrize("R,E,N,K", [(5, 4, 131, 144), (33, 2, 257, 272), (60, 30, 130, 144), (70, 3, 131, 400), (500, 40, 136, 160)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_tiles_that_end_with_the_rows(lm, R, E, N, K, out):
    # experts whose tiles reach past the last row start earlier and leave the rows before their own alone
    a = matmul_case(R, E, N, K, E4M3, E4M3)
    last = torch.full((E + 1,), R, dtype=torch.int32, device="cuda")
    last[:-1] = torch.arange(E, device="cuda").int() + R - E          # one row each, the last rows
    for offs in (split(R, E, 3, empty=0.0), last, torch.clamp(last, max=R - 1)):
        check_matmul(lm, *a, offs, out, True)
        buf = torch.full((3 + R * N,), 7.25, dtype=out, device="cuda")
        check_matmul(lm, *a, offs, out, True, out=buf[3:].view(R, N))
        assert bool((buf[:3] == 7.25).all())


def test_matmul_bad_offsets_are_clamped(lm):
    for R, N in ((12, 256), (200, 700), (1200, 5000)):
        a = matmul_case(R, 2, N, 144, E4M3, E4M3)
        y = torch.full((R + 64, N), 7.25, device="cuda")
        for offs in ([0, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, R // 2, R], [-5, -5, R + 7]):
            check_matmul(lm, *a, torch.tensor(offs, dtype=torch.int32, device="cuda"), torch.float32, True, out=y[:R])
            assert bool((y[R:] == 7.25).all())


@pytest.mark.parametrize("R,N,K", [(3, 128, 4096), (12, 256, 4096), (200, 700, 2048), (1200, 5000, 144)])
def test_matmul_offsets_that_go_back_end_in_bounds(lm, R, N, K):
    # decreasing offsets name rows several times: the products are anyone's, but the call ends, reports
    # nothing and writes rows 0 .. R - 1 only (the first two sizes split K over a cluster)
    E = 6
    a, a_s, w, w_s = matmul_case(R, E, N, K, E4M3, E4M3)
    y = torch.full((R + 64, N), 7.25, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for offs in ([0, R, 0, R, 0, R, 0], [R, 0, R, 0, R, 0, R], [0, R, 1, R, 2, R, R]):
        off = torch.tensor(offs, dtype=torch.int32, device="cuda")
        lm.lmoe_matmul_fp8(a, a_s, w, w_s, y[:R], offsets=off, status=status)
        torch.cuda.synchronize()
        assert int(status) == 0 and bool((y[R:] == 7.25).all())


@pytest.mark.parametrize("R,N,K", [(3, 264, 256), (50, 1000, 400), (600, 5000, 256)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_matmul_output_at_any_element(lm, R, N, K, out):
    for base in (1, 3):
        buf = torch.full((base + R * N + 16,), 7.25, dtype=out, device="cuda")
        check_matmul(lm, *matmul_case(R, 1, N, K, E4M3, E4M3), None, out, True, out=buf[base:base + R * N].view(R, N))
        assert bool((buf[:base] == 7.25).all()) and bool((buf[base + R * N:] == 7.25).all())


def test_matmul_no_rows(lm):
    a, a_s, w, w_s = matmul_case(0, 1, 64, 128, E4M3, E4M3)
    lm.lmoe_matmul_fp8(a, a_s, w[0], w_s[0], torch.zeros(0, 64, device="cuda"))


def test_not_finite_scales_stay_in_their_rows(lm):
    for R, N, K in ((6, 256, 256), (100, 640, 400), (600, 5000, 256)):
        a, a_s, w, w_s = matmul_case(R, 1, N, K, E4M3, E4M3)
        clean = check_matmul(lm, a, a_s, w, w_s, None, torch.float32, True).clone()
        a_s[1, R // 2] = float("inf")
        y = torch.zeros(R, N, device="cuda")
        lm.lmoe_matmul_fp8(a, a_s, w[0], w_s[0], y)
        keep = torch.arange(R, device="cuda") != R // 2
        assert torch.equal(y[keep], clean[keep])
        assert not bool(torch.isfinite(y[R // 2]).all())


# ------------------------------------------------------------------ weight gradients
def wgrad_case(lm, R, E, N, K, yf, xf, seed=0, exact=True):
    """Padded, blocked operands for a split of R rows; offsets; padded rows of each expert."""
    offsets = split(R, E, R + E + seed)
    Rp = lm.lmoe_fp8_padded_rows(R, E)
    live = torch.zeros(Rp, dtype=torch.bool, device="cuda")
    ranges, at = [], 0
    for lo, hi in tu.groups(offsets, R):
        live[at:at + hi - lo] = True
        n = -(-(hi - lo) // 128) * 128
        ranges.append((at, at + n))
        at += n
    if exact:
        dy, x = integers((N, Rp), yf, seed + 1), integers((K, Rp), xf, seed + 2)
        ds, xs = powers((Rp // 128, N), seed + 3), powers((Rp // 128, K), seed + 4)
    else:
        dy = (torch.randn(N, Rp, generator=gen(seed + 1), device="cuda") * 60).to(yf)
        x = (torch.randn(K, Rp, generator=gen(seed + 2), device="cuda") * 60).to(xf)
        ds = torch.rand(Rp // 128, N, generator=gen(seed + 3), device="cuda") + 0.1
        xs = torch.rand(Rp // 128, K, generator=gen(seed + 4), device="cuda") + 0.1
    dy.view(torch.uint8)[:, ~live] = 0
    x.view(torch.uint8)[:, ~live] = 0
    if at < Rp:   # behind the last expert's blocks anything may stand
        dy.view(torch.uint8)[:, at:] = 0x7f
        x.view(torch.uint8)[:, at:] = 0x7f
        ds[at // 128:] = xs[at // 128:] = float("nan")
    return dy, ds, x, xs, offsets, ranges


def check_wgrad(lm, case, N, K, out_dtype, exact, accumulate=False, dw=None):
    dy, ds, x, xs, offsets, ranges = case
    E = len(ranges)
    if dw is None:
        dw = torch.empty(E, N, K, dtype=out_dtype, device="cuda")
    before = torch.randint(-9, 9, (E, N, K), generator=gen(5), device="cuda").to(out_dtype)
    dw.copy_(before)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lm.lmoe_matmul_fp8_wgrad(dy, ds, x, xs, dw, offsets=offsets, accumulate=accumulate, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for e, (lo, hi) in enumerate(ranges):
        was = before[e].double() if accumulate else 0.0
        if hi == lo:
            assert bool((dw[e].double() == was).all())
            continue
        b = slice(lo // 128, hi // 128)
        want, tol = tu.product(tu.values(dy[:, lo:hi], ds[b], False), tu.values(x[:, lo:hi], xs[b], False))
        if exact:
            assert torch.equal(dw[e], (want + was).to(torch.float32).to(out_dtype)), e
        else:
            want = want + was
            assert_close(dw[e], want, tol + (want.abs() + tol) * (tu.HALF[out_dtype] + 2.0 ** -23), f"expert {e}")


WGRAD = [(1, 1, 16, 16), (1, 5, 128, 128), (128, 1, 256, 100), (129, 1, 130, 257), (1000, 3, 200, 400), (1500, 16, 144, 513),
         (60, 300, 64, 48), (700, 1024, 17, 16), (4000, 2, 1000, 1030), (512, 2, 3000, 256)]


@pytest.mark.parametrize("R,E,N,K", WGRAD)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_wgrad(lm, R, E, N, K, out):
    check_wgrad(lm, wgrad_case(lm, R, E, N, K, E5M2, E4M3), N, K, out, True)
    check_wgrad(lm, wgrad_case(lm, R, E, N, K, E4M3, E4M3, 3), N, K, out, True, accumulate=True)
    check_wgrad(lm, wgrad_case(lm, R, E, N, K, E5M2, E5M2, 9, exact=False), N, K, out, False, accumulate=R % 2 == 1)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_wgrad_output_at_any_element(lm, out):
    N, K, E = 140, 264, 3
    case = wgrad_case(lm, 400, E, N, K, E5M2, E4M3)
    for base in (1, 3):
        for accumulate in (False, True):
            buf = torch.full((base + E * N * K + 16,), 7.25, dtype=out, device="cuda")
            check_wgrad(lm, case, N, K, out, True, accumulate, dw=buf[base:base + E * N * K].view(E, N, K))
            assert bool((buf[:base] == 7.25).all()) and bool((buf[base + E * N * K:] == 7.25).all())


def test_wgrad_without_rows(lm):
    e = torch.empty
    for E in (1, 3):
        dw = torch.full((E, 40, 50), 3.0, device="cuda")
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        args = (e(40, 0, dtype=E5M2, device="cuda"), e(0, 40, device="cuda"), e(50, 0, dtype=E4M3, device="cuda"),
                e(0, 50, device="cuda"), dw)
        lm.lmoe_matmul_fp8_wgrad(*args, offsets=off, accumulate=True)
        assert bool((dw == 3).all())
        lm.lmoe_matmul_fp8_wgrad(*args, offsets=off)
        assert bool((dw == 0).all())


def test_wgrad_bad_offsets_are_clamped(lm):
    # the same clamping as lmoe_quantize_fp8_cols: what does not fit in the padded rows is left out
    src_y, src_x = source(200, 144, torch.float32), source(200, 80, torch.float32)
    for offs in ([0, 90, 2 ** 31 - 1], [-50, 60, 200], [150, 20, 200], [200, 200, 200]):
        o = torch.tensor(offs, dtype=torch.int32, device="cuda")
        Rp = lm.lmoe_fp8_padded_rows(200, 2)
        dy, ds, x, xs = bytes_(E5M2, 144, Rp, fill=0), torch.zeros(Rp // 128, 144, device="cuda"), \
            bytes_(E4M3, 80, Rp, fill=0), torch.zeros(Rp // 128, 80, device="cuda")
        lm.lmoe_quantize_fp8_cols(src_y, dy, ds, o)
        lm.lmoe_quantize_fp8_cols(src_x, x, xs, o)
        dw = torch.zeros(2, 144, 80, device="cuda")
        lm.lmoe_matmul_fp8_wgrad(dy, ds, x, xs, dw, offsets=o)
        at = 0
        for e, (lo, hi) in enumerate(tu.groups(o, 200)):
            n = -(-(hi - lo) // 128) * 128
            if at + n > Rp:   # (does not happen with offsets that do not overlap)
                break
            b = slice(at // 128, (at + n) // 128)
            want, tol = tu.product(tu.values(dy[:, at:at + n], ds[b], False), tu.values(x[:, at:at + n], xs[b], False))
            assert_close(dw[e], want, tol + 2.0 ** -24 * want.abs(), f"{offs} {e}")
            at += n


# ------------------------------------------------------------------ streams, graphs
def test_same_bits_on_another_stream_and_from_a_graph(lm):
    shapes = [(1, 1, 4096, 4096), (8, 64, 512, 1024), (100, 1, 2048, 4096), (2000, 6, 2048, 512)]
    s = torch.cuda.Stream()
    for R, E, N, K in shapes:
        a, a_s, w, w_s = matmul_case(R, E, N, K, E4M3, E4M3, exact=False)
        off = split(R, E, 1)
        y0, y1 = torch.zeros(R, N, device="cuda"), torch.zeros(R, N, device="cuda")
        lm.lmoe_matmul_fp8(a, a_s, w, w_s, y0, offsets=off)
        torch.cuda.synchronize()
        lm.lmoe_matmul_fp8(a, a_s, w, w_s, y1, offsets=off, stream=s)
        s.synchronize()
        assert torch.equal(y0, y1)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lm.lmoe_matmul_fp8(a, a_s, w, w_s, y1, offsets=off)
        off.copy_(split(R, E, 2))   # another split when it is replayed
        y1.zero_()
        y0.zero_()
        graph.replay()
        lm.lmoe_matmul_fp8(a, a_s, w, w_s, y0, offsets=off)
        assert torch.equal(y0, y1)


def test_two_calls_at_once(lm):
    # two streams, each with its own products, side by side
    c1, c2 = matmul_case(3000, 4, 2048, 1024, E4M3, E4M3, 1), matmul_case(5, 1, 8192, 4096, E4M3, E4M3, 2)
    off = split(3000, 4, 9)
    y1, y2 = torch.zeros(3000, 2048, device="cuda"), torch.zeros(5, 8192, device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        lm.lmoe_matmul_fp8(*c1[:4], y1, offsets=off, stream=s1)
        lm.lmoe_matmul_fp8(c2[0], c2[1], c2[2][0], c2[3][0], y2, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(y1, check_matmul(lm, *c1, off, torch.float32, True))
    assert torch.equal(y2, check_matmul(lm, *c2, None, torch.float32, True))


def test_long_rows_pass_32_bit_offsets(lm):
    # out [2^17 + 5, 2^14 + 8] bf16 has more than 2^31 elements; checked at its first and last rows
    R, N, K = (1 << 17) + 5, (1 << 14) + 8, 128
    a, a_s = integers((R, K), E4M3, 1), powers((1, R), 3)
    w, w_s = integers((1, N, K), E4M3, 2), powers((1, -(-N // 128), 1), 4)
    y = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    lm.lmoe_matmul_fp8(a, a_s, w[0], w_s[0], y)
    wv = tu.values(w[0], w_s[0], True)
    for lo in (0, R // 2, R - 200):
        want = tu.values(a[lo:lo + 200], a_s[:, lo:lo + 200], False) @ wv.t()
        assert torch.equal(y[lo:lo + 200], want.float().bfloat16())


def test_refusals_on_the_device(lm):
    dev = dict(device="cuda")
    s, q, sc = torch.zeros(8, 256, **dev), bytes_(E4M3, 8, 256), torch.zeros(2, 8, **dev)
    w, ws, y = bytes_(E4M3, 2, 64, 256), torch.zeros(2, 1, 2, **dev), torch.zeros(8, 64, **dev)
    off = torch.zeros(3, dtype=torch.int32, **dev)
    d, x, ds, xs = bytes_(E5M2, 64, 256), bytes_(E4M3, 48, 256), torch.zeros(2, 64, **dev), torch.zeros(2, 48, **dev)
    M, W = lm.lmoe_matmul_fp8, lm.lmoe_matmul_fp8_wgrad
    for match, fn in [
            ("codes: dtype", lambda: lm.lmoe_quantize_fp8_rows(s, q.view(torch.uint8), sc)),
            ("scales: shape", lambda: lm.lmoe_quantize_fp8_rows(s, q, sc.t().contiguous())),
            ("codes must be contiguous", lambda: lm.lmoe_quantize_fp8_rows(s, bytes_(E4M3, 256, 8).t(), sc)),
            ("row_index: dtype", lambda: lm.lmoe_quantize_fp8_rows(s, q, sc, torch.zeros(8, dtype=torch.int64, **dev))),
            ("codes: shape", lambda: lm.lmoe_quantize_fp8_rows(s, q, sc, torch.zeros(9, dtype=torch.int32, **dev))),
            ("src must be contiguous", lambda: lm.lmoe_quantize_fp8_weight(s[:, :128], q[:, :128], ws[0, :, :1])),
            ("codes_t: dtype", lambda: lm.lmoe_quantize_fp8_weight(s, q, torch.zeros(1, 2, **dev), bytes_(E5M2, 256, 8))),
            ("codes_t: shape", lambda: lm.lmoe_quantize_fp8_cols(s, bytes_(E4M3, 256, 128), sc, off)),
            ("offsets .E . 1.", lambda: lm.lmoe_quantize_fp8_cols(s, bytes_(E4M3, 256, 128), sc, off[:1])),
            ("a_scales: shape", lambda: M(q, sc.t().contiguous(), w, ws, y, off)),
            ("w_scales: shape", lambda: M(q, sc, w, ws[:1], y, off)),
            ("w: shape", lambda: M(q, sc, w[:, :, :128].contiguous(), ws, y, off)),
            ("out: shape", lambda: M(q, sc, w, ws, y[:, :32].contiguous(), off)),
            ("out: dtype", lambda: M(q, sc, w, ws, y.half(), off)),
            ("offsets: shape", lambda: M(q, sc, w, ws, y, off[:2])),
            ("status: dtype", lambda: M(q, sc, w, ws, y, off, torch.zeros(1, **dev))),
            ("x_t: shape", lambda: W(d, ds, x[:, :128].contiguous(), xs, torch.zeros(64, 48, **dev))),
            ("dy_scales: shape", lambda: W(d, ds[:1], x, xs, torch.zeros(64, 48, **dev))),
            ("dw: shape", lambda: W(d, ds, x, xs, torch.zeros(48, 64, **dev)))]:
        with pytest.raises(ValueError, match=match):
            fn()
    for fn in (lambda: M(q, sc, w, ws, y),                                        # several experts, no offsets
               lambda: lm.lmoe_quantize_fp8_rows(s[:, :248], bytes_(E4M3, 8, 248), sc),   # K no multiple of 16
               lambda: M(bytes_(E4M3, 8 * 256 + 1)[1:].view(8, 256), sc, w, ws, y, off)):  # codes not 16-byte aligned
        with pytest.raises(lm.LmoeError):
            fn()
