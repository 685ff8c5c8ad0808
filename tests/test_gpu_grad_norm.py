"""The norm over many tensors and the clip, against 64 bits.  The norm's bound: a thread sums at most 64 squares in fp32
(each addition and multiplication off by 2^-24, all terms positive: at most 65 2^-24 of a partial sum), the rest is fp64,
the square root halves it, and one rounding to fp32 is added: 34 2^-24."""
import pytest
import torch

import expert_util as xu
from expert_util import BF16, close

pytestmark = pytest.mark.gpu
F32 = torch.float32
NORM = 34 * 2.0 ** -24


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


def normal(n, dtype, seed, std=1.0):
    return (torch.randn(n, generator=gen(seed), device="cuda") * std).to(dtype)


def packed(sizes, dtypes, seed, base=0, std=1.0):
    """Tensors of those sizes, one behind the other from element ``base`` on, with guard elements around."""
    out = []
    for kind in (F32, BF16):
        mine = [i for i, d in enumerate(dtypes) if d == kind]
        flat = torch.full((base + sum(sizes[i] for i in mine) + 16,), 77.0, dtype=kind, device="cuda")
        at = base
        for i in mine:
            flat[at:at + sizes[i]] = normal(sizes[i], kind, seed * 1000 + i, std)
            out.append((i, flat[at:at + sizes[i]], flat))
            at += sizes[i]
    out.sort(key=lambda v: v[0])
    return [t for _, t, _ in out], {id(f): f for _, _, f in out}.values()


def workspace(lm, n):
    return torch.full((lm.lmoe_grad_norm_workspace_size(n),), 0xff, dtype=torch.uint8, device="cuda")


def check(lm, grads, max_norm, out=None):
    """Norm and clip by every way, against 64 bits."""
    want = xu.norm(grads)
    norm, ws = torch.full((1,), -1.0, device="cuda"), workspace(lm, len(grads))
    lm.lmoe_grad_norm(grads, norm, ws)
    assert abs(float(norm) - float(want)) <= NORM * float(want) + 2.0 ** -149, (float(norm), float(want))
    expect = [xu.clipped(g, norm, max_norm) for g in grads]
    outs = [torch.zeros_like(g) for g in grads] if out is None else out
    lm.lmoe_grad_clip(grads, norm, max_norm, out=outs)
    for o, (v, tol) in zip(outs, expect):
        close(o, v, tol)
    both, again = torch.full((1,), -1.0, device="cuda"), [torch.zeros_like(g) for g in grads]
    lm.lmoe_clip_grad_norm(grads, both, max_norm, ws, out=again)
    assert torch.equal(both, norm)
    for o, a in zip(outs, again):
        assert torch.equal(o, a)
    lm.lmoe_clip_grad_norm(grads, both, max_norm, ws)      # in place
    assert torch.equal(both, norm)
    for o, g in zip(outs, grads):
        assert torch.equal(o, g)


SIZES = [[1], [7], [8], [9], [2047], [2048], [16384], [16385], [100000, 3, 0, 1, 16, 33333], [0, 0, 5],
         [i % 37 for i in range(70)], [1 + i % 500 for i in range(1500)], [1 << 20, 12345, 1 << 16]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("base", [0, 1, 3])
@pytest.mark.parametrize("max_norm", [0.5, 1e6])
def test_norm_and_clip(lm, sizes, kind, base, max_norm):
    dtypes = [{"f32": F32, "bf16": BF16, "mixed": (F32, BF16)[i % 2]}[kind] for i in range(len(sizes))]
    grads, flats = packed(sizes, dtypes, len(sizes) + base, base)
    check(lm, grads, max_norm)
    for f in flats:   # elements around the tensors stay
        assert bool((f[:base] == 77).all()) and bool((f[-16:] == 77).all())


@pytest.mark.parametrize("kind", [F32, BF16], ids=["f32", "bf16"])
def test_outputs_aligned_otherwise(lm, kind):
    grads, _ = packed([1000, 5, 4097], [kind] * 3, 1, 1)
    flat = torch.full((6000,), 5.0, dtype=kind, device="cuda")
    outs = [flat[2:1002], flat[1005:1010], flat[1010:5107]]
    check(lm, grads, 0.25, outs)
    assert bool((flat[:2] == 5).all()) and bool((flat[1002:1005] == 5).all()) and bool((flat[5107:] == 5).all())


@pytest.mark.parametrize("kind", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-22, 1e-15, 1e15, 1e19, 3e30])
def test_squares_beyond_fp32(lm, kind, scale):
    grads = [normal(5000, kind, 1, scale), normal(3, kind, 2, scale), torch.zeros(4000, dtype=kind, device="cuda")]
    want, norm = xu.norm(grads), torch.zeros(1, device="cuda")
    lm.lmoe_grad_norm(grads, norm, workspace(lm, 3))
    assert abs(float(norm) - float(want)) <= NORM * float(want) + 2.0 ** -149
    # one large value among small ones, and the other way round
    grads[0][777] = 1e18
    want = xu.norm(grads)
    lm.lmoe_grad_norm(grads, norm, workspace(lm, 3))
    assert abs(float(norm) - float(want)) <= NORM * float(want)


def test_norm_beyond_fp32_infinities_and_nan(lm):
    big = [torch.full((1000,), 3e38, device="cuda"), normal(100, F32, 1)]
    norm, ws = torch.zeros(1, device="cuda"), workspace(lm, 4)
    lm.lmoe_grad_norm(big, norm, ws)
    assert float(norm) == float("inf")
    outs = [torch.ones_like(g) for g in big]
    lm.lmoe_clip_grad_norm(big, norm, 1.0, ws, out=outs)
    assert bool((outs[0] == 0).all()) and bool((outs[1] == 0).all())
    for bad, kind in ((float("inf"), F32), (float("nan"), BF16), (-float("inf"), BF16)):
        for at in (0, 3, 1000, 4998):
            g = [normal(5000, kind, 2)[1:], normal(64, F32, 3)]
            g[0][at] = bad
            outs = [torch.zeros_like(t) for t in g]
            lm.lmoe_clip_grad_norm(g, norm, 1.0, ws, out=outs)
            if bad != bad:
                assert bool(torch.isnan(norm).all()) and all(bool(torch.isnan(o).all()) for o in outs)
            else:
                assert float(norm) == float("inf") and bool(torch.isnan(outs[0][at]))
                outs[0][at] = 0
                assert all(bool((o == 0).all()) for o in outs)


def test_nothing_to_clip(lm):
    norm, ws = torch.full((1,), 5.0, device="cuda"), workspace(lm, 3)
    for grads in ([], [torch.zeros(0, device="cuda")], [torch.zeros(100, device="cuda", dtype=BF16)]):
        norm.fill_(5)
        lm.lmoe_clip_grad_norm(grads, norm, 1.0, ws)
        assert float(norm) == 0
        norm.fill_(5)
        lm.lmoe_grad_norm(grads, norm, ws)
        assert float(norm) == 0
    g = normal(1000, F32, 1)
    keep = g.clone()
    lm.lmoe_clip_grad_norm([g], norm, 0.0, ws)
    assert bool((g == 0).all())
    g.copy_(keep)
    lm.lmoe_clip_grad_norm([g], norm, float("inf"), ws)
    assert torch.equal(g, keep)


def test_any_iterable_of_tensors(lm):
    grads = [normal(100, F32, i) for i in range(3)]
    norm, again, ws = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda"), workspace(lm, 3)
    lm.lmoe_grad_norm(grads, norm, ws)
    lm.lmoe_grad_norm((g for g in grads), again, ws)
    assert float(norm) > 0 and torch.equal(norm, again)
    outs = [torch.zeros_like(g) for g in grads]
    lm.lmoe_clip_grad_norm(iter(grads), again, 0.5, ws, out=iter(outs))
    for g, o in zip(grads, outs):
        v, tol = xu.clipped(g, norm, 0.5)
        close(o, v, tol)


def test_lists_that_do_not_fit(lm):
    g, norm, ws = torch.ones(64, device="cuda"), torch.ones(1, device="cuda"), workspace(lm, 3)
    out = torch.zeros(64, device="cuda")

    class Mine(torch.Tensor):
        pass
    for grads, match in (([g, g.cpu()], "grads: all tensors must be on cuda:0"), ([g, g[::2]], "grads: tensors must be contiguous"),
                         ([g.half()], "grads: tensors must be float32 or bfloat16"), ([g, None], "grads: element 1 is not a tensor"),
                         ([g.to_sparse()], "grads: tensors must be contiguous")):
        for call in (lambda: lm.lmoe_grad_norm(grads, norm, ws), lambda: lm.lmoe_grad_clip(grads, norm, 0.5),
                     lambda: lm.lmoe_clip_grad_norm(grads, norm, 0.5, ws)):
            with pytest.raises(ValueError, match=match):
                call()
    for o, match in (([out, out], "out: as many"), ([], "out: as many"), ([out[:32]], "out: sizes"), ([out.bfloat16()], "out: sizes"),
                     ([out.cpu()], "out: all tensors")):
        with pytest.raises(ValueError, match=match):
            lm.lmoe_clip_grad_norm([g], norm, 0.5, ws, out=o)
    assert bool((g == 1).all()) and bool((norm == 1).all()) and bool((out == 0).all())
    grads = [torch.nn.Parameter(g.clone()), g.clone().as_subclass(Mine), g.clone().reshape(8, 8).t().contiguous()]
    lm.lmoe_clip_grad_norm(grads, norm, 1.0, ws)
    v, tol = xu.clipped(g, norm, 1.0)
    for t in grads:
        close(t.detach().as_subclass(torch.Tensor).reshape(-1), v, tol)


def test_overlapping_outputs_are_refused(lm):
    flat = torch.ones(1000, device="cuda")
    norm, ws = torch.ones(1, device="cuda"), workspace(lm, 3)
    a, b = flat[:600], flat[500:]
    other = torch.zeros(1000, device="cuda")
    for grads, out in (([a, b], None), ([flat, flat], None), ([a], [flat[1:601]]), ([a, a], [other[:600], other[400:]])):
        for call in (lambda: lm.lmoe_grad_clip(grads, norm, 0.5, out=out),
                     lambda: lm.lmoe_clip_grad_norm(grads, norm, 0.5, ws, out=out)):
            with pytest.raises(lm.LmoeError) as e:
                call()
            assert e.value.status == -1
    assert bool((flat == 1).all()) and bool((other == 0).all())
    lm.lmoe_grad_norm([a, b, flat], norm, ws)       # read alone: any overlap counts as often as it is named
    assert abs(float(norm) - 2100 ** 0.5) < 1e-4
    outs = [torch.zeros(600, device="cuda") for _ in range(2)]
    lm.lmoe_grad_clip([a, a], torch.full((1,), 2.0, device="cuda"), 1.0, out=outs)   # (each read for an output of its own)
    assert torch.equal(outs[0], outs[1]) and bool(((outs[0] - 0.5).abs() < 1e-6).all())


def test_a_captured_step(lm):
    """Accumulated gradients clipped in a graph, replayed: a larger call and another graph's share no workspace."""
    grads = [normal(70000, F32, 1), normal(333, BF16, 2), normal(4097, F32, 3)]
    norm = torch.zeros(1, device="cuda")
    ws = workspace(lm, 3)
    fresh = [g.clone() for g in grads]
    graph = torch.cuda.CUDAGraph()
    lm.lmoe_clip_grad_norm([g.clone() for g in grads], norm, 1.0, ws)
    with torch.cuda.graph(graph):
        lm.lmoe_clip_grad_norm(grads, norm, 1.0, ws)
    for scale in (1.0, 0.5):
        for g, f in zip(grads, fresh):
            g.copy_(f * scale)
        want = xu.norm(grads)
        graph.replay()
        assert abs(float(norm) - float(want)) <= NORM * float(want)
        for g, f in zip(grads, fresh):
            v, tol = xu.clipped(f * scale, norm, 1.0)
            close(g, v, tol)


def test_more_than_32_bits_of_bytes(lm):
    n = (1 << 31) + 12345
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[0], g[1 << 30], g[n - 1] = 3, 4, 12
    norm = torch.zeros(1, device="cuda")
    lm.lmoe_clip_grad_norm([g], norm, 1.0, workspace(lm, 1))
    assert float(norm) == 13
    for at, v in ((0, 3), (1 << 30, 4), (n - 1, 12)):
        assert abs(float(g[at]) * 13 - v) <= 2.0 ** -7 * v
    assert int(torch.count_nonzero(g[: 1 << 30])) == 1 and int(torch.count_nonzero(g[1 << 30:])) == 2
