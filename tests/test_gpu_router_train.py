"""Router losses and router gradient against plain forms in 64 bits.

Tolerances (U = 2^-24, half a step of fp32): a probability is off by at most U (6 r + 45) of itself, r the
largest magnitude of a logit: the exponent's argument (l - m) log2 e takes three roundings, exp2 two ulps,
the row's sum V + 5 <= 37 additions, then a reciprocal and a product.  Its sums over rows add at most
256 further additions of positive terms (rows of a lane, groups, warps, CTAs, clusters).  lse is off by
U (5 max|l| + 80).  bf16 results take half a step of 2^-8 more.  Counts are exact."""
import pytest
import torch

import train_util as tu
from train_util import U, assert_close

pytestmark = pytest.mark.gpu


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


def made(T, E, k, dtype=torch.float32, seed=0, pad=0, base=0, masked=None, bias=False, spread=2.0):
    """Logits [T, E] with rows of E + pad from element ``base`` on, ids of the k largest, mask, bias."""
    g = gen(1000 * seed + 7 * T + E)
    buf = torch.full((base + T * (E + pad) + 8,), float("nan"), device="cuda", dtype=dtype)
    logits = buf[base:base + T * (E + pad)].view(T, E + pad)[:, :E]
    logits.copy_(spread * torch.randn(T, E, generator=g, device="cuda"))
    b = torch.randn(E, generator=g, device="cuda") if bias else None
    idx = (logits.float() + (0 if b is None else b)).topk(k, 1).indices.int()
    mask = None
    if masked is not None:
        mask = (torch.rand(T, generator=g, device="cuda") >= masked).to(torch.uint8)
    return dict(logits=logits, idx=idx, bias=b, mask=mask, gen=g)


def losses(lm, x, out=None, stream=None):
    T, E = x["logits"].shape
    if out is None:
        out = (torch.full((2,), 9.0, device="cuda"), torch.full((E,), 9.0, device="cuda"),
               torch.full((E + 1,), -9, dtype=torch.int32, device="cuda"),
               torch.full((lm.lmoe_router_losses_workspace_size(T, E),), 0xff, dtype=torch.uint8, device="cuda"))
    ls, mean, counts, ws = out
    lm.lmoe_router_losses(x["logits"], x["idx"], counts, mean, ls, ws, router_bias=x["bias"], row_mask=x["mask"],
                          stream=stream)
    return ls, mean, counts


def check_losses(x, got):
    ls, mean, counts = got
    want_l, want_m, want_c = tu.router_losses(x["logits"], x["idx"], x["bias"], x["mask"])
    assert torch.equal(counts.long(), want_c)
    l = x["logits"].double() + (0 if x["bias"] is None else x["bias"].double())
    l = l[tu.live_rows(l, x["mask"])]
    top = float(torch.where(torch.isfinite(l), l, 0.0).abs().max()) if l.numel() else 0.0
    rel = U * (6 * top + (2 * top if x["bias"] is not None else 0) + 45 + 256)
    assert_close(mean, want_m, want_m * rel + 1e-37, "mean probabilities")
    lse = float(torch.logsumexp(l, 1).abs().max()) if l.numel() else 0.0
    tol = torch.stack([want_l[0] * (rel + 64 * U),
                       2 * lse * U * ((7 if x["bias"] is not None else 5) * top + 80) + 300 * U * want_l[1]])
    assert_close(ls, want_l, tol + 1e-37, "losses")


def grad_inputs(x, weights=True, terms=True):
    T, k = x["idx"].shape
    E = x["logits"].shape[1]
    gw = torch.randn(T, k, generator=x["gen"], device="cuda") if weights else None
    gl = torch.tensor([0.3, -0.7], device="cuda") if terms else None
    counts = tu.router_losses(x["logits"], x["idx"], x["bias"], x["mask"])[2].int() if terms else None
    return gw, gl, counts


def check_grad(lm, x, weights=True, terms=True, in_place=False, ldo_pad=0):
    gw, gl, counts = grad_inputs(x, weights, terms)
    logits, (T, E) = x["logits"], x["logits"].shape
    d, tol = tu.router_grad(logits, x["idx"], counts, gw, gl, x["bias"], x["mask"])
    buf = torch.full((T, E + ldo_pad), 77.0, device="cuda", dtype=logits.dtype)
    out = logits if in_place else buf[:, :E]
    lm.lmoe_router_grad(logits, x["idx"], counts, out, gw, gl, x["bias"], x["mask"])
    if logits.dtype == torch.bfloat16:
        tol = tol + (d.abs() + tol) * 2.0 ** -8
    assert_close(out, d, tol, "gradient")
    dead = ~tu.live_rows(logits if not in_place else out, x["mask"]) if x["mask"] is not None else None
    if dead is not None:
        assert bool((out[~x["mask"].bool()] == 0).all())
    if ldo_pad:
        assert bool((buf[:, E:] == 77.0).all())   # between the rows: untouched


# one row, one expert; each layout of lanes and values at its ends; odd lengths (element loads)
SIZES = [(1, 1, 1), (1, 2, 2), (5, 3, 2), (33, 16, 4), (70, 17, 3), (100, 64, 8), (129, 65, 16), (257, 128, 8),
         (1000, 130, 7), (513, 256, 8), (300, 257, 16), (65, 512, 2), (40, 516, 5), (200, 1023, 16), (67, 1024, 1),
         (4999, 24, 4), (9000, 256, 8), (2500, 1000, 4)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_losses(lm, T, E, k, dtype):
    for x in (made(T, E, k, dtype), made(T, E, k, dtype, seed=1, masked=0.3, bias=True)):
        check_losses(x, losses(lm, x))


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_gradient(lm, T, E, k, dtype):
    check_grad(lm, made(T, E, k, dtype))
    check_grad(lm, made(T, E, k, dtype, seed=1, masked=0.3, bias=True), ldo_pad=3)


@pytest.mark.parametrize("weights,terms", [(True, False), (False, True)])
@pytest.mark.parametrize("T,E,k", [(7, 4, 2), (300, 100, 8), (50, 256, 8), (33, 900, 16)])
def test_gradient_of_one_kind(lm, T, E, k, weights, terms):
    check_grad(lm, made(T, E, k, masked=0.2), weights, terms)


@pytest.mark.parametrize("T,E,k,pad,base", [(60, 64, 4, 0, 1), (60, 64, 4, 4, 0), (60, 64, 4, 3, 2), (31, 200, 8, 24, 0),
                                            (90, 250, 8, 6, 0), (20, 1024, 16, 1, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_strided_and_unaligned_rows(lm, T, E, k, pad, base, dtype):
    x = made(T, E, k, dtype, pad=pad, base=base, masked=0.1)
    check_losses(x, losses(lm, x))
    check_grad(lm, x, ldo_pad=pad)
    check_grad(lm, x, in_place=True)


@pytest.mark.parametrize("E", [12, 64, 256, 700])
def test_in_place(lm, E):
    for dtype in (torch.float32, torch.bfloat16):
        check_grad(lm, made(333, E, 5, dtype, masked=0.25), in_place=True)


@pytest.mark.parametrize("E,k", [(8, 3), (100, 6), (256, 8), (600, 16)])
def test_masked_rows_may_hold_anything(lm, E, k):
    x = made(200, E, k, masked=0.4)
    off = ~x["mask"].bool()
    x["logits"][off] = float("nan")
    x["idx"][off] = 123456789
    some = off.nonzero()[:, 0]
    x["logits"][some[0]] = float("inf")
    x["logits"][some[1]] = torch.finfo(torch.float32).max
    x["idx"][some[1]] = -5
    check_losses(x, losses(lm, x))
    gw, gl, counts = grad_inputs(x)
    gw[off] = float("nan")
    d, tol = tu.router_grad(x["logits"], x["idx"], counts, gw, gl, None, x["mask"])
    out = torch.full_like(x["logits"], 5.0)
    lm.lmoe_router_grad(x["logits"], x["idx"], counts, out, gw, gl, None, x["mask"])
    assert_close(out, d, tol)


@pytest.mark.parametrize("E,k", [(5, 2), (64, 4), (256, 8), (900, 3)])
def test_experts_masked_by_infinity_and_rows_left_empty(lm, E, k):
    x = made(150, E, k)
    hide = torch.rand(150, E, generator=x["gen"], device="cuda") < 0.5
    x["logits"].masked_fill_(hide, -float("inf"))
    x["logits"][::7] = -float("inf")             # nothing left of these rows: not live
    x["logits"][3, :] = -float("inf")
    x["logits"][3, E - 1] = 1.5                  # one expert left
    x["idx"] = x["logits"].topk(k, 1).indices.int()   # names some of the hidden experts too
    check_losses(x, losses(lm, x))
    check_grad(lm, x)


@pytest.mark.parametrize("E", [10, 40, 200, 800])
def test_lowest_values_as_a_mask(lm, E):
    # masked experts hold the type's lowest value; one live row holds nothing else: its probabilities are
    # even, its lse^2 is past fp32's range
    for dtype in (torch.float32, torch.bfloat16):
        x = made(64, E, 4, dtype)
        low = torch.finfo(dtype).min
        x["logits"][:, ::3] = low
        x["idx"] = x["logits"].float().topk(4, 1).indices.int()
        tol = U * (6 * 12 + 45 + 256)   # (the unmasked logits stay below 12)
        want_l, want_m, want_c = tu.router_losses(x["logits"], x["idx"])
        ls, mean, counts = losses(lm, x)
        assert torch.equal(counts.long(), want_c) and torch.isfinite(ls).all()
        assert_close(mean, want_m, want_m * tol + 1e-37)
        x["logits"][5, :] = low
        want_l, want_m, want_c = tu.router_losses(x["logits"], x["idx"])
        ls, mean, counts = losses(lm, x)
        assert_close(mean, want_m, want_m * tol + 1e-37)
        assert_close(ls[:1], want_l[:1], want_l[:1] * (tol + 64 * U))
        assert float(ls[1]) == float("inf")
        gw, gl, c = grad_inputs(x)
        gl[1] = 0
        out = torch.empty_like(x["logits"])
        lm.lmoe_router_grad(x["logits"], x["idx"], c, out, gw, gl)
        d = tu.router_grad(x["logits"], x["idx"], c, gw, gl)[0]
        size = gw.double().abs().sum(1, keepdim=True) + 0.3 * E / 64 * 2
        assert_close(out, d, size * U * (12 * 12 + 4 * 12 + 160) + d.abs() * tu.HALF[dtype])


def test_large_logits(lm):
    y = made(80, 100, 8, spread=1.0)
    y["logits"] += 60.0
    check_losses(y, losses(lm, y))
    check_grad(lm, y)


def test_empty_slots_and_an_expert_named_twice(lm):
    for E in (6, 30, 100, 256, 500, 1000):
        x = made(120, E, 6)
        r = torch.randint(0, 6, (120, 6), generator=x["gen"], device="cuda")
        x["idx"] = x["idx"].gather(1, r)                       # repeats
        x["idx"][::5, 2] = -1
        x["idx"][::4, 0] = E                                   # outside: empty
        x["idx"][1::9] = -1                                    # every slot empty
        x["idx"] = x["idx"].contiguous()
        check_losses(x, losses(lm, x))
        check_grad(lm, x)
        gw, gl, counts = grad_inputs(x)
        gw[(x["idx"] < 0) | (x["idx"] >= E)] = float("nan")    # what an empty slot gets is not used
        d, tol = tu.router_grad(x["logits"], x["idx"], counts, gw, gl)
        out = torch.empty_like(x["logits"])
        lm.lmoe_router_grad(x["logits"], x["idx"], counts, out, gw, gl)
        assert_close(out, d, tol)


@pytest.mark.parametrize("E", [4, 256, 1024])
def test_no_rows_and_no_live_rows(lm, E):
    x = made(0, E, 2)
    for t in losses(lm, x):
        assert bool((t == 0).all())
    lm.lmoe_router_grad(x["logits"], x["idx"], None, x["logits"], torch.zeros(0, 2, device="cuda"))
    x = made(700, E, 2)
    x["mask"] = torch.zeros(700, dtype=torch.bool, device="cuda")   # bool as well as bytes
    for t in losses(lm, x):
        assert bool((t == 0).all())
    check_grad(lm, x)


def test_one_live_row_in_many(lm):
    x = made(16384, 64, 2)
    x["mask"] = torch.zeros(16384, dtype=torch.uint8, device="cuda")
    x["mask"][16383] = 200   # any byte but 0
    check_losses(x, losses(lm, x))
    check_grad(lm, x)


def test_uniform_routing_has_balance_one(lm):
    T, E = 4096, 16
    x = dict(logits=torch.zeros(T, E, device="cuda"), bias=None, mask=None,
             idx=(torch.arange(T, device="cuda")[:, None] * 2 + torch.arange(2, device="cuda")).remainder(E).int())
    ls, mean, counts = losses(lm, x)
    assert bool((counts[:E] == T * 2 // E).all())
    assert abs(float(ls[0]) - 1) <= 64 * U and abs(float(ls[1]) - float(torch.tensor(16.0).log() ** 2)) <= 400 * U * 8


@pytest.mark.parametrize("T,E,k", [(9, 6, 2), (40, 20, 3), (24, 130, 8)])
def test_gradient_against_differences(lm, T, E, k):
    # central differences of the objective in float64: off by h^2 / 6 times a third derivative below
    # 16 (|gw| + |gb| E + |gz| (|lse| + 3)) here, and by the objective's rounding over h
    x = made(T, E, k, masked=0.2, bias=True, spread=1.0)
    gw, gl, counts = grad_inputs(x)
    out = torch.empty_like(x["logits"])
    lm.lmoe_router_grad(x["logits"], x["idx"], counts, out, gw, gl, x["bias"], x["mask"])
    h = 1e-4
    slack = h * h / 6 * 16 * (float(gw.abs().max()) + 0.3 * E + 0.7 * 12) + 1e-9
    tol = tu.router_grad(x["logits"], x["idx"], counts, gw, gl, x["bias"], x["mask"])[1]
    pick = torch.randperm(T * E, generator=torch.Generator().manual_seed(1))[:60].tolist()
    for i in pick:
        t, e = divmod(i, E)
        f = []
        for s in (h, -h):
            y = x["logits"].double().clone()
            y[t, e] += s
            f.append(tu.router_objective(y, x["idx"], counts, gw, gl, x["bias"], x["mask"]))
        diff = float((f[0] - f[1]) / (2 * h))
        assert abs(float(out[t, e]) - diff) <= float(tol[t, e]) + slack, (t, e)


def test_bias_gradient_is_the_sum_over_rows(lm):
    x = made(50, 24, 3, bias=True, spread=1.0)
    gw, gl, counts = grad_inputs(x)
    out = torch.empty_like(x["logits"])
    lm.lmoe_router_grad(x["logits"], x["idx"], counts, out, gw, gl, x["bias"])
    b = x["bias"].double().requires_grad_()
    tu.router_objective(x["logits"], x["idx"], counts, gw, gl, b).backward()
    tol = tu.router_grad(x["logits"], x["idx"], counts, gw, gl, x["bias"])[1].sum(0)
    assert_close(out.double().sum(0), b.grad, tol + 1e-12)


def test_same_bits_every_time_and_on_another_stream(lm):
    x = made(5000, 200, 8, masked=0.1)
    gw, gl, counts = grad_inputs(x)
    first = [t.clone() for t in losses(lm, x)]
    d0 = torch.empty_like(x["logits"])
    lm.lmoe_router_grad(x["logits"], x["idx"], counts, d0, gw, gl, None, x["mask"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for i in range(3):
        d1 = torch.empty_like(x["logits"])
        out = None
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = losses(lm, x, out)
            lm.lmoe_router_grad(x["logits"], x["idx"], counts, d1, gw, gl, None, x["mask"])
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again)) and torch.equal(d0, d1)


def test_captured_and_replayed_with_a_shared_workspace(lm):
    # two captured graphs and eager calls share one workspace, one after another
    shapes = [(4000, 128, 4), (9000, 128, 2)]
    n = max(lm.lmoe_router_losses_workspace_size(T, E) for T, E, _ in shapes)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    runs = []
    for T, E, k in shapes:
        x = made(T, E, k)
        gw, gl, _ = grad_inputs(x)
        out = (torch.empty(2, device="cuda"), torch.empty(E, device="cuda"),
               torch.empty(E + 1, dtype=torch.int32, device="cuda"), ws)
        d = torch.empty_like(x["logits"])

        def step(x=x, out=out, d=d, gw=gw, gl=gl):
            losses(lm, x, out)
            lm.lmoe_router_grad(x["logits"], x["idx"], out[2], d, gw, gl)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        runs.append((x, out, d, step, graph))
    for again in range(2):
        for x, out, d, step, graph in runs:
            x["logits"].mul_(0.5)
            step()
            want = [t.clone() for t in (*out[:3], d)]
            for t in (*out[:3], d):
                t.fill_(3)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(want, (*out[:3], d)))
            check_losses(x, out[:3])


@pytest.mark.parametrize("T,shape", [(1, "nvfp4"), (1, "bf16"), (37, "bf16"), (300, "bf16")])
def test_block_methods(lm, T, shape):
    """The losses and the gradient from what a forward call left in the workspace."""
    import workloads
    from gpu_util import run, views
    E, k = 24, 3
    w = workloads.Workload(f"rt{T}{shape}", T=T, D=256, L=256, E=E, I=256, k=k, weights=shape, routing="zipf")
    inp = workloads.make_inputs(w, torch.device("cuda:0"))
    out, idx, blk, cfg = run(inp)
    bias = inp.router_bias
    v = views(blk, cfg)
    x = dict(logits=torch.tensor(v["logits"], device="cuda").float(), idx=idx, bias=bias, mask=None)
    got = blk.router_losses(cfg, router_bias=bias)
    check_losses(x, got)
    gw = torch.randn(T, k, generator=gen(T), device="cuda")
    gl = torch.tensor([0.01, 0.001], device="cuda")
    d, tol = tu.router_grad(x["logits"], idx, got[2], gw, gl, bias)
    assert_close(blk.router_grad(cfg, gw, gl, got[2], bias), d, tol)
    # the weights whose gradient it takes are the block's routing weights
    wts = tu.router_weights(x["logits"].double() + (0 if bias is None else bias.double()), idx)[0]
    assert_close(torch.tensor(v["topk_w"], device="cuda"), wts, wts * 1e-5 + 1e-7)
    torch.cuda.synchronize()
    with pytest.raises(ValueError):
        blk.router_losses(blk.config(1 << 14))
    empty = blk.router_losses(blk.config(0))
    assert all(bool((t == 0).all()) for t in empty)


def test_block_workspace_outlives_a_captured_call(lm):
    # a call captured at a small T replays after one at a large T, whose losses need more workspace
    import workloads
    from gpu_util import run
    w = workloads.Workload("rtcap", T=3000, D=256, L=128, E=24, I=128, k=3)
    inp = workloads.make_inputs(w, torch.device("cuda:0"))
    _, _, blk, big = run(inp)                       # (the block's own workspace has its full size from here on)
    small = blk.config(40, "bf16" if inp.x.dtype == torch.bfloat16 else "f32")
    x = inp.x[:40].contiguous()
    blk.forward(x)
    want = [t.clone() for t in blk.router_losses(small)]
    ws = blk._loss_ws.data_ptr()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = blk.router_losses(small)
    blk.forward(inp.x)
    blk.router_losses(big)
    assert blk._loss_ws.data_ptr() == ws and blk._loss_ws.numel() >= lm.lmoe_router_losses_workspace_size(1 << 20, 24)
    blk.forward(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals_on_the_device(lm):
    x = made(8, 16, 2)
    dev = dict(device="cuda")
    c, m, ls = torch.zeros(17, dtype=torch.int32, **dev), torch.zeros(16, **dev), torch.zeros(2, **dev)
    ws = torch.zeros(1 << 12, dtype=torch.uint8, **dev)
    R, G = lm.lmoe_router_losses, lm.lmoe_router_grad
    for match, fn in [
            ("topk_idx: dtype", lambda: R(x["logits"], x["idx"].long(), c, m, ls, ws)),
            ("topk_idx: shape", lambda: R(x["logits"], x["idx"][:7], c, m, ls, ws)),
            ("topk_idx must be contiguous", lambda: R(x["logits"], x["idx"].t().contiguous().t(), c, m, ls, ws)),
            ("counts: shape", lambda: R(x["logits"], x["idx"], c[:16], m, ls, ws)),
            ("mean_probs: shape", lambda: R(x["logits"], x["idx"], c, m[:15], ls, ws)),
            ("losses: shape", lambda: R(x["logits"], x["idx"], c, m, ls[:1], ws)),
            ("router_bias: shape", lambda: R(x["logits"], x["idx"], c, m, ls, ws, router_bias=m[:3])),
            ("row_mask: dtype", lambda: R(x["logits"], x["idx"], c, m, ls, ws, row_mask=torch.ones(8, **dev))),
            ("rows must be contiguous", lambda: R(x["logits"].t().contiguous().t(), x["idx"], c, m, ls, ws)),
            ("rows overlap", lambda: R(x["logits"][:1].expand(8, 16), x["idx"], c, m, ls, ws)),
            ("counts must be a CUDA tensor", lambda: R(x["logits"], x["idx"], c.cpu(), m, ls, ws)),
            ("workspace", lambda: R(x["logits"], x["idx"], c, m, ls, ws.cpu())),
            ("dlogits: dtype", lambda: G(x["logits"], x["idx"], c, x["logits"].bfloat16(), torch.zeros(8, 2, **dev))),
            ("topk_w_grad: shape", lambda: G(x["logits"], x["idx"], c, x["logits"], torch.zeros(8, 3, **dev))),
            ("loss_grads: shape", lambda: G(x["logits"], x["idx"], c, x["logits"], None, torch.zeros(3, **dev)))]:
        with pytest.raises(ValueError, match=match):
            fn()
    for fn in (lambda: R(x["logits"], x["idx"], c, m, ls, ws[:8]), lambda: G(x["logits"], x["idx"], c, x["logits"]),
               lambda: G(x["logits"], x["idx"], None, x["logits"], None, torch.zeros(2, **dev))):
        with pytest.raises(lm.LmoeError):
            fn()
