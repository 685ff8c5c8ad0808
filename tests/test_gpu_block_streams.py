"""LatentMoEBlock's methods on a stream that is not the current one: what they allocate belongs to that stream,
so that neither the current stream's pending work nor another stream's calls touch it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BUSY = 400_000_000   # cycles that the current stream sleeps: 0.2 s


@pytest.fixture(scope="module")
def setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    import workloads
    from gpu_util import make_block
    w = workloads.Workload("streams", T=3000, D=256, L=128, E=24, I=128, k=3)
    inp = workloads.make_inputs(w, torch.device("cuda:0"))
    return inp, make_block


def handles():
    s = torch.cuda.Stream()
    return [s, s.cuda_stream]   # a torch stream, a raw handle


def while_busy(shapes, call):
    """Runs ``call`` while the current stream sleeps and, behind that, has yet to read tensors of ``shapes`` that are
    freed already; returns (call's result, what it then read)."""
    torch.cuda.synchronize()
    held = [torch.full(s, 7.0, dtype=d, device="cuda") for s, d in shapes]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    read = [t + 0 for t in held]
    del held
    out = call()
    torch.cuda.synchronize()
    return out, read


@pytest.mark.parametrize("which", [0, 1])
def test_results_are_not_taken_from_the_current_stream(setup, which):
    inp, make_block = setup
    blk = make_block(inp)
    T, E, k = 3000, 24, 3
    cfg = blk.config(T)
    base = blk.forward(inp.x)
    want_l = [t.clone() for t in blk.router_losses(cfg)]
    gl = torch.tensor([0.01, 0.001], device="cuda")
    want_g = blk.router_grad(cfg, loss_grads=gl, counts=want_l[2]).clone()
    s = handles()[which]
    f32 = torch.float32

    def same(got, want, read):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(bool((t == 7).all()) for t in read)
    n = blk._loss_ws.numel()
    out, read = while_busy([((2,), f32), ((E,), f32), ((E + 1,), f32), ((n,), torch.uint8)] * 3, lambda: blk.router_losses(cfg, stream=s))
    same(out, want_l, read)
    out, read = while_busy([((T, E), f32)] * 3, lambda: blk.router_grad(cfg, loss_grads=gl, counts=want_l[2], stream=s))
    same([out], [want_g], read)
    out, read = while_busy([((T, 256), f32)] * 3, lambda: blk.forward(inp.x, stream=s))
    same([out], [base], read)
    # a first call: workspace and losses' workspace too
    fresh = make_block(inp)
    (out, losses), read = while_busy([((blk._ws.numel(),), torch.uint8)],
                                     lambda: (fresh.forward(inp.x, stream=s), fresh.router_losses(cfg, stream=s)))
    same([out, *losses], [base, *want_l], read)


def test_a_larger_workspace_on_another_stream(setup):
    # the first call's workspace is used by s and replaced on the current stream while s is still at work
    inp, make_block = setup
    x = inp.x[:500].contiguous()
    want = make_block(inp).forward(x).clone()
    torch.cuda.synchronize()
    for _ in range(3):
        blk = make_block(inp)
        s = torch.cuda.Stream()
        blk.workspace(blk.config(500))            # zeroed on the current stream,
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY // 4)
        out = blk.forward(x, stream=s)            # used on s, later,
        ws = blk._ws.data_ptr()
        blk.workspace(blk.config(3000))           # and replaced
        junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        assert blk._ws.data_ptr() != ws
        assert torch.equal(out, want)
        del junk


def test_workspace_zeroed_behind_pending_work(setup):
    # the current stream zeroes the workspace only after its sleep; the call on s waits for that
    inp, make_block = setup
    x = inp.x[:500].contiguous()
    want = make_block(inp).forward(x).clone()
    blk = make_block(inp)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY // 2)
    blk.workspace(blk.config(500))
    out = blk.forward(x, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_losses_on_two_streams_at_once(setup):
    inp, make_block = setup
    blk = make_block(inp)
    cfg = blk.config(3000)
    blk.forward(inp.x)
    masks = [(torch.arange(3000, device="cuda") % m != 0).to(torch.uint8) for m in (3, 7, 11)]
    want = [[t.clone() for t in blk.router_losses(cfg, row_mask=m)] for m in masks]
    streams = [torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[blk.router_losses(cfg, row_mask=m, stream=s) for m, s in zip(masks, streams)] for _ in range(40)]
    torch.cuda.synchronize()
    for one in got:
        for a, b in zip(one, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_captured_graphs_of_the_losses_at_once(setup):
    inp, make_block = setup
    blk = make_block(inp)
    cfg = blk.config(3000)
    blk.forward(inp.x)
    masks = [(torch.arange(3000, device="cuda") % m != 0).to(torch.uint8) for m in (3, 7)]
    want = [[t.clone() for t in blk.router_losses(cfg, row_mask=m)] for m in masks]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for m in masks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(blk.router_losses(cfg, row_mask=m))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(40):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_calls_survive_a_larger_workspace(setup):
    inp, make_block = setup
    x = inp.x[:40].contiguous()
    ref = make_block(inp)
    want = [ref.forward(x).clone(), *(t.clone() for t in ref.router_losses(ref.config(40)))]
    blk = make_block(inp)
    cfg = blk.config(40)
    blk.forward(x)
    blk.router_losses(cfg)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [blk.forward(x), *blk.router_losses(cfg)]
    small = blk._ws
    size, ptr = small.numel(), small.data_ptr()
    del small
    big = blk.forward(inp.x)                     # replaces the workspace
    big_l = [t.clone() for t in blk.router_losses(blk.config(3000))]
    assert blk._ws.data_ptr() != ptr
    junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]   # takes what was freed
    assert all(t.data_ptr() != ptr for t in junk)
    for t in got:
        t.fill_(3)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 255).all()) for t in junk)      # the replays wrote their own workspace only
    assert torch.equal(blk.forward(inp.x), big)
    assert all(torch.equal(a, b) for a, b in zip(blk.router_losses(blk.config(3000)), big_l))


def test_a_block_whose_first_call_is_captured(setup):
    # (other blocks have run these kernels before: a library call's first set-up is not part of the capture)
    inp, make_block = setup
    ref = make_block(inp)
    want = [ref.forward(inp.x).clone(), *(t.clone() for t in ref.router_losses(ref.config(3000)))]
    blk = make_block(inp)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [blk.forward(inp.x), *blk.router_losses(blk.config(3000))]
    eager = [blk.forward(inp.x), *blk.router_losses(blk.config(3000))]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(eager, want))
