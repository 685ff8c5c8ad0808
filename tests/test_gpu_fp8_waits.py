"""8-bit products whose device waits give up: the call ends, says so in its error word, writes nothing behind
its output, and the next call is right."""
import ctypes

import pytest
import torch

import train_util as tu
from train_util import E4M3, E5M2

pytestmark = pytest.mark.gpu
WAITS = 0x1 | 0x2 | 0x4 | 0x10   # the error word's bits of waits that gave up


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    return lm


def integers(shape, fmt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-4, 5, shape, generator=g, device="cuda").float().to(fmt)


def run(lm, name, dims, budget, accumulate, out, status, *args):
    from latent_mixture_experts_router_gb300 import _lib
    rows, N, K, E, af, bf = dims
    shape = _lib.lmoe_fp8_matmul(rows, N, K, E, af, bf, 0 if out.dtype == torch.float32 else 1, accumulate)
    shape.wait_budget_cycles = budget
    st = getattr(_lib._lib(), name)(ctypes.byref(shape), *[t.data_ptr() for t in args], out.data_ptr(), status.data_ptr(),
                                    torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    return int(status.item()) & 0xffffffff


@pytest.mark.parametrize("R,E,N,K", [(6, 1, 256, 256), (6, 1, 256, 2048), (100, 1, 640, 400), (100, 1, 640, 2048),
                                     (600, 1, 5000, 256), (40, 9, 520, 512), (3000, 6, 1000, 1024)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_matmul_waits_that_give_up(lm, R, E, N, K, out):
    a, w = integers((R, K), E4M3, 1), integers((E, N, K), E4M3, 2)
    kb, nb = -(-K // 128), -(-N // 128)
    a_s, w_s = torch.ones(kb, R, device="cuda"), torch.ones(E, nb, kb, device="cuda")
    off = (torch.arange(E + 1, device="cuda") * R // E).int()
    buf = torch.full((R + 8, N), 7.25, dtype=out, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda budget: run(lm, "lmoe_matmul_fp8", (R, N, K, E, 0, 0), budget, 0, buf, status, a, a_s, w, w_s, off)
    for _ in range(3):
        word = call(1)
        assert word & ~WAITS == 0
    assert bool((buf[R:] == 7.25).all())
    status.zero_()
    assert call(0) == 0
    want = torch.cat([a[off[e]:off[e + 1]].double() @ w[e].double().t() for e in range(E)])
    assert torch.equal(buf[:R], want.float().to(out))


@pytest.mark.parametrize("R,E,N,K", [(300, 1, 130, 260), (1000, 5, 264, 144), (60, 40, 144, 272), (128, 300, 64, 32)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_wgrad_waits_that_give_up(lm, R, E, N, K, out, accumulate):
    # some experts without rows: their tiles store nothing when the call adds
    P = lm.lmoe_fp8_padded_rows(R, E)
    cuts = torch.sort(torch.randint(0, R + 1, (E - 1,), generator=torch.Generator().manual_seed(E)))[0]
    off = torch.cat([torch.zeros(1), cuts, torch.full((1,), R)]).int().cuda()
    dy, x = integers((N, P), E5M2, 1), integers((K, P), E4M3, 2)
    ds, xs = torch.ones(P // 128, N, device="cuda"), torch.ones(P // 128, K, device="cuda")
    buf = torch.zeros(E * N * K + 64, dtype=out, device="cuda")
    buf[E * N * K:] = 7.25
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda budget: run(lm, "lmoe_matmul_fp8_wgrad", (P, N, K, E, 1, 0), budget, accumulate, buf, status, dy, ds, x, xs, off)
    for _ in range(3):
        word = call(1)
        assert word & ~WAITS == 0
    assert bool((buf[E * N * K:] == 7.25).all())
    status.zero_()
    buf[:E * N * K] = 0
    assert call(0) == 0
    at = 0
    for e, (lo, hi) in enumerate(tu.groups(off, R)):
        n = -(-(hi - lo) // 128) * 128
        want = dy[:, at:at + n].double() @ x[:, at:at + n].double().t()
        assert torch.equal(buf[:E * N * K].view(E, N, K)[e], want.float().to(out)), e
        at += n


def test_calls_without_a_status_word_report_too(lm):
    assert lm.lmoe_fp8_check_status()[0] in (0, -6)          # (whatever came before: cleared now)
    a, w = integers((300, 256), E4M3, 1), integers((5000, 256), E4M3, 2)
    one, y = torch.ones(2, 300, device="cuda"), torch.zeros(300, 5000, device="cuda")
    lm.lmoe_matmul_fp8(a, one, w, torch.ones(40, 2, device="cuda"), y)
    assert lm.lmoe_fp8_check_status() == (0, 0)
    s = torch.cuda.Stream()
    lm.lmoe_fp8_wait_selftest(100_000, stream=s)             # a wait that gives up
    st, word = lm.lmoe_fp8_check_status(stream=s)
    assert st == -6 and word & WAITS and word & ~WAITS == 0
    assert lm.lmoe_fp8_check_status() == (0, 0)              # read once
    # a product of its own, with a budget that cannot do: no status word of the caller's
    from latent_mixture_experts_router_gb300 import _lib
    shape = _lib.lmoe_fp8_matmul(300, 5000, 256, 1, 0, 0, 0, 0, 1)
    ws = torch.ones(40, 2, device="cuda")
    for _ in range(3):
        assert _lib._lib().lmoe_matmul_fp8(ctypes.byref(shape), a.data_ptr(), one.data_ptr(), w.data_ptr(), ws.data_ptr(), None,
                                           y.data_ptr(), None, torch.cuda.current_stream().cuda_stream) == 0
    assert lm.lmoe_fp8_check_status()[0] == -6
    lm.lmoe_matmul_fp8(a, one, w, ws, y)
    assert lm.lmoe_fp8_check_status() == (0, 0)
    assert torch.equal(y, (a.double() @ w.double().t()).float())


def test_budget_is_checked(lm):
    from latent_mixture_experts_router_gb300 import _lib
    t = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = t.data_ptr()
    for name in ("lmoe_matmul_fp8", "lmoe_matmul_fp8_wgrad"):
        shape = _lib.lmoe_fp8_matmul(128, 16, 128, 1, 0, 0, 0, 0, -1)
        assert getattr(_lib._lib(), name)(ctypes.byref(shape), p, p, p, p, None, p, None, None) == -1
