"""Waits of pairs of CTAs that give up in the middle of long calls, at any of their places: the calls end, report it, and leave
nothing behind that the next ones would meet."""
import ctypes

import pytest
import torch

import expert_util as xu
from expert_util import BF16

pytestmark = pytest.mark.gpu
F32 = torch.float32
WAITS = 0x1 | 0x2 | 0x4 | 0x10


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    return lm


def ints(shape, seed):
    return torch.randint(-2, 3, shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)


@pytest.mark.parametrize("out", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("op", ["nt", "nn", "wgrad", "gated", "gated_grad"])
def test_pairs_that_give_up(lm, op, out):
    """Tiles of 256 blocks take some 100 us, three and more to a pair, so budgets below that run out in the epilogue, which then
    stops the MMAs and they the producers, each where it is."""
    from latent_mixture_experts_router_gb300 import _lib
    if out == F32 and op.startswith("gated"):
        pytest.skip("bf16 only")
    R, N, K = (16384, 4096, 4096) if op == "wgrad" else (3000, 6000, 16384)
    a = ints((R, K), 1)
    w = ints((R, N), 2) if op == "wgrad" else ints((K, N) if op in ("nn", "gated_grad") else (N, K), 2)
    y = [torch.full((N if op == "wgrad" else R, K if op == "wgrad" else N), 7.25, dtype=out, device="cuda") for _ in range(3)]
    g = ints((R, N), 3) if op == "gated_grad" else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(budget):
        shape = _lib.lmoe_bf16_matmul(R, N, K, 1, 0 if out == F32 else 1, 1 if op == "nn" else 0, 0, budget)
        name, args = {"wgrad": ("lmoe_matmul_bf16_wgrad", (w, a, None, None, y[0], None)),
                      "gated": ("lmoe_gated_ffn", (a, w, w, None, *y)),
                      "gated_grad": ("lmoe_gated_ffn_grad", (a, w, g, g, None, *y[:2]))}.get(
                          op, ("lmoe_matmul_bf16", (a, w, None, None, None, y[0])))
        st = getattr(_lib._lib(), name)(ctypes.byref(shape), *[t if t is None else t.data_ptr() for t in args], status.data_ptr(),
                                        torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0
        word = int(status) & 0xffffffff
        status.zero_()
        return word
    assert call(0) == 0
    want = [t.clone() for t in y]
    exact = xu.product(a[:64], w, None, op == "nn")[0] if op in ("nt", "nn") else \
        w[:, :64].double().t() @ a.double() if op == "wgrad" else None
    if exact is not None:
        assert torch.equal(want[0][:64], exact.float().to(out))
    gave_up = 0
    for budget in (1, 30000, 60000, 100000, 150000, 200000):
        word = call(budget)
        assert word & ~WAITS == 0
        gave_up += word != 0
        for t in y:
            t.fill_(7.25)
        assert call(0) == 0
        for t, v in zip(y, want):
            assert torch.equal(t, v)
    assert gave_up > 0 or out == F32   # (fp32 sums end every 12 blocks: no wait is as long)
    assert lm.lmoe_bf16_check_status() == (0, 0)
