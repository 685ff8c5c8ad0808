"""The weight gradient reads no block that the column quantiser left unwritten, whatever the offsets say."""
import ctypes

import pytest
import torch

import train_util as tu
from train_util import E4M3, E5M2, assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    return lm


TABLES = [(200, [0, 90, 2 ** 31 - 1]), (200, [-50, 60, 200]), (200, [150, 20, 200]), (200, [200, 200, 200]),
          (300, [0, 500, 600]), (1, [0, 1, 128, 300]), (127, [0, 400, 400]), (500, [-2 ** 31, 2 ** 31 - 1, 7, 501]),
          (129, [129, 129, 130, 385]), (640, [0, 128, 300, 640])]


@pytest.mark.parametrize("R,offs", TABLES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_blocks_never_written_are_never_read(lm, R, offs, accumulate):
    N, K, E = 144, 80, len(offs) - 1
    g = torch.Generator(device="cuda").manual_seed(R)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    P = lm.lmoe_fp8_padded_rows(R, E)

    def cols(width, fmt):   # NaN wherever the quantiser does not write
        src = torch.randn(R, width, generator=g, device="cuda")
        q = torch.full((width, P), 0x7f, dtype=torch.uint8, device="cuda").view(fmt)
        s = torch.full((P // 128, width), float("nan"), device="cuda")
        lm.lmoe_quantize_fp8_cols(src, q, s, o)
        return q, s
    (dy, ds), (x, xs) = cols(N, E5M2), cols(K, E4M3)
    dw = torch.full((E, N, K), 2.0, device="cuda")
    lm.lmoe_matmul_fp8_wgrad(dy, ds, x, xs, dw, offsets=o, accumulate=accumulate, rows=R)
    at = 0
    for e, (lo, hi) in enumerate(tu.groups(o, R)):
        n = min(-(-(hi - lo) // 128) * 128, P - at)   # (tables that go back may name more blocks than there are)
        b = slice(at // 128, (at + n) // 128)
        want, tol = tu.product(tu.values(dy[:, at:at + n], ds[b], False), tu.values(x[:, at:at + n], xs[b], False))
        want = want + (2.0 if accumulate else 0.0)
        assert_close(dw[e], want, tol + 2.0 ** -23 * (want.abs() + tol), f"expert {e}")
        at += n


def test_rows_are_checked(lm):
    dy, x = torch.zeros(64, 256, dtype=torch.uint8, device="cuda").view(E5M2), torch.zeros(48, 256, dtype=torch.uint8, device="cuda").view(E4M3)
    ds, xs, dw = torch.zeros(2, 64, device="cuda"), torch.zeros(2, 48, device="cuda"), torch.zeros(1, 64, 48, device="cuda")
    off = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    for rows in (129, 200, 256):
        lm.lmoe_matmul_fp8_wgrad(dy, ds, x, xs, dw, offsets=off, rows=rows)
    for rows in (128, 257, -1):      # padded, those are not 256
        with pytest.raises(lm.LmoeError):
            lm.lmoe_matmul_fp8_wgrad(dy, ds, x, xs, dw, offsets=off, rows=rows)
    with pytest.raises(ValueError, match="rows 0"):
        lm.lmoe_matmul_fp8_wgrad(dy, ds, x, xs, dw, offsets=off, rows=0)
    from latent_mixture_experts_router_gb300 import _lib
    shape = _lib.lmoe_fp8_matmul(128, 16, 128, 1, 0, 0, 0, 0, 0, 128)   # a product of rows has no padding
    p = dy.data_ptr()
    assert _lib._lib().lmoe_matmul_fp8(ctypes.byref(shape), p, p, p, p, None, p, None, None) == -1
