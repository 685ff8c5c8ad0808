"""Sizes beyond 32 bits, which the library does not take: refused, not cut to what is left of them (no GPU: tensors without memory,
and a library that is not reached)."""
import pytest
import torch

BIG = 2 ** 32 + 8
BF, F32, F8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


@pytest.fixture
def lm(monkeypatch):
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    from latent_mixture_experts_router_gb300 import _lib

    def reached(*args):
        raise AssertionError(f"{args[1]} was called")
    monkeypatch.setattr(_lib, "_want", lambda *a, **k: None)
    monkeypatch.setattr(_lib, "_bf16_at", lambda *a: 1 << 20)
    monkeypatch.setattr(_lib, "_call", reached)
    return lm


def z(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="meta")


def calls(lm):
    s = z(1, 1, dtype=F32)
    yield "ffn-N", lambda: lm.lmoe_gated_ffn(z(4, 8), z(BIG, 8), z(BIG, 8), z(4, BIG))
    yield "ffn-K", lambda: lm.lmoe_gated_ffn(z(4, BIG), z(8, BIG), z(8, BIG), z(4, 8))
    yield "ffn-E", lambda: lm.lmoe_gated_ffn(z(4, 8), z(BIG, 8, 8), z(BIG, 8, 8), z(4, 8))
    yield "ffn_grad-N", lambda: lm.lmoe_gated_ffn_grad(z(4, 8), z(8, BIG), *[z(4, BIG)] * 4)
    yield "matmul-N", lambda: lm.lmoe_matmul_bf16(z(4, 8), z(BIG, 8), z(4, BIG))
    yield "matmul-K", lambda: lm.lmoe_matmul_bf16(z(4, BIG), z(BIG, 8), z(4, 8), transposed=True)
    yield "wgrad-N", lambda: lm.lmoe_matmul_bf16_wgrad(z(4, BIG), z(4, 8), z(BIG, 8))
    yield "wgrad-K", lambda: lm.lmoe_matmul_bf16_wgrad(z(4, 8), z(4, BIG), z(8, BIG))
    yield "fp8-N", lambda: lm.lmoe_matmul_fp8(z(4, 128, dtype=F8), s, z(BIG, 128, dtype=F8), s, z(4, BIG))
    yield "fp8-K", lambda: lm.lmoe_matmul_fp8(z(4, BIG, dtype=F8), s, z(8, BIG, dtype=F8), s, z(4, 8))
    yield "fp8_wgrad-N", lambda: lm.lmoe_matmul_fp8_wgrad(z(BIG, 128, dtype=F8), s, z(8, 128, dtype=F8), s, z(BIG, 8))
    yield "fp8_rows-K", lambda: lm.lmoe_quantize_fp8_rows(z(4, BIG), z(4, BIG, dtype=F8), s)
    yield "fp8_weight-N", lambda: lm.lmoe_quantize_fp8_weight(z(BIG, 128), z(BIG, 128, dtype=F8), s)
    yield "fp8_weight-E", lambda: lm.lmoe_quantize_fp8_weight(z(BIG, 8, 8), z(BIG, 8, 8, dtype=F8), s)
    yield "fp8_cols-K", lambda: lm.lmoe_quantize_fp8_cols(z(4, BIG), z(BIG, 128, dtype=F8), s)
    yield "fp8_padded_rows", lambda: lm.lmoe_fp8_padded_rows(128, BIG)
    logits, idx = z(BIG, 8), z(BIG, 2, dtype=I32)
    yield "losses-T", lambda: lm.lmoe_router_losses(logits, idx, z(9, dtype=I32), s, s, s)
    yield "router_grad-T", lambda: lm.lmoe_router_grad(logits, idx, None, logits)
    yield "losses_workspace", lambda: lm.lmoe_router_losses_workspace_size(BIG, 8)
    yield "permute-T", lambda: lm.lmoe_permute_noalloc(idx, 8, s, s, s)
    yield "grad_norm_workspace", lambda: lm.lmoe_grad_norm_workspace_size(BIG)
    yield "nvfp4-K", lambda: lm.lmoe_quantize_nvfp4(z(1, BIG, dtype=F32), s, s)


@pytest.mark.parametrize("i", range(22))
def test_a_size_beyond_32_bits_is_refused(lm, i):
    cases = list(calls(lm))
    assert len(cases) == 22
    with pytest.raises(ValueError, match="beyond 32 bits"):
        cases[i][1]()
