"""Host side of the router's training operators and of the 8-bit ones: sizes, and what they refuse before
any launch (no GPU: the C entries get made-up pointers that they never follow)."""
import ctypes
import os
import subprocess

import pytest
import torch

import train_util as tu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -4
P = 1 << 20   # never dereferenced


@pytest.fixture(scope="module")
def lm():
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    return lm


@pytest.fixture(scope="module")
def C(lm):
    return lm._lib._lib()   # with the argument types set


# ------------------------------------------------------------------ sizes
@pytest.mark.parametrize("E", [1, 3, 16, 17, 300, 1024])
def test_losses_workspace(lm, E):
    for T in (0, 1, 100, 5000, 1 << 20):
        n = lm.lmoe_router_losses_workspace_size(T, E)
        assert 0 < n <= 64 * (8 * E + 8)
    with pytest.raises(lm.LmoeError):
        lm.lmoe_router_losses_workspace_size(-1, E)
    with pytest.raises(lm.LmoeError):
        lm.lmoe_router_losses_workspace_size(1, 1025)


@pytest.mark.parametrize("rows,E", [(0, 4), (1, 1), (1, 7), (127, 1), (128, 1), (129, 1), (5, 9), (1000, 3), (257, 64)])
def test_padded_rows_hold_every_split(lm, rows, E):
    n = lm.lmoe_fp8_padded_rows(rows, E)
    assert n % 128 == 0
    # the worst split: as many experts as can be have one row more than whole blocks
    live = min(E, rows)
    need = 0
    if live:
        extra, rest = live, rows - live
        full = rest // 128
        need = (extra + full) * 128
        worst = max(need, -(-rows // 128) * 128)
        assert n >= worst
        assert n <= (rows + 127 * live) // 128 * 128
    else:
        assert n == 0
    assert lm.lmoe_fp8_padded_rows(-3, 4) == 0 and lm.lmoe_fp8_padded_rows(4, 0) == 0


def test_product_shape_matches_the_header(lm, tmp_path):
    import shutil
    from latent_mixture_experts_router_gb300._lib import lmoe_fp8_matmul as S
    cc, inc = shutil.which("gcc") or shutil.which("cc"), "/usr/local/cuda/include"
    if cc is None or not os.path.exists(os.path.join(inc, "cuda_runtime.h")):
        pytest.skip("no host compiler or CUDA headers")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "latent_moe.h"', "int main(void) {",
             '  printf("size %zu\\n", sizeof(lmoe_fp8_matmul));']
    lines += [f'  printf("{f} %zu\\n", offsetof(lmoe_fp8_matmul, {f}));' for f, _ in S._fields_]
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), "-I", inc, str(src), "-o", str(exe)], check=True)
    got = dict(ln.split() for ln in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(S)
    for f, _ in S._fields_:
        assert int(got[f]) == getattr(S, f).offset, f


# ------------------------------------------------------------------ the C entries
LOSSES = dict(logits=P, dt=0, ld=64, bias=None, mask=None, idx=P, T=8, E=64, k=2, counts=P, mean=P, losses=P, ws=P,
              n=1 << 20, stream=None)
GRAD = dict(logits=P, dt=0, ld=64, bias=None, mask=None, idx=P, gw=P, counts=P, gl=P, T=8, E=64, k=2, out=P, ldo=64,
            stream=None)
ROWS = dict(src=P, dt=0, ld=256, index=None, n=8, rows=8, K=256, fmt=0, pow2=0, codes=P, scales=P, stream=None)
WEIGHT = dict(src=P, dt=0, E=2, N=64, K=256, fmt=0, pow2=0, codes=P, scales=P, codes_t=P, scales_t=P, stream=None)
COLS = dict(src=P, dt=0, ld=256, index=None, n=8, rows=8, K=256, offsets=P, E=2, padded=256, fmt=0, pow2=0, codes=P,
            scales=P, stream=None)
MATMUL = dict(rows=8, N=64, K=256, E=2, af=0, bf=0, out=0, acc=0, a=P, a_s=P, w=P, w_s=P, offsets=P, y=P, status=None,
              stream=None)


def call(C, name, args, **change):
    v = dict(args, **change)
    if "af" in v:
        from latent_mixture_experts_router_gb300._lib import lmoe_fp8_matmul
        names = list(v)
        shape = lmoe_fp8_matmul(*[v[n] for n in names[:8]])
        return getattr(C, name)(ctypes.byref(shape), *[v[n] for n in names[8:]])
    return getattr(C, name)(*v.values())


BAD = [
    ("lmoe_router_losses", LOSSES, [
        (ARG, dict(T=-1)), (ARG, dict(T=(1 << 20) + 1)), (ARG, dict(E=0)), (ARG, dict(k=0)), (ARG, dict(k=17)),
        (ARG, dict(E=4, k=5)), (ARG, dict(ld=63)), (UNSUPPORTED, dict(E=1025, ld=1025)), (UNSUPPORTED, dict(dt=2)),
        (UNSUPPORTED, dict(dt=-1)), (ARG, dict(logits=None)), (ARG, dict(idx=None)), (ARG, dict(counts=None)),
        (ARG, dict(mean=None)), (ARG, dict(losses=None)), (ALIGN, dict(logits=P + 2)), (ALIGN, dict(dt=1, logits=P + 1)),
        (ALIGN, dict(bias=P + 2)), (ALIGN, dict(idx=P + 2)), (ALIGN, dict(counts=P + 1)), (ALIGN, dict(mean=P + 2)),
        (ALIGN, dict(losses=P + 2)), (ALIGN, dict(ws=P + 2)), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(n=16))]),
    ("lmoe_router_grad", GRAD, [
        (ARG, dict(T=-1)), (ARG, dict(E=0)), (ARG, dict(k=0)), (ARG, dict(k=17)), (ARG, dict(E=4, k=5)), (ARG, dict(ld=63)),
        (ARG, dict(ldo=63)), (UNSUPPORTED, dict(E=1025, ld=1025, ldo=1025)), (UNSUPPORTED, dict(dt=2)),
        (ARG, dict(logits=None)), (ARG, dict(out=None)), (ARG, dict(gw=None, gl=None)), (ARG, dict(counts=None)),
        (ARG, dict(idx=None)), (ARG, dict(ldo=128)), (ALIGN, dict(logits=P + 2)), (ALIGN, dict(out=P + 2)),
        (ALIGN, dict(gw=P + 2)), (ALIGN, dict(gl=P + 1)), (ALIGN, dict(counts=P + 2)), (ALIGN, dict(idx=P + 2))]),
    ("lmoe_quantize_fp8_rows", ROWS, [
        (ARG, dict(rows=-1)), (ARG, dict(n=-1)), (ARG, dict(K=0)), (ARG, dict(ld=255)), (ARG, dict(fmt=2)), (ARG, dict(n=7)),
        (ARG, dict(src=None)), (ARG, dict(codes=None)), (ARG, dict(scales=None)), (UNSUPPORTED, dict(dt=2)),
        (UNSUPPORTED, dict(K=248)), (UNSUPPORTED, dict(K=(1 << 20) + 16, ld=1 << 21)),
        (UNSUPPORTED, dict(rows=(1 << 24) + 1, index=P)), (ALIGN, dict(src=P + 2)), (ALIGN, dict(codes=P + 8)),
        (ALIGN, dict(scales=P + 2)), (ALIGN, dict(index=P + 2))]),
    ("lmoe_quantize_fp8_weight", WEIGHT, [
        (ARG, dict(E=-1)), (ARG, dict(N=0)), (ARG, dict(K=0)), (ARG, dict(fmt=2)), (ARG, dict(scales_t=None)),
        (ARG, dict(codes_t=None)), (ARG, dict(src=None)), (ARG, dict(codes=None)), (ARG, dict(scales=None)),
        (UNSUPPORTED, dict(dt=2)), (UNSUPPORTED, dict(K=248)), (UNSUPPORTED, dict(N=72)),
        (UNSUPPORTED, dict(K=1 << 21)), (UNSUPPORTED, dict(N=1 << 21)), (UNSUPPORTED, dict(E=1 << 30, N=1024, K=1024)),
        (ALIGN, dict(src=P + 2)), (ALIGN, dict(codes=P + 4)), (ALIGN, dict(codes_t=P + 4)), (ALIGN, dict(scales=P + 2)),
        (ALIGN, dict(scales_t=P + 2))]),
    ("lmoe_quantize_fp8_cols", COLS, [
        (ARG, dict(rows=-1)), (ARG, dict(n=-1)), (ARG, dict(K=0)), (ARG, dict(ld=255)), (ARG, dict(fmt=2)), (ARG, dict(n=7)),
        (ARG, dict(E=0, padded=0)), (ARG, dict(offsets=None)), (ARG, dict(padded=128)), (ARG, dict(padded=384)),
        (ARG, dict(src=None)), (ARG, dict(codes=None)), (ARG, dict(scales=None)), (UNSUPPORTED, dict(dt=2)),
        (UNSUPPORTED, dict(K=248)), (UNSUPPORTED, dict(E=1025, padded=8 * 128)), (ALIGN, dict(src=P + 2)),
        (ALIGN, dict(codes=P + 8)), (ALIGN, dict(scales=P + 2)), (ALIGN, dict(index=P + 2)), (ALIGN, dict(offsets=P + 2))]),
    ("lmoe_matmul_fp8", MATMUL, [
        (ARG, dict(rows=-1)), (ARG, dict(N=0)), (ARG, dict(K=0)), (ARG, dict(E=0)), (ARG, dict(af=2)), (ARG, dict(bf=-1)),
        (ARG, dict(acc=1)), (ARG, dict(offsets=None)), (UNSUPPORTED, dict(out=2)), (UNSUPPORTED, dict(E=1025)),
        (UNSUPPORTED, dict(K=248)), (UNSUPPORTED, dict(K=1 << 21)), (UNSUPPORTED, dict(N=1 << 21)),
        (UNSUPPORTED, dict(rows=(1 << 24) + 1)), (UNSUPPORTED, dict(rows=1 << 24, N=1 << 20)), (ARG, dict(a=None)),
        (ARG, dict(a_s=None)), (ARG, dict(w=None)), (ARG, dict(w_s=None)), (ARG, dict(y=None)), (ALIGN, dict(a=P + 8)),
        (ALIGN, dict(w=P + 8)), (ALIGN, dict(a_s=P + 2)), (ALIGN, dict(w_s=P + 2)), (ALIGN, dict(offsets=P + 2)),
        (ALIGN, dict(y=P + 2)), (ALIGN, dict(out=1, y=P + 1)), (ALIGN, dict(status=P + 2))]),
    ("lmoe_matmul_fp8_wgrad", dict(MATMUL, rows=256), [
        (ARG, dict(rows=-128)), (ARG, dict(rows=100)), (ARG, dict(N=0)), (ARG, dict(K=0)), (ARG, dict(E=0)), (ARG, dict(af=2)),
        (ARG, dict(offsets=None)), (UNSUPPORTED, dict(out=2)), (UNSUPPORTED, dict(E=1025)),
        (UNSUPPORTED, dict(K=1 << 21)), (UNSUPPORTED, dict(N=1 << 21)), (UNSUPPORTED, dict(rows=(1 << 24) + 128)),
        (UNSUPPORTED, dict(N=1 << 20, K=1 << 20, E=1024)), (ARG, dict(a=None)), (ARG, dict(a_s=None)), (ARG, dict(w=None)),
        (ARG, dict(w_s=None)), (ARG, dict(y=None)), (ALIGN, dict(a=P + 8)), (ALIGN, dict(w=P + 8)), (ALIGN, dict(a_s=P + 2)),
        (ALIGN, dict(w_s=P + 2)), (ALIGN, dict(offsets=P + 2)), (ALIGN, dict(y=P + 2)), (ALIGN, dict(status=P + 2))]),
]


@pytest.mark.parametrize("name,args,status,change", [
    pytest.param(n, a, st, ch, id=f"{n[5:]}-{'-'.join(f'{x}={y}' for x, y in ch.items())}")
    for n, a, cases in BAD for st, ch in cases])
def test_refused_without_launching(lm, C, name, args, status, change):
    n0 = lm.lmoe_kernel_launches()
    assert call(C, name, args, **change) == status
    assert lm.lmoe_kernel_launches() == n0


@pytest.mark.parametrize("name,args", [("lmoe_router_grad", dict(GRAD, T=0)), ("lmoe_quantize_fp8_rows", dict(ROWS, rows=0)),
                                       ("lmoe_quantize_fp8_weight", dict(WEIGHT, E=0)),
                                       ("lmoe_quantize_fp8_cols", dict(COLS, rows=0, padded=0)),
                                       ("lmoe_matmul_fp8", dict(MATMUL, rows=0)),
                                       ("lmoe_matmul_fp8_wgrad", dict(MATMUL, rows=0, acc=1))])
def test_nothing_to_do_launches_nothing(lm, C, name, args):
    n0 = lm.lmoe_kernel_launches()
    assert call(C, name, args) == 0
    assert lm.lmoe_kernel_launches() == n0


def test_no_shape_is_refused(C):
    for name in ("lmoe_matmul_fp8", "lmoe_matmul_fp8_wgrad"):
        assert getattr(C, name)(None, P, P, P, P, P, P, None, None) == ARG
    assert C.lmoe_router_losses_workspace_size(8, 8, None) == ARG


# ------------------------------------------------------------------ the binding
def _refusals(lm):
    f32, i32, bf = torch.float32, torch.int32, torch.bfloat16

    def z(*shape, dtype=f32):
        return torch.zeros(*shape, dtype=dtype)
    l, idx, c, m, ls, ws = z(8, 64), z(8, 2, dtype=i32), z(65, dtype=i32), z(64), z(2), z(1 << 16, dtype=torch.uint8)
    R, G = lm.lmoe_router_losses, lm.lmoe_router_grad
    yield "logits: dtype", lambda: R(l.double(), idx, c, m, ls, ws)
    yield "logits .T, E.", lambda: R(l[0], idx, c, m, ls, ws)
    yield "logits must be a CUDA tensor", lambda: R(l, idx, c, m, ls, ws)
    yield "logits: dtype", lambda: G(l.half(), idx, c, l.half())
    yield "logits must be a CUDA tensor", lambda: G(l, idx, c, l)
    s, q, sc = z(8, 256), z(8, 256, dtype=tu.E4M3), z(2, 8)
    yield "src .rows, K.", lambda: lm.lmoe_quantize_fp8_rows(s[0], q, sc)
    yield "src: dtype", lambda: lm.lmoe_quantize_fp8_rows(s.double(), q, sc)
    yield "src must be a CUDA tensor", lambda: lm.lmoe_quantize_fp8_rows(s, q, sc)
    yield "src .N, K. or", lambda: lm.lmoe_quantize_fp8_weight(s[0], q, sc)
    yield "src must be a CUDA tensor", lambda: lm.lmoe_quantize_fp8_weight(s, q, z(1, 2))
    yield "src must be a CUDA tensor", lambda: lm.lmoe_quantize_fp8_cols(s, z(256, 128, dtype=tu.E4M3), z(1, 256))
    a, w = z(8, 256, dtype=tu.E4M3), z(2, 64, 256, dtype=tu.E4M3)
    yield "a .rows, K. and w", lambda: lm.lmoe_matmul_fp8(a, sc, w[0, 0], z(2, 1, 2), z(8, 64))
    yield "a: dtype", lambda: lm.lmoe_matmul_fp8(a.to(bf), sc, w, z(2, 1, 2), z(8, 64))
    yield "a must be a CUDA tensor", lambda: lm.lmoe_matmul_fp8(a, sc, w, z(2, 1, 2), z(8, 64))
    d = z(64, 256, dtype=tu.E5M2)
    yield "P must be a multiple", lambda: lm.lmoe_matmul_fp8_wgrad(d[:, :200], z(2, 64), d[:, :200], z(2, 64), z(64, 64))
    yield "dy_t .N, P.", lambda: lm.lmoe_matmul_fp8_wgrad(d[0], z(2, 64), d, z(2, 64), z(64, 64))
    yield "dy_t must be a CUDA tensor", lambda: lm.lmoe_matmul_fp8_wgrad(d, z(2, 64), d, z(2, 64), z(64, 64))


@pytest.mark.parametrize("i", range(17))
def test_binding_refuses_what_does_not_fit(lm, i):
    cases = list(_refusals(lm))
    assert len(cases) == 17
    match, fn = cases[i]
    with pytest.raises(ValueError, match=match):
        fn()


def test_block_methods_want_a_forward_call_first(lm):
    D, L, E, I = 256, 128, 8, 128
    z = torch.zeros
    blk = lm.LatentMoEBlock(z(E, D), z(L, D), z(L), z(E, I, L), z(E, I, L), z(E, L, I), z(E, L), z(D, L), z(D), z(D), 2)
    for fn in (blk.router_losses, blk.router_grad):
        with pytest.raises(ValueError, match="forward call"):
            fn(blk.config(4))
