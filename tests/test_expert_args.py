"""Host side of the bf16 experts' operators and of the gradients' norm: sizes, and what they refuse before any launch
(no GPU: the C entries get made-up pointers that they never follow)."""
import ctypes
import os
import subprocess

import pytest
import torch

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


def test_shape_matches_the_header(lm, tmp_path):
    import shutil
    from latent_mixture_experts_router_gb300._lib import lmoe_bf16_matmul as S
    cc, inc = shutil.which("gcc") or shutil.which("cc"), "/usr/local/cuda/include"
    if cc is None or not os.path.exists(os.path.join(inc, "cuda_runtime.h")):
        pytest.skip("no host compiler or CUDA headers")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "latent_moe.h"', "int main(void) {",
             '  printf("size %zu\\n", sizeof(lmoe_bf16_matmul));']
    lines += [f'  printf("{f} %zu\\n", offsetof(lmoe_bf16_matmul, {f}));' for f, _ in S._fields_]
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), "-I", inc, str(src), "-o", str(exe)], check=True)
    got = dict(ln.split() for ln in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(S)
    for f, _ in S._fields_:
        assert int(got[f]) == getattr(S, f).offset, f


# ------------------------------------------------------------------ the C entries
SHAPE = dict(rows=8, N=64, K=256, E=2, out=1, transposed=0, acc=0, budget=0)
FFN = dict(SHAPE, x=P, wg=P, wu=P, offsets=P, h=P, gate=P, up=P, status=None, stream=None)
FFN_GRAD = dict(SHAPE, dy=P, wd=P, gate=P, up=P, offsets=P, dgate=P, dup=P, status=None, stream=None)
MATMUL = dict(SHAPE, a=P, w=P, a2=P, w2=P, offsets=P, y=P, status=None, stream=None)
WGRAD = dict(SHAPE, dy=P, x=P, dy2=P, offsets=P, dw=P, dw2=P, status=None, stream=None)


def call(C, name, args, **change):
    from latent_mixture_experts_router_gb300._lib import lmoe_bf16_matmul
    v = dict(args, **change)
    names = list(v)
    shape = lmoe_bf16_matmul(*[v[n] for n in names[:8]])
    return getattr(C, name)(ctypes.byref(shape), *[v[n] for n in names[8:]])


COMMON = [(ARG, dict(rows=-1)), (ARG, dict(N=0)), (ARG, dict(K=0)), (ARG, dict(E=0)), (ARG, dict(budget=-1)),
          (ARG, dict(offsets=None)), (UNSUPPORTED, dict(out=2)), (UNSUPPORTED, dict(out=-1)), (UNSUPPORTED, dict(E=1025)),
          (UNSUPPORTED, dict(K=252)), (UNSUPPORTED, dict(N=60)), (UNSUPPORTED, dict(K=(1 << 20) + 8)),
          (UNSUPPORTED, dict(N=(1 << 20) + 8)), (UNSUPPORTED, dict(rows=(1 << 24) + 1)), (ALIGN, dict(offsets=P + 2)),
          (ALIGN, dict(status=P + 2))]


def pointers(*names):
    return [(ARG, {n: None}) for n in names] + [(ALIGN, {n: P + 8}) for n in names]


BAD = [
    ("lmoe_gated_ffn", FFN, COMMON + pointers("x", "wg", "wu", "h") + [
        (ARG, dict(transposed=1)), (ARG, dict(acc=1)), (UNSUPPORTED, dict(out=0)), (ARG, dict(gate=None)), (ARG, dict(up=None)),
        (ALIGN, dict(gate=P + 8)), (ALIGN, dict(up=P + 8)), (UNSUPPORTED, dict(rows=1 << 24, N=1 << 20, E=1024))]),
    ("lmoe_gated_ffn_grad", FFN_GRAD, COMMON + pointers("dy", "wd", "gate", "up", "dgate", "dup") + [
        (ARG, dict(transposed=1)), (ARG, dict(acc=1)), (UNSUPPORTED, dict(out=0))]),
    ("lmoe_matmul_bf16", MATMUL, COMMON + pointers("a", "w", "y") + [
        (ARG, dict(acc=1)), (ARG, dict(a2=None)), (ARG, dict(w2=None)), (ALIGN, dict(a2=P + 8)), (ALIGN, dict(w2=P + 8))]),
    ("lmoe_matmul_bf16_wgrad", WGRAD, COMMON + pointers("dy", "x", "dw") + [
        (ARG, dict(transposed=1)), (ARG, dict(dy2=None)), (ARG, dict(dw2=None)), (ALIGN, dict(dy2=P + 8)),
        (ALIGN, dict(dw2=P + 8)), (UNSUPPORTED, dict(N=1 << 20, K=1 << 20, E=1024))]),
]


@pytest.mark.parametrize("name,args,status,change", [
    pytest.param(n, a, st, ch, id=f"{n[5:]}-{'-'.join(f'{x}={y}' for x, y in ch.items())}")
    for n, a, cases in BAD for st, ch in cases])
def test_refused_without_launching(lm, C, name, args, status, change):
    n0 = lm.lmoe_kernel_launches()
    assert call(C, name, args, **change) == status
    assert lm.lmoe_kernel_launches() == n0


@pytest.mark.parametrize("name,args", [("lmoe_gated_ffn", FFN), ("lmoe_gated_ffn_grad", FFN_GRAD), ("lmoe_matmul_bf16", MATMUL),
                                       ("lmoe_matmul_bf16_wgrad", dict(WGRAD, acc=1))])
def test_no_rows_launch_nothing(lm, C, name, args):
    n0 = lm.lmoe_kernel_launches()
    assert call(C, name, args, rows=0) == 0
    assert lm.lmoe_kernel_launches() == n0


G = 1 << 30   # apart from one another: 8 rows of 256 are 4 KB, the weights 64 KB
FFN_APART = dict(FFN, x=P, wg=P + G, wu=P + 2 * G, offsets=P + 3 * G, h=P + 4 * G, gate=P + 5 * G, up=P + 6 * G)
GRAD_APART = dict(FFN_GRAD, dy=P, wd=P + G, gate=P + 2 * G, up=P + 3 * G, offsets=P + 4 * G, dgate=P + 5 * G, dup=P + 6 * G)
MATMUL_APART = dict(MATMUL, a=P, w=P + G, a2=P + 2 * G, w2=P + 3 * G, offsets=P + 4 * G, y=P + 5 * G)
WGRAD_APART = dict(WGRAD, dy=P, x=P + G, dy2=P + 2 * G, offsets=P + 3 * G, dw=P + 4 * G, dw2=P + 5 * G)
SHARED = [("lmoe_gated_ffn", FFN_APART, [("h", "x", 0), ("h", "wg", 65520), ("gate", "h", 0), ("up", "gate", 1008), ("up", "wu", 16),
                                         ("h", "offsets", 0)]),
          ("lmoe_gated_ffn_grad", GRAD_APART, [("dgate", "up", 0), ("dup", "gate", 0), ("dgate", "gate", 16), ("dup", "dgate", 0),
                                               ("dgate", "dy", 4080), ("dup", "wd", 0)]),
          ("lmoe_matmul_bf16", MATMUL_APART, [("y", "a", 0), ("y", "a2", 4080), ("y", "w", 0), ("y", "w2", 16)]),
          ("lmoe_matmul_bf16_wgrad", WGRAD_APART, [("dw", "dy", 0), ("dw2", "x", 0), ("dw2", "dw", 16), ("dw", "dy2", 0)])]


@pytest.mark.parametrize("name,args,result,other,at", [
    pytest.param(n, a, *c, id=f"{n[5:]}-{c[0]}-in-{c[1]}+{c[2]}") for n, a, cases in SHARED for c in cases])
def test_results_that_share_memory_are_refused(lm, C, name, args, result, other, at):
    n0 = lm.lmoe_kernel_launches()
    assert call(C, name, args, **{result: args[other] + at}) == ARG
    assert lm.lmoe_kernel_launches() == n0


def test_no_shape_is_refused(C):
    for name, args in (("lmoe_gated_ffn", FFN), ("lmoe_gated_ffn_grad", FFN_GRAD), ("lmoe_matmul_bf16", MATMUL),
                       ("lmoe_matmul_bf16_wgrad", WGRAD)):
        assert getattr(C, name)(None, *list(args.values())[8:]) == ARG


def lists(ptrs, sizes, kinds):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_longlong * n)(*sizes), (ctypes.c_int * n)(*kinds))


def grads(C, name, ptrs, sizes, kinds, out=None, count=None, norm=P, ws=P, nws=1 << 20, max_norm=1.0, drop=None):
    p, s, k = lists(ptrs, sizes, kinds)
    o = (ctypes.c_void_p * len(ptrs))(*(ptrs if out is None else out))
    a = {"p": p, "o": o, "s": s, "k": k}
    if drop:
        a[drop] = None
    n = len(ptrs) if count is None else count
    if name == "lmoe_grad_norm":
        return C.lmoe_grad_norm(a["p"], a["s"], a["k"], n, norm, ws, nws, None)
    if name == "lmoe_grad_clip":
        return C.lmoe_grad_clip(a["p"], a["o"], a["s"], a["k"], n, norm, max_norm, None)
    return C.lmoe_clip_grad_norm(a["p"], a["o"], a["s"], a["k"], n, norm, max_norm, ws, nws, None)


Q = P + 4096
ONE = ([P], [100], [0])
ALL, CLIPS, NORMS = ("lmoe_grad_norm", "lmoe_grad_clip", "lmoe_clip_grad_norm"), ("lmoe_grad_clip", "lmoe_clip_grad_norm"), \
    ("lmoe_grad_norm", "lmoe_clip_grad_norm")
GRADS_BAD = [
    (ALL, ARG, ONE, dict(count=-1)), (ALL, ARG, ([P], [-1], [0]), {}), (ALL, ARG, ([None], [1], [0]), {}),
    (ALL, UNSUPPORTED, ([P], [1], [2]), {}), (ALL, UNSUPPORTED, ([P], [1], [-1]), {}), (ALL, UNSUPPORTED, ONE, dict(count=(1 << 20) + 1)),
    (ALL, UNSUPPORTED, ([P], [(1 << 40) + 1], [0]), {}), (ALL, ALIGN, ([P + 2], [1], [0]), {}), (ALL, ALIGN, ([P + 1], [1], [1]), {}),
    (ALL, ARG, ONE, dict(norm=None)), (ALL, ALIGN, ONE, dict(norm=P + 2)), (ALL, ARG, ONE, dict(drop="p")),
    (ALL, ARG, ONE, dict(drop="s")), (ALL, ARG, ONE, dict(drop="k")), (CLIPS, ARG, ONE, dict(drop="o")),
    (CLIPS, ARG, ONE, dict(out=[None])), (CLIPS, ALIGN, ONE, dict(out=[Q + 2])), (CLIPS, ARG, ONE, dict(max_norm=-1.0)),
    (CLIPS, ARG, ONE, dict(max_norm=float("nan"))), (NORMS, WORKSPACE, ONE, dict(ws=None)), (NORMS, WORKSPACE, ONE, dict(nws=64)),
    (NORMS, ALIGN, ONE, dict(ws=P + 4)),
    # overlaps: twice the same, a part of another, an output in another's input, in its own a little further on
    (CLIPS, ARG, ([P, P], [100, 100], [0, 0]), {}), (CLIPS, ARG, ([P, P + 396], [100, 100], [0, 0]), {}),
    (CLIPS, ARG, ([P + 396, P], [100, 100], [0, 0]), {}), (CLIPS, ARG, ([P, Q], [100, 100], [0, 0]), dict(out=[Q, P])),
    (CLIPS, ARG, ONE, dict(out=[P + 4])), (CLIPS, ARG, ([P, Q], [100, 100], [0, 1]), dict(out=[P + 8192, P + 8192 + 396])),
    (CLIPS, ARG, ([P, P + 8], [1000, 1], [0, 0]), dict(out=[Q, P + 100])),
]


@pytest.mark.parametrize("name,change", [
    (n, c) for n in ALL for c in (dict(out=[Q], norm=Q + 396), dict(norm=P + 396), dict(out=[Q], ws=Q - 8), dict(ws=P + 392),
                                  dict(norm=Q + 4096, ws=Q), dict(norm=Q, ws=Q))
    if not (n == "lmoe_grad_clip" and "ws" in c) and not (n == "lmoe_grad_norm" and "out" in c)])
def test_norm_and_workspace_that_share_memory_are_refused(lm, C, name, change):
    far = dict(norm=P + (1 << 24), ws=P + (1 << 25))
    n0 = lm.lmoe_kernel_launches()
    assert grads(C, name, *ONE, **{**far, **change}) == ARG
    assert lm.lmoe_kernel_launches() == n0


@pytest.mark.parametrize("name,i", [(n, i) for i, c in enumerate(GRADS_BAD) for n in c[0]])
def test_gradients_refused_without_launching(lm, C, name, i):
    _, status, args, change = GRADS_BAD[i]
    n0 = lm.lmoe_kernel_launches()
    assert grads(C, name, *args, **change) == status
    assert lm.lmoe_kernel_launches() == n0


def test_norm_workspace(lm, C):
    for n in (0, 1, 64, 65, 1024, 1025, 1 << 20):
        assert 0 < lm.lmoe_grad_norm_workspace_size(n) <= 32768 + 16 * n
    for n in (-1, (1 << 20) + 1):
        with pytest.raises(lm.LmoeError):
            lm.lmoe_grad_norm_workspace_size(n)
    assert C.lmoe_grad_norm_workspace_size(1, None) == ARG


# ------------------------------------------------------------------ the binding
def _refusals(lm):
    bf, f32 = torch.bfloat16, torch.float32

    def z(*shape, dtype=bf):
        return torch.zeros(*shape, dtype=dtype)
    x, w, h = z(8, 64), z(2, 32, 64), z(8, 32)
    F, G, M, W = lm.lmoe_gated_ffn, lm.lmoe_gated_ffn_grad, lm.lmoe_matmul_bf16, lm.lmoe_matmul_bf16_wgrad
    yield "x .rows, K.", lambda: F(x[0], w, w, h)
    yield "w_gate .N, K.", lambda: F(x, w[0, 0], w, h)
    yield "x: dtype", lambda: F(x.float(), w, w, h)
    yield "x must be a CUDA tensor", lambda: F(x, w, w, h)
    yield "dy .rows, K.", lambda: G(x[0], w, h, h, h, h)
    yield "w_down .K, N.", lambda: G(x, x[0], h, h, h, h)
    yield "dy: dtype", lambda: G(x.half(), w, h, h, h, h)
    yield "dy must be a CUDA tensor", lambda: G(x, w.transpose(1, 2), h, h, h, h)
    yield "a .rows, K.", lambda: M(x[0], w, h)
    yield "w .N, K.", lambda: M(x, w[0, 0], h)
    yield "a: dtype", lambda: M(x.float(), w, h)
    yield "a must be a CUDA tensor", lambda: M(x, w, h)
    yield "dw .N, K.", lambda: W(h, x, x[0])
    yield "dy .rows, N.", lambda: W(h[0], x, w)
    yield "dy: dtype", lambda: W(h.float(), x, w)
    yield "dy must be a CUDA tensor", lambda: W(h, x, w)
    n, ws = z(1, dtype=f32), z(1 << 16, dtype=torch.uint8)
    yield "norm: dtype", lambda: lm.lmoe_grad_norm([x], z(1), ws)
    yield "norm: shape", lambda: lm.lmoe_grad_clip([x], z(2, dtype=f32), 1.0)
    yield "norm must be a CUDA tensor", lambda: lm.lmoe_clip_grad_norm([x], n, 1.0, ws)


@pytest.mark.parametrize("i", range(19))
def test_binding_refuses_what_does_not_fit(lm, i):
    cases = list(_refusals(lm))
    assert len(cases) == 19
    match, fn = cases[i]
    with pytest.raises(ValueError, match=match):
        fn()


def test_lists_of_gradients_that_do_not_fit(lm):
    from latent_mixture_experts_router_gb300._lib import _tensors
    t = torch.zeros(4)
    for grads, match in (([t], "g: all tensors must be on cuda:0"), ([t, 1], "g: all tensors must be on cuda:0"),
                         ([None, t], "g: element 0 is not a tensor"), (iter(["t"]), "g: element 0 is not a tensor")):
        with pytest.raises(ValueError, match=match):
            _tensors.gradients(grads, "g", 0)
    for grads in (None, 3):
        with pytest.raises(TypeError):
            _tensors.gradients(grads, "g", 0)

    def broken():
        yield t
        raise KeyError("its own")
    with pytest.raises(KeyError, match="its own"):
        _tensors.gradients(broken(), "g", 0)
    assert _tensors.gradients([], "g", 0) == (b"", b"", b"", 0)


def test_addresses_of_what_does_not_fit(lm):
    from latent_mixture_experts_router_gb300._lib import _tensors
    t = torch.zeros(2, 8, dtype=torch.bfloat16)
    for x in (t, None, 1, t.to_sparse(), torch.empty(2, 8, dtype=torch.bfloat16, device="meta")):
        assert _tensors.bf16_at(x, (2, 8), 0) == -1
    for args in ((t, [2, 8], 0), (t, (2, 8)), (t, (2, 8), "0")):
        with pytest.raises(TypeError):
            _tensors.bf16_at(*args)
