"""The operators that train and serve the experts in bf16, case by case: inputs, a plain form in
elementary torch operations, the library's calls, and the values in 64 bits.

op "ffn"    the gated feed-forward block: both projections, silu and the product (saved for the backward pass)
op "grad"   its gradient, together with the down projection's input gradient
op "matmul" product of rows with their expert's weights (down projection), or with the weights the
            other way round (input gradient), from one pair of operands or summed over two
op "wgrad"  weight gradient over each expert's rows, of one weight or of the two that share x
op "clip"   norm over all gradients and the gradients scaled down to a largest norm

Set ``own`` to run the library's calls instead of the plain forms.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a small model's micro-batch, values saved for the backward pass: the time of a call
        dict(name="ffn-R128-E16", op="ffn", R=128, E=16, N=512, K=256, save=True),
        # serving: one token on 8 of 64 experts, their weights streamed
        dict(name="ffn-T1-E64", op="ffn", R=8, E=64, N=4096, K=4096, save=False),
        # training: 4096 tokens on 8 of 64 experts each
        dict(name="ffn-R32768-E64", op="ffn", R=32768, E=64, N=4096, K=4096, save=True),
        # the backward pass of half as many experts and tokens
        dict(name="grad-R16384-E32", op="grad", R=16384, E=32, N=4096, K=4096),
        # a dense layer's, an odd number of rows
        dict(name="grad-dense-R1001", op="grad", R=1001, E=1, N=4096, K=8192),
        # down projection of a batch of 128 decoded tokens, to fp32
        dict(name="matmul-R1024-E64", op="matmul", R=1024, E=64, N=4096, K=4096, pairs=1, transposed=False, out="f32"),
        # a dense layer over an odd number of tokens
        dict(name="matmul-dense-R2047", op="matmul", R=2047, E=1, N=8192, K=4096, pairs=1, transposed=False, out="bf16"),
        # input gradient of gate and up together
        dict(name="matmul-dx-R16384-E32", op="matmul", R=16384, E=32, N=4096, K=4096, pairs=2, transposed=True,
             out="bf16"),
        # weight gradients of gate and up of 16 experts over 8192 routed rows, to fp32
        dict(name="wgrad-R8192-E16", op="wgrad", R=8192, E=16, N=4096, K=4096, pairs=2, out="f32"),
        # weight gradient of a dense layer over 1000 tokens
        dict(name="wgrad-dense-R1000", op="wgrad", R=1000, E=1, N=4096, K=8192, pairs=1, out="bf16"),
        # the gradients of a small model: many tensors of any size, packed without gaps
        dict(name="clip-200x4k", op="clip", tensors=200, n=819200, dtype="mixed", packed=True),
        # the gradients of 32 experts' weights in fp32
        dict(name="clip-96x16M", op="clip", tensors=96, n=805306368, dtype="f32", packed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "grad", "matmul", "wgrad", "clip", "ffn", "matmul"])
    if op == "clip":
        tensors = _log(rng, 1, 1500)
        return dict(op=op, tensors=tensors, n=max(tensors, _log(rng, 100, 800000000)),
                    dtype=rng.choice(["f32", "bf16", "mixed"]), packed=rng.random() < 0.5)
    K, N = 8 * _log(rng, 2, 1024), 8 * _log(rng, 2, 1024)
    E = max(1, min(_log(rng, 1, 256), 1073741824 // (N * K)))
    if op == "wgrad":
        E = max(1, min(E, 268435456 // (N * K)))
    R = max(1, min(_log(rng, 1, 32768), 549755813888 // (N * K)))
    if op == "ffn":
        return dict(op=op, R=R, E=E, N=N, K=K, save=rng.random() < 0.5)
    if op == "grad":
        return dict(op=op, R=R, E=E, N=N, K=K)
    pairs = rng.randint(1, 2)
    if op == "matmul":
        return dict(op=op, R=R, E=max(1, E // pairs), N=N, K=K, pairs=pairs, transposed=rng.random() < 0.5,
                    out=rng.choice(["bf16", "f32"]))
    return dict(op=op, R=R, E=E, N=N, K=K, pairs=pairs, out=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------ inputs
def _gen(seed, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + n)
    return g


def _normal(shape, seed, n, std=1.0):
    return torch.randn(shape, generator=_gen(seed, n), device="cuda").mul_(std).to(BF16)


def _weights(E, shape, seed, n, std):
    w = torch.empty(E, *shape, dtype=BF16, device="cuda")
    for e in range(E):
        w[e] = torch.randn(shape, generator=_gen(seed, n + e), device="cuda").mul_(std)
    return w


def _counts(R, E, seed):
    """Rows of each expert: uneven, some experts often without any."""
    w = torch.exp(0.7 * torch.randn(E, generator=_gen(seed, 90), device="cuda"))
    ids = torch.multinomial(w, R, replacement=True, generator=_gen(seed, 91))
    return torch.bincount(ids, minlength=E)


def _sizes(tensors, n):
    """Sizes of that many tensors, n elements in all, each at least 1: within a factor of ten or so."""
    g = torch.Generator()
    g.manual_seed(tensors)
    w = torch.exp(0.8 * torch.randn(tensors, generator=g, dtype=torch.float64))
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * (n - tensors)).long()
    return (torch.diff(cut, prepend=cut.new_zeros(1)) + 1).tolist()


def _gradients(st, seed):
    kinds = ["f32", "bf16"] if st["dtype"] == "mixed" and st["tensors"] > 1 else [st["dtype"].replace("mixed", "f32")]
    parts = [st["tensors"] // 2, st["tensors"] - st["tensors"] // 2] if len(kinds) > 1 else [st["tensors"]]
    st["flat"], st["out"], st["grads"], st["outs"] = [], [], [], []
    for i, (kind, tensors) in enumerate(zip(kinds, parts)):
        n = max(tensors, st["n"] // len(kinds))
        sizes = _sizes(tensors, n)
        # packed: one after the other, wherever that is; else each on 256 bytes, as an allocator gives them
        room = sizes if st["packed"] else [(s + 127) // 128 * 128 for s in sizes]
        flat = torch.zeros(sum(room), dtype=DTYPE[kind], device="cuda")
        flat.normal_(0.0, 3.0 / math.sqrt(max(1, st["n"])), generator=_gen(seed, 50 + i))
        out = torch.zeros_like(flat)
        at = 0
        for s, r in zip(sizes, room):
            flat[at + s:at + r] = 0
            st["grads"].append(flat[at:at + s])
            st["outs"].append(out[at:at + s])
            at += r
        st["flat"].append(flat)
        st["out"].append(out)
    st["norm"] = torch.zeros(1, device="cuda")
    st["ws"] = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")   # the workspace a program keeps
    st["max_norm"] = 1.0


def prepare(case, seed):
    op, st = case["op"], dict(case)
    if op == "clip":
        _gradients(st, seed)
        return st
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    counts = _counts(R, E, seed)
    bounds = [0] + counts.cumsum(0).tolist()
    st["groups"] = [(e, bounds[e], bounds[e + 1]) for e in range(E) if op == "wgrad" or bounds[e + 1] > bounds[e]]
    st["offsets"] = torch.tensor(bounds, dtype=torch.int32, device="cuda") if E > 1 else None
    if op == "ffn":
        st["x"] = _normal((R, K), seed, 1)
        st["w_gate"] = _weights(E, (N, K), seed, 1000, K ** -0.5)
        st["w_up"] = _weights(E, (N, K), seed, 3000, K ** -0.5)
        st["h"] = torch.zeros(R, N, dtype=BF16, device="cuda")
        st["gate"] = torch.zeros_like(st["h"]) if case["save"] else None
        st["up"] = torch.zeros_like(st["h"]) if case["save"] else None
    elif op == "grad":
        st["dy"] = _normal((R, K), seed, 1, 1e-3)
        st["w_down"] = _weights(E, (K, N), seed, 1000, N ** -0.5)
        st["gate"], st["up"] = _normal((R, N), seed, 2), _normal((R, N), seed, 3)
        st["dgate"], st["dup"] = torch.zeros_like(st["gate"]), torch.zeros_like(st["up"])
    elif op == "matmul":
        shape = (K, N) if case["transposed"] else (N, K)
        st["a"] = [_normal((R, K), seed, 1 + i) for i in range(case["pairs"])]
        st["w"] = [_weights(E, shape, seed, 1000 + 2000 * i, K ** -0.5) for i in range(case["pairs"])]
        st["y"] = torch.zeros(R, N, dtype=DTYPE[case["out"]], device="cuda")
    else:
        st["dy"] = [_normal((R, N), seed, 1 + i, 1e-3) for i in range(case["pairs"])]
        st["x"] = _normal((R, K), seed, 5)
        st["dw"] = [torch.zeros(E, N, K, dtype=DTYPE[case["out"]], device="cuda") for _ in range(case["pairs"])]
    return st


# ------------------------------------------------------------------ plain forms
def _plain_ffn(st):
    R, N = st["R"], st["N"]
    h = torch.empty(R, N, dtype=BF16, device="cuda")
    gate, up = (torch.empty_like(h), torch.empty_like(h)) if st["save"] else (None, None)
    for e, lo, hi in st["groups"]:
        x = st["x"][lo:hi].float()
        g, u = torch.matmul(x, st["w_gate"][e].float().t()), torch.matmul(x, st["w_up"][e].float().t())
        h[lo:hi] = (g / (1 + torch.exp(-g)) * u).to(BF16)
        if st["save"]:
            gate[lo:hi], up[lo:hi] = g.to(BF16), u.to(BF16)
    return (h, gate, up) if st["save"] else h


def _plain_grad(st):
    dgate, dup = torch.empty_like(st["gate"]), torch.empty_like(st["up"])
    for e, lo, hi in st["groups"]:
        dh = torch.matmul(st["dy"][lo:hi].float(), st["w_down"][e].float())
        g, u = st["gate"][lo:hi].float(), st["up"][lo:hi].float()
        s = 1 / (1 + torch.exp(-g))
        dgate[lo:hi] = (dh * u * (s * (1 + g * (1 - s)))).to(BF16)
        dup[lo:hi] = (dh * (g * s)).to(BF16)
    return dgate, dup


def _plain_matmul(st):
    y = torch.empty(st["R"], st["N"], dtype=DTYPE[st["out"]], device="cuda")
    for e, lo, hi in st["groups"]:
        w = [w[e].float() if st["transposed"] else w[e].float().t() for w in st["w"]]
        y[lo:hi] = sum(torch.matmul(a[lo:hi].float(), m) for a, m in zip(st["a"], w)).to(y.dtype)
    return y


def _plain_wgrad(st):
    dw = [torch.empty(st["E"], st["N"], st["K"], dtype=DTYPE[st["out"]], device="cuda") for _ in st["dy"]]
    for e, lo, hi in st["groups"]:
        x = st["x"][lo:hi].float()
        for d, dy in zip(dw, st["dy"]):
            d[e] = torch.matmul(dy[lo:hi].float().t(), x).to(d.dtype)
    return dw


def _plain_clip(st):
    total = sum((f.double() * f.double()).sum() for f in st["flat"])
    norm = torch.sqrt(total).float().reshape(1)
    scale = (st["max_norm"] / (norm + 1e-6)).clamp_max(1.0)
    return [norm] + [(f.float() * scale).to(f.dtype) for f in st["flat"]]


# ------------------------------------------------------------------ one pass
def run(state):
    st, op = state, state["op"]
    if not own:
        return {"ffn": _plain_ffn, "grad": _plain_grad, "matmul": _plain_matmul, "wgrad": _plain_wgrad,
                "clip": _plain_clip}[op](st)
    import latent_mixture_experts_router_gb300 as lm
    if op == "ffn":
        lm.lmoe_gated_ffn(st["x"], st["w_gate"], st["w_up"], st["h"], gate=st["gate"], up=st["up"],
                          offsets=st["offsets"])
        return (st["h"], st["gate"], st["up"]) if st["save"] else st["h"]
    if op == "grad":
        lm.lmoe_gated_ffn_grad(st["dy"], st["w_down"], st["gate"], st["up"], st["dgate"], st["dup"],
                               offsets=st["offsets"])
        return st["dgate"], st["dup"]
    if op == "matmul":
        a2, w2 = (st["a"][1], st["w"][1]) if st["pairs"] == 2 else (None, None)
        lm.lmoe_matmul_bf16(st["a"][0], st["w"][0], st["y"], offsets=st["offsets"], a2=a2, w2=w2,
                            transposed=st["transposed"])
        return st["y"]
    if op == "wgrad":
        dy2, dw2 = (st["dy"][1], st["dw"][1]) if st["pairs"] == 2 else (None, None)
        lm.lmoe_matmul_bf16_wgrad(st["dy"][0], st["x"], st["dw"][0], offsets=st["offsets"], dy2=dy2, dw2=dw2)
        return st["dw"]
    lm.lmoe_clip_grad_norm(st["grads"], st["norm"], st["max_norm"], st["ws"], out=st["outs"])
    return [st["norm"]] + st["out"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "clip":
        n, b = case["n"], {"f32": 4, "bf16": 2, "mixed": 3}[case["dtype"]]
        return {"bytes": 2 * n * b + 4, "flops": 3 * n}
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    live = E * (1 - (1 - 1 / E) ** R)   # experts that R rows reach, about
    if op == "ffn":
        return {"bytes": 2 * (R * K + 2 * live * N * K + R * N * (3 if case["save"] else 1)), "flops": 4 * R * N * K}
    if op == "grad":
        return {"bytes": 2 * (R * K + live * N * K + 4 * R * N), "flops": 2 * R * N * K}
    ob, p = 2 if case["out"] == "bf16" else 4, case["pairs"]
    if op == "matmul":
        return {"bytes": 2 * p * (R * K + live * N * K) + R * N * ob, "flops": 2 * p * R * N * K}
    return {"bytes": 2 * R * (p * N + K) + p * E * N * K * ob, "flops": 2 * p * R * N * K}


# ------------------------------------------------------------------ the values in 64 bits
def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for g in st["grads"]:
            total += torch.linalg.vector_norm(g.double()) ** 2
        norm = total.sqrt()
        scale = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
        return [norm.reshape(1)] + [f.double() * scale for f in st["flat"]]
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    if op == "wgrad":
        dw = [torch.zeros(E, N, K, dtype=torch.float64, device="cuda") for _ in st["dy"]]
        for e, lo, hi in st["groups"]:
            for d, dy in zip(dw, st["dy"]):
                d[e] = torch.einsum("rn,rk->nk", dy[lo:hi].double(), st["x"][lo:hi].double())
        return dw
    outs = [torch.zeros(R, N, dtype=torch.float64, device="cuda") for _ in range(3)]
    for e, lo, hi in st["groups"]:
        if op == "ffn":
            x = st["x"][lo:hi].double()
            g = torch.einsum("rk,nk->rn", x, st["w_gate"][e].double())
            u = torch.einsum("rk,nk->rn", x, st["w_up"][e].double())
            outs[0][lo:hi], outs[1][lo:hi], outs[2][lo:hi] = g * torch.sigmoid(g) * u, g, u
        elif op == "grad":
            dh = torch.einsum("rk,kn->rn", st["dy"][lo:hi].double(), st["w_down"][e].double())
            g, u = st["gate"][lo:hi].double(), st["up"][lo:hi].double()
            sig = torch.sigmoid(g)
            outs[0][lo:hi] = dh * u * (sig + g * sig * torch.sigmoid(-g))
            outs[1][lo:hi] = dh * g * sig
        else:
            for a, w in zip(st["a"], st["w"]):
                form = "rk,kn->rn" if case["transposed"] else "rk,nk->rn"
                outs[0][lo:hi] += torch.einsum(form, a[lo:hi].double(), w[e].double())
    if op == "ffn":
        return tuple(outs) if case["save"] else outs[0]
    return (outs[0], outs[1]) if op == "grad" else outs[0]
