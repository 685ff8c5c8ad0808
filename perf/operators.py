"""The operators that train and serve the router and 8-bit experts, case by case: inputs, a plain
form in elementary torch operations, the library's calls, and the values in 64 bits.

op "losses"   the router's balance loss and z loss with per-expert counts and mean probabilities
op "grad"     the gradient of the router logits: routing weights, balance loss and z loss together
op "rows"     8-bit quantisation of rows, a scale per 1 x 128 block, rows gathered by token
op "weight"   8-bit quantisation of weights, a scale per 128 x 128 block, also transposed
op "cols"     8-bit quantisation along the token axis, transposed, expert by expert
op "matmul"   product of 8-bit rows with 8-bit weights (one matrix, or one per expert)
op "wgrad"    weight gradient from 8-bit operands that are blocked along the token axis

Set ``own`` to run the library's calls instead of the plain forms.
"""
import math

import torch

own = False

MAXIMUM = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
SMALLEST = 2.0 ** -126        # the smallest scale: an all-zero block keeps a finite reciprocal
BLOCK = 128


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a small model's micro-batch: the time of a call
        dict(name="losses-T64-E16", op="losses", T=64, E=16, k=2, dtype="f32", live=64),
        # a long prefill or training chunk over 256 experts, its last rows padding
        dict(name="losses-T16384-E256", op="losses", T=16384, E=256, k=8, dtype="f32", live=16001),
        # a batch of decoded tokens trained on afterwards
        dict(name="grad-T512-E256", op="grad", T=512, E=256, k=8, dtype="f32", live=512),
        # a training chunk with logits in 16 bits and padded rows
        dict(name="grad-T16384-E256-bf16", op="grad", T=16384, E=256, k=8, dtype="bf16", live=16001),
        # 4096 tokens copied to their 8 experts' rows on the way into 8 bits
        dict(name="rows-T4096-k8", op="rows", T=4096, k=8, K=4096, dtype="bf16", fmt="e4m3"),
        # a group of experts' weights in 8 bits after an optimiser step, both orientations
        dict(name="weight-E8", op="weight", E=8, N=4096, K=4096, dtype="bf16", fmt="e4m3"),
        # gradients of 16384 routed rows, expert by expert, for the weight gradient
        dict(name="cols-R16384-E32", op="cols", R=16384, E=32, K=4096, dtype="bf16", fmt="e5m2"),
        # serving: one token, 8 experts' weights streamed
        dict(name="matmul-T1-E64", op="matmul", R=8, E=64, N=4096, K=4096, a_fmt="e4m3", out="bf16"),
        # prefill: 4096 tokens on 8 of 64 experts each
        dict(name="matmul-T4096-E64", op="matmul", R=32768, E=64, N=4096, K=4096, a_fmt="e4m3", out="bf16"),
        # the input gradient of a dense layer, gradients in e5m2, an odd number of rows
        dict(name="matmul-dense-M2047", op="matmul", R=2047, E=1, N=8192, K=4096, a_fmt="e5m2", out="f32"),
        # weight gradients of 16 experts over 8192 routed rows
        dict(name="wgrad-R8192-E16", op="wgrad", R=8192, E=16, N=4096, K=2048, a_fmt="e5m2", out="f32"),
        # weight gradient of a dense layer over 1000 tokens
        dict(name="wgrad-dense-R1000", op="wgrad", R=1000, E=1, N=4096, K=8192, a_fmt="e5m2", out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["losses", "grad", "rows", "weight", "cols", "matmul", "wgrad", "matmul"])
    dtype = rng.choice(["f32", "bf16"])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    if op in ("losses", "grad"):
        E = _log(rng, 2, 1024)
        T = min(_log(rng, 1, 16384), 4194304 // E)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 16)), dtype=dtype,
                    live=max(1, T - rng.randint(0, T // 8)))
    K = 16 * _log(rng, 4, 512)
    if op == "rows":
        k = rng.randint(1, 8)
        T = _log(rng, 1, max(2, 134217728 // (K * k) // (2 if dtype == "f32" else 1)))
        return dict(op=op, T=T, k=k, K=K, dtype=dtype, fmt=fmt)
    if op == "weight":
        N = 16 * _log(rng, 4, 256)
        return dict(op=op, E=_log(rng, 1, max(2, 67108864 // (N * K))), N=N, K=K, dtype=dtype, fmt=fmt)
    E = _log(rng, 1, 64)
    if op == "cols":
        return dict(op=op, R=_log(rng, 1, max(2, 33554432 // K)), E=E, K=K, dtype=dtype, fmt=fmt)
    N = _log(rng, 64, 8192)
    E = max(1, min(E, 536870912 // (N * K)))
    R = min(_log(rng, 1, 32768), 250000000000 // (N * K), 134217728 // max(N, K))
    if op == "wgrad":
        E = max(1, min(E, 134217728 // (N * K)))
    return dict(op=op, R=max(1, R), E=E, N=N, K=K, a_fmt=fmt, out=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------ inputs
def _gen(seed, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + n)
    return g


def _normal(shape, seed, n, std=1.0):
    return torch.randn(shape, generator=_gen(seed, n), device="cuda") * std


def _counts(R, E, seed):
    """Rows of each expert: uneven, some experts often without any."""
    w = torch.exp(0.7 * _normal((E,), seed, 90))
    ids = torch.multinomial(w, R, replacement=True, generator=_gen(seed, 91))
    return torch.bincount(ids, minlength=E)


def _offsets(counts):
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def _padded(counts):
    return (counts + BLOCK - 1) // BLOCK * BLOCK


def _made(x, fmt, rows_blocked):
    """Codes and scales of x [rows, K] as a program that has them in 8 bits keeps them: a scale per
    128 x 128 block (rows_blocked) or per 1 x 128 block, the latter with the block index first."""
    rows, K = x.shape
    R = BLOCK if rows_blocked else 1
    p = torch.nn.functional.pad(x, (0, -K % BLOCK, 0, -rows % R))
    p = p.view(p.shape[0] // R, R, p.shape[1] // BLOCK, BLOCK)
    s = (p.abs().amax((1, 3)) / MAXIMUM[fmt]).clamp_min(SMALLEST)
    q = (p / s[:, None, :, None]).to(F8[fmt]).view(torch.uint8)
    codes = q.reshape(q.shape[0] * R, -1)[:rows, :K].contiguous().view(F8[fmt])
    return codes, (s if rows_blocked else s.t()).contiguous()


def prepare(case, seed):
    op, st = case["op"], dict(case)
    if op in ("losses", "grad"):
        T, E, k = case["T"], case["E"], case["k"]
        bias = 0.5 * _normal((E,), seed, 1)
        logits = (1.5 * _normal((T, E), seed, 2) + bias).to(DTYPE[case["dtype"]])
        mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
        mask[torch.randperm(T, generator=_gen(seed, 3), device="cuda")[: case["live"]]] = 1
        idx = logits.float().topk(k, dim=1).indices.to(torch.int32)
        st.update(logits=logits, mask=mask, idx=idx)
        live = mask.bool()
        counts = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        if op == "losses":
            ws = 4 * (2 * E + 4) * 256   # the workspace a program keeps
            st.update(counts=counts, mean_probs=torch.zeros(E, device="cuda"), losses=torch.zeros(2, device="cuda"),
                      ws=torch.zeros(ws, dtype=torch.uint8, device="cuda"))
        else:
            counts[:E] = torch.bincount(idx[live].reshape(-1).long(), minlength=E).int()
            counts[E] = live.sum().int()
            st.update(counts=counts, gw=_normal((T, k), seed, 4), gl=torch.tensor([0.01, 0.001], device="cuda"),
                      dlogits=torch.empty_like(logits))
        return st
    if op in ("rows", "weight", "cols"):
        dt, fmt, K = DTYPE[case["dtype"]], case["fmt"], case["K"]
        kb = -(-K // BLOCK)
        if op == "rows":
            T, R = case["T"], case["T"] * case["k"]
            st["src"] = (_normal((T, K), seed, 1) * torch.exp(_normal((T, 1), seed, 2))).to(dt)
            st["index"] = (torch.randperm(R, generator=_gen(seed, 3), device="cuda") // case["k"]).to(torch.int32)
            st["codes"] = torch.zeros(R, K, dtype=torch.uint8, device="cuda").view(F8[fmt])
            st["scales"] = torch.zeros(kb, R, device="cuda")
        elif op == "weight":
            E, N = case["E"], case["N"]
            st["src"] = _normal((E, N, K), seed, 1, K ** -0.5).to(dt)
            nb = -(-N // BLOCK)
            st["codes"] = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda").view(F8[fmt])
            st["codes_t"] = torch.zeros(E, K, N, dtype=torch.uint8, device="cuda").view(F8[fmt])
            st["scales"] = torch.zeros(E, nb, kb, device="cuda")
            st["scales_t"] = torch.zeros(E, kb, nb, device="cuda")
        else:
            R, E = case["R"], case["E"]
            counts = _counts(R, E, seed)
            st["src"] = (_normal((R, K), seed, 1) * torch.exp(_normal((1, K), seed, 2)) * 1e-3).to(dt)
            st["offsets"] = _offsets(counts)
            Rp = int(_capacity(R, E))
            st["codes"] = torch.zeros(K, Rp, dtype=torch.uint8, device="cuda").view(F8[fmt])
            st["scales"] = torch.zeros(Rp // BLOCK, K, device="cuda")
            # where each row goes in the padded order, for the plain form
            shift = (_padded(counts).cumsum(0) - _padded(counts)) - (counts.cumsum(0) - counts)
            st["place"] = torch.arange(R, device="cuda") + torch.repeat_interleave(shift, counts)
            st["rows_padded"] = int(_padded(counts).sum())
        return st
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    counts = _counts(R, E, seed)
    st["offsets"] = _offsets(counts) if E > 1 else None
    bounds = [0] + counts.cumsum(0).tolist()
    if op == "matmul":
        st["groups"] = [(e, bounds[e], bounds[e + 1]) for e in range(E) if bounds[e + 1] > bounds[e]]
        st["a"], st["a_s"] = _made(_normal((R, K), seed, 1), case["a_fmt"], False)
        w = [_made(_normal((N, K), seed, 100 + e, K ** -0.5), "e4m3", True) for e in range(E)]
        st["w"] = torch.stack([c.view(torch.uint8) for c, _ in w]).view(F8["e4m3"])
        st["w_s"] = torch.stack([s for _, s in w])
        st["y"] = torch.zeros(R, N, dtype=DTYPE[case["out"]], device="cuda")
        return st
    padded = _padded(counts)
    st["groups"] = [(e, int(p) // BLOCK, int(p + n) // BLOCK) for e, (p, n) in
                    enumerate(zip((padded.cumsum(0) - padded).tolist(), padded.tolist()))]
    Rp = int(_capacity(R, E))
    shift = (padded.cumsum(0) - padded) - (counts.cumsum(0) - counts)
    place = torch.arange(R, device="cuda") + torch.repeat_interleave(shift, counts)
    for name, n, dim, fmt in (("dy", 1, N, case["a_fmt"]), ("x", 2, K, "e4m3")):
        t = torch.zeros(dim, Rp, device="cuda")
        t[:, place] = _normal((R, dim), seed, n).t() * (1e-3 if name == "dy" else 1.0)
        st[name], st[name + "_s"] = _made(t, fmt, False)
        del t
    st["dw"] = torch.zeros(E, N, K, dtype=DTYPE[case["out"]], device="cuda")
    return st


def _capacity(R, E):
    """Columns that any split of R rows among E experts fits in, each expert's rows padded to 128."""
    return (R + 127 * min(E, R)) // BLOCK * BLOCK


# ------------------------------------------------------------------ plain forms
def _plain_losses(st):
    T, E, k = st["T"], st["E"], st["k"]
    live = st["mask"].bool()
    l = st["logits"].float()
    m = l.amax(1, keepdim=True)
    ex = torch.exp(l - m)
    tot = ex.sum(1, keepdim=True)
    lse = (m + torch.log(tot))[:, 0].double()
    n = live.sum()
    nd = n.clamp_min(1).double()
    ids = torch.where(live[:, None], st["idx"].long(), E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=l.device)
    counts.scatter_add_(0, ids.reshape(-1), torch.ones_like(ids).reshape(-1))
    counts[E] = n
    mean = torch.where(live[:, None], ex / tot, 0.0).double().sum(0) / nd
    balance = E * (counts[:E].double() / (k * nd) * mean).sum()
    z = torch.where(live, lse * lse, 0.0).sum() / nd
    return counts.int(), mean.float(), torch.stack([balance, z]).float()


def _plain_grad(st):
    E, k = st["E"], st["k"]
    live = st["mask"].bool()[:, None]
    l = st["logits"].float()
    m = l.amax(1, keepdim=True)
    ex = torch.exp(l - m)
    tot = ex.sum(1, keepdim=True)
    p, lse = ex / tot, m + torch.log(tot)
    n = st["counts"][E].clamp_min(1).float()
    f = st["counts"][:E].float() / (k * n)
    d = st["gl"][0] * (E / n) * p * (f - (p * f).sum(1, keepdim=True)) + st["gl"][1] * (2.0 / n) * lse * p
    ids = st["idx"].long()
    sel = l.gather(1, ids)
    w = torch.exp(sel - sel.amax(1, keepdim=True))
    w = w / w.sum(1, keepdim=True)
    gw = st["gw"]
    d = d.scatter_add(1, ids, w * (gw - (w * gw).sum(1, keepdim=True)))
    return torch.where(live, d, 0.0).to(st["logits"].dtype)


def _plain_blocks(p, dims, fmt):
    """p: [..] split in blocks whose own axes are `dims`; codes and scales."""
    top = torch.tensor(MAXIMUM[fmt], device=p.device)
    s = (p.abs().amax(dims, keepdim=True) / top).clamp_min(SMALLEST)
    return (p * torch.reciprocal(s)).to(F8[fmt]).view(torch.uint8), s


def _plain_rows(st):
    x = st["src"].float()[st["index"].long()]
    R, K = x.shape
    q, s = _plain_blocks(torch.nn.functional.pad(x, (0, -K % BLOCK)).view(R, -1, BLOCK), (2,), st["fmt"])
    return q.view(R, -1)[:, :K].contiguous().view(F8[st["fmt"]]), s[:, :, 0].t().contiguous()


def _plain_weight(st):
    x = st["src"].float()
    E, N, K = x.shape
    p = torch.nn.functional.pad(x, (0, -K % BLOCK, 0, -N % BLOCK))
    p = p.view(E, p.shape[1] // BLOCK, BLOCK, p.shape[2] // BLOCK, BLOCK)
    q, s = _plain_blocks(p, (2, 4), st["fmt"])
    q = q.reshape(E, p.shape[1] * BLOCK, p.shape[3] * BLOCK)[:, :N, :K].contiguous()
    s = s[:, :, 0, :, 0].contiguous()
    return q.view(F8[st["fmt"]]), s, q.transpose(1, 2).contiguous().view(F8[st["fmt"]]), s.transpose(1, 2).contiguous()


def _plain_cols(st):
    x = st["src"].float()
    K = x.shape[1]
    n = st["rows_padded"]
    p = torch.zeros(n, K, device=x.device)
    p[st["place"]] = x
    q, s = _plain_blocks(p.t().reshape(K, -1, BLOCK), (2,), st["fmt"])
    free = st["codes"].shape[1] - n   # behind the last expert's columns
    codes = torch.nn.functional.pad(q.reshape(K, n), (0, free))
    return codes.view(F8[st["fmt"]]), torch.nn.functional.pad(s[:, :, 0].t(), (0, 0, 0, free // BLOCK))


def _values(codes, scales, rows_blocked):
    """fp32 values of [rows, K] codes with their block scales."""
    rows, K = codes.shape
    if rows_blocked:
        s = scales.repeat_interleave(BLOCK, 0)[:rows]
    else:
        s = scales.t()
    return codes.float() * s.repeat_interleave(BLOCK, 1)[:, :K]


def _plain_matmul(st):
    y = torch.empty(st["R"], st["N"], dtype=DTYPE[st["out"]], device="cuda")
    for e, lo, hi in st["groups"]:
        a = _values(st["a"][lo:hi], st["a_s"][:, lo:hi], False)
        y[lo:hi] = torch.matmul(a, _values(st["w"][e], st["w_s"][e], True).t()).to(y.dtype)
    return y


def _plain_wgrad(st):
    dw = torch.empty(st["E"], st["N"], st["K"], dtype=DTYPE[st["out"]], device="cuda")
    for e, lo, hi in st["groups"]:
        dy = _values(st["dy"][:, lo * BLOCK:hi * BLOCK], st["dy_s"][lo:hi], False)
        x = _values(st["x"][:, lo * BLOCK:hi * BLOCK], st["x_s"][lo:hi], False)
        dw[e] = torch.matmul(dy, x.t()).to(dw.dtype)
    return dw


# ------------------------------------------------------------------ one pass
def run(state):
    st, op = state, state["op"]
    if not own:
        return {"losses": _plain_losses, "grad": _plain_grad, "rows": _plain_rows, "weight": _plain_weight,
                "cols": _plain_cols, "matmul": _plain_matmul, "wgrad": _plain_wgrad}[op](st)
    import latent_mixture_experts_router_gb300 as lm
    if op == "losses":
        lm.lmoe_router_losses(st["logits"], st["idx"], st["counts"], st["mean_probs"], st["losses"], st["ws"],
                              row_mask=st["mask"])
        return st["counts"], st["mean_probs"], st["losses"]
    if op == "grad":
        lm.lmoe_router_grad(st["logits"], st["idx"], st["counts"], st["dlogits"], topk_w_grad=st["gw"],
                            loss_grads=st["gl"], row_mask=st["mask"])
        return st["dlogits"]
    if op == "rows":
        lm.lmoe_quantize_fp8_rows(st["src"], st["codes"], st["scales"], row_index=st["index"])
        return st["codes"], st["scales"]
    if op == "weight":
        lm.lmoe_quantize_fp8_weight(st["src"], st["codes"], st["scales"], st["codes_t"], st["scales_t"])
        return st["codes"], st["scales"], st["codes_t"], st["scales_t"]
    if op == "cols":
        lm.lmoe_quantize_fp8_cols(st["src"], st["codes"], st["scales"], offsets=st["offsets"])
        return st["codes"], st["scales"]
    if op == "matmul":
        lm.lmoe_matmul_fp8(st["a"], st["a_s"], st["w"], st["w_s"], st["y"], offsets=st["offsets"])
        return st["y"]
    lm.lmoe_matmul_fp8_wgrad(st["dy"], st["dy_s"], st["x"], st["x_s"], st["dw"], offsets=st["offsets"])
    return st["dw"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("losses", "grad"):
        T, E, k, n = case["T"], case["E"], case["k"], case["live"]
        b = 2 if case["dtype"] == "bf16" else 4
        if op == "losses":
            return {"bytes": n * (E * b + 4 * k) + T + 4 * (2 * E + 3), "flops": 6 * n * E}
        return {"bytes": n * (E * b + 8 * k) + T * (E * b + 1) + 4 * (E + 3), "flops": 12 * n * E}
    if op in ("rows", "weight", "cols"):
        K, b = case["K"], 2 if case["dtype"] == "bf16" else 4
        kb = -(-K // BLOCK)
        if op == "rows":
            T, R = case["T"], case["T"] * case["k"]
            return {"bytes": T * K * b + R * (K + 4 * kb + 4), "flops": 3 * R * K}
        if op == "weight":
            n = case["E"] * case["N"] * K
            return {"bytes": n * b + 2 * n + 8 * case["E"] * kb * -(-case["N"] // BLOCK), "flops": 3 * n}
        n = case["R"] * K
        return {"bytes": n * b + n + 4 * K * -(-case["R"] // BLOCK), "flops": 3 * n}
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    ob = 2 if case["out"] == "bf16" else 4
    if op == "matmul":
        live = E * (1 - (1 - 1 / E) ** R)   # experts that R rows reach, about
        return {"bytes": R * K + live * N * K + R * N * ob, "flops": 2 * R * N * K}
    return {"bytes": R * (N + K) + E * N * K * ob, "flops": 2 * R * N * K}


# ------------------------------------------------------------------ the values in 64 bits
def _nearest(v, fmt):
    """v (float64) rounded to the nearest value of the 8-bit format, ties to even."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    _, e = torch.frexp(v)
    step = (((e.long() - 1).clamp_min(low) - bits + 1023) << 52).view(torch.float64)   # a power of two
    return (torch.round(v / step) * step).clamp(-MAXIMUM[fmt], MAXIMUM[fmt])


def _exact_blocks(x, axes, fmt):
    """The rule in its own words: scale = fp32(amax / largest), code = nearest(fp32(x * fp32(1 / scale)))."""
    s = (x.abs().amax(axes, keepdim=True) / MAXIMUM[fmt]).float().double().clamp_min(SMALLEST)
    r = (1.0 / s).float().double()
    return _nearest((x * r).float().double(), fmt), s


def _exact_product(p, ps, q, qs):
    """sum over blocks of 128: ps[i, b] qs[j, b] (p[i, block b] . q[j, block b]), all float64."""
    K = p.shape[1]
    kb = -(-K // BLOCK)
    out = torch.zeros(p.shape[0], q.shape[0], dtype=torch.float64, device=p.device)
    for b0 in range(0, kb, 8):
        b1 = min(kb, b0 + 8)
        cols = slice(b0 * BLOCK, min(K, b1 * BLOCK))
        left = p[:, cols].double() * ps[:, b0:b1].double().repeat_interleave(BLOCK, 1)[:, : p[:, cols].shape[1]]
        right = q[:, cols].double() * qs[:, b0:b1].double().repeat_interleave(BLOCK, 1)[:, : p[:, cols].shape[1]]
        out += left @ right.t()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("losses", "grad"):
        E, k = case["E"], case["k"]
        rows = st["mask"].nonzero()[:, 0]
        n = rows.numel()
        l = st["logits"][rows].double()
        p, lse = torch.softmax(l, 1), torch.logsumexp(l, 1)
        counts = torch.bincount(st["idx"][rows].reshape(-1).long(), minlength=E)
        f = counts.double() / (k * n)
        if op == "losses":
            loss = torch.stack([E * (f * p.mean(0)).sum(), (lse ** 2).mean()])
            return torch.cat([counts, counts.new_tensor([n])]).int(), p.mean(0), loss
        g = st["gl"].double()
        d = g[0] * (E / n) * p * (f - (p @ f)[:, None]) + g[1] * (2.0 / n) * lse[:, None] * p
        ids = st["idx"][rows].long()
        w = torch.softmax(l.gather(1, ids), 1)
        gw = st["gw"][rows].double()
        d.scatter_add_(1, ids, w * (gw - (w * gw).sum(1, keepdim=True)))
        full = torch.zeros(case["T"], E, dtype=torch.float64, device="cuda")
        full[rows] = d
        return full
    if op in ("rows", "weight", "cols"):
        fmt, K = case["fmt"], case["K"]
        x = st["src"].double()
        if op == "rows":
            x = x[st["index"].long()]
            p = torch.nn.functional.pad(x, (0, -K % BLOCK)).unflatten(1, (-1, BLOCK))
            q, s = _exact_blocks(p, (2,), fmt)
            return q.flatten(1)[:, :K], s[..., 0].t()
        if op == "weight":
            qs, ss = [], []
            for m in x:
                p = torch.nn.functional.pad(m, (0, -K % BLOCK, 0, -case["N"] % BLOCK))
                q, s = _exact_blocks(p.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK)), (1, 3), fmt)
                qs.append(q.flatten(2).flatten(0, 1)[: case["N"], :K])
                ss.append(s[:, 0, :, 0])
            q, s = torch.stack(qs), torch.stack(ss)
            return q, s, q.transpose(1, 2), s.transpose(1, 2)
        codes = torch.zeros(st["codes"].shape, dtype=torch.float64, device="cuda")
        scales = torch.zeros(st["scales"].shape, dtype=torch.float64, device="cuda")
        off, at = st["offsets"].tolist(), 0
        for lo, hi in zip(off[:-1], off[1:]):
            for r in range(lo, hi, BLOCK):
                q, s = _exact_blocks(x[r:min(hi, r + BLOCK)], (0,), fmt)
                codes[:, at:at + q.shape[0]] = q.t()
                scales[at // BLOCK] = s[0]
                at += BLOCK
        return codes, scales
    if op == "matmul":
        y = torch.zeros(case["R"], case["N"], dtype=torch.float64, device="cuda")
        for e, lo, hi in st["groups"]:
            ws = st["w_s"][e].repeat_interleave(BLOCK, 0)[: case["N"]]
            y[lo:hi] = _exact_product(st["a"][lo:hi], st["a_s"][:, lo:hi].t(), st["w"][e], ws)
        return y
    dw = torch.zeros(case["E"], case["N"], case["K"], dtype=torch.float64, device="cuda")
    for e, lo, hi in st["groups"]:
        cols = slice(lo * BLOCK, hi * BLOCK)
        dw[e] = _exact_product(st["dy"][:, cols], st["dy_s"][lo:hi].t(), st["x"][:, cols], st["x_s"][lo:hi].t())
    return dw
