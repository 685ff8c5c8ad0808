"""Plain forms in 64 bits of the router's losses and gradient, of the 8-bit quantisers and of the 8-bit
products, written from the formulas of include/latent_moe.h."""
import torch

MAXIMUM = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, E4M3: 2.0 ** -4, E5M2: 2.0 ** -3}
U = 2.0 ** -24


# ------------------------------------------------------------------ the router
def live_rows(l, mask):
    on = (l > -float("inf")).any(1)   # (a comparison with NaN is false: such rows are masked in the tests)
    return on if mask is None else on & mask.bool()


def router_losses(logits, idx, bias=None, mask=None):
    """(losses [2], mean probabilities [E], counts [E + 1]) in float64 and int64."""
    l = logits.double() + (0 if bias is None else bias.double())
    E, k = l.shape[1], idx.shape[1]
    on = live_rows(l, mask)
    l, ids = l[on], idx[on].long().reshape(-1)
    n = l.shape[0]
    counts = torch.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
    if n == 0:
        mean, loss = l.new_zeros(E), l.new_zeros(2)
    else:
        mean = torch.softmax(l, 1).mean(0)
        loss = torch.stack([E * (counts.double() / (k * n) * mean).sum(), (torch.logsumexp(l, 1) ** 2).mean()])
    return loss, mean, torch.cat([counts, counts.new_tensor([n])])


def router_weights(l, idx):
    """Softmax of the selected logits over a row's slots; empty slots and rows without any: 0."""
    E = l.shape[1]
    ok = (idx >= 0) & (idx < E)
    sel = torch.where(ok, l.gather(1, idx.long().clamp(0, E - 1)), -float("inf"))
    m = sel.amax(1, keepdim=True)
    w = torch.where(m > -float("inf"), torch.exp(sel - torch.where(m > -float("inf"), m, 0.0)), 0.0)
    return w / w.sum(1, keepdim=True).clamp_min(1e-300), ok


def router_objective(logits, idx, counts, gw=None, gl=None, bias=None, mask=None):
    """What the gradient is that of: gl . losses (the counts constant) + sum w gw over the live rows."""
    l = logits.double() + (0 if bias is None else bias.double())
    E, k = l.shape[1], idx.shape[1]
    on = live_rows(l, mask)
    l, idx = l[on], idx[on]
    total = l.new_zeros(())
    if gl is not None:
        n = max(int(counts[E]), 1)
        f = counts[:E].double() / (k * n)
        total = total + gl[0].double() * E * (f * torch.softmax(l, 1).sum(0) / n).sum()
        total = total + gl[1].double() * (torch.logsumexp(l, 1) ** 2).sum() / n
    if gw is not None:
        w, ok = router_weights(l, idx)
        total = total + (w * torch.where(ok, gw[on].double(), 0.0)).sum()
    return total


def router_grad(logits, idx, counts, gw=None, gl=None, bias=None, mask=None):
    """(gradient [T, E], bound of its fp32 evaluation) by the formula, float64."""
    l = logits.double() + (0 if bias is None else bias.double())
    T, E = l.shape
    k = idx.shape[1]
    on = live_rows(l, mask)
    d, tol = l.new_zeros(T, E), l.new_zeros(T, E)
    if not bool(on.any()):
        return d, tol
    lv, iv = l[on], idx[on]
    fin = torch.where(torch.isfinite(lv), lv, 0.0)
    top = float(fin.abs().max())
    part, bound = torch.zeros_like(lv), torch.zeros_like(lv)
    if gl is not None:
        n = max(int(counts[E]), 1)
        f = counts[:E].double() / (k * n)
        p, lse = torch.softmax(lv, 1), torch.logsumexp(lv, 1)[:, None]
        gb, gz = gl[0].double() * E / n, gl[1].double() * 2 / n
        dot = (p * f).sum(1, keepdim=True)
        part += p * (gb * (f - dot) + gz * lse)
        # p and dot: the exponent's argument (three roundings of |l - m| <= 2 top, and the bias added
        # to l and to m), two ulps of exp2, sums over at most 32 + 5 terms a lane, a reciprocal and two
        # products; lse: five half steps of its largest logit and the sum's
        rel = U * (3 * 2 * top + 2 * top + 4 + 37 + 37 + 8)
        bound += p * (gb.abs() * (f + dot) * 3 + (gz * lse).abs() * 2) * rel + p * gz.abs() * U * (5 * top + 80)
    if gw is not None:
        w, ok = router_weights(lv, iv)
        g = torch.where(ok, gw[on].double(), 0.0)
        mean = (w * g).sum(1, keepdim=True)
        slots = w * (g - mean)
        size = w * (g.abs() + (w * g.abs()).sum(1, keepdim=True)) * U * (2 * 3 * 2 * top + 4 * top + 60)
        ids = iv.long().clamp(0, E - 1)
        part.scatter_add_(1, ids, torch.where(ok, slots, 0.0))
        bound.scatter_add_(1, ids, torch.where(ok, size, 0.0))
    d[on], tol[on] = part, bound + 1e-37
    return d, tol


# ------------------------------------------------------------------ 8 bits
def nearest(v, fmt):
    """v (float64) rounded to the nearest value of the 8-bit format, ties to even, saturating."""
    bits, low = (3, -6) if fmt == E4M3 else (2, -14)
    _, e = torch.frexp(v)
    step = (((e.long() - 1).clamp_min(low) - bits + 1023) << 52).view(torch.float64)   # a power of two
    return (torch.round(v / step) * step).clamp(-MAXIMUM[fmt], MAXIMUM[fmt])


def rule(x, axes, fmt, pow2=False):
    """Codes' values and scales of x (float64 of fp32 values) with blocks over ``axes``."""
    s = (x.abs().amax(axes, keepdim=True) / MAXIMUM[fmt]).float().double().clamp_min(2.0 ** -126)
    if pow2:
        m, e = torch.frexp(s)
        s = ((e.long() - (m == 0.5).long() + 1023) << 52).view(torch.float64)
    r = (1.0 / s).float().double()
    return nearest((x * r).float().double(), fmt), s


def blocks(x, dim):
    """x with ``dim`` padded by zeros to whole blocks of 128 and split in (blocks, 128)."""
    n = x.shape[dim]
    zeros = x.new_zeros(*x.shape[:dim], -n % 128, *x.shape[dim + 1:])
    return torch.cat([x, zeros], dim).unflatten(dim, (-(-n // 128), 128))


def gathered(src, index):
    x = src.double()
    if index is None:
        return x
    ok = (index >= 0) & (index < src.shape[0])
    if src.shape[0] == 0:
        return x.new_zeros(index.shape[0], src.shape[1])
    return torch.where(ok[:, None], x[index.long().clamp(0, src.shape[0] - 1)], 0.0)


def quantize_rows(x, fmt, pow2=False):
    q, s = rule(blocks(x, 1), (2,), fmt, pow2)
    return q.flatten(1)[:, :x.shape[1]], s[..., 0].t()


def quantize_weight(x, fmt, pow2=False):
    """x [N, K]"""
    q, s = rule(blocks(blocks(x, 1), 0), (1, 3), fmt, pow2)
    return q.flatten(2).flatten(0, 1)[:x.shape[0], :x.shape[1]], s[:, 0, :, 0]


def groups(offsets, rows):
    """[(first row, end)] of the experts, clamped as documented."""
    if offsets is None:
        return [(0, rows)]
    o = offsets.tolist()
    out = []
    for lo, hi in zip(o[:-1], o[1:]):
        lo = min(max(lo, 0), rows)
        out.append((lo, min(max(hi, lo), rows)))
    return out


def quantize_cols(x, offsets, fmt, pow2=False):
    """(codes' values [K, used columns], scales [blocks, K]) of x's rows, expert by expert."""
    q, s = [x.new_zeros(x.shape[1], 0)], [x.new_zeros(0, x.shape[1])]
    for lo, hi in groups(offsets, x.shape[0]):
        if hi > lo:
            qe, se = rule(blocks(x[lo:hi].t(), 1), (2,), fmt, pow2)
            q.append(qe.flatten(1))
            s.append(se[..., 0].t())
    return torch.cat(q, 1), torch.cat(s, 0)


def values(codes, scales, rows_blocked):
    """float64 values of [rows, K] codes; scales [K/128, rows] or, rows_blocked, [rows/128, K/128]."""
    s = scales.double()
    s = s.repeat_interleave(128, 0)[:codes.shape[0]] if rows_blocked else s.t()
    return codes.double() * s.repeat_interleave(128, 1)[:, :codes.shape[1]]


def product(p, q):
    """(p q^T, bound of an fp32 sum of its terms in any order) in float64.

    Per term three products' roundings (two scales, one of them on the block's sum), and n additions
    whose partial sums stay below the sum of the magnitudes, each off by at most a whole step 2^-23
    (the tensor cores may cut off instead of rounding)."""
    n = p.shape[1] + p.shape[1] // 128 + 4
    return p @ q.t(), (p.abs() @ q.abs().t()) * (n * 2.0 ** -23)


def assert_close(got, want, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() > tol
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for "
                             f"{float(want[i])} (tolerance {float(tol[i])})")
