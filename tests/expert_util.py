"""Plain forms in 64 bits of the bf16 experts' operators and of the gradients' norm, written from the formulas of
include/latent_moe.h, each with a bound of the error that its arithmetic allows.

Bounds.  A product of two bf16 values is exact in fp32.  A sum of K of them in fp32, in any order, each addition off by
at most 2^-23 of the running sum (a rounding is half of that; tensor cores may truncate), is off by at most
K 2^-23 S, S the sum of the products' magnitudes.  A result stored in bf16 is rounded once: 2^-8 of it."""
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF16 = torch.bfloat16
TINY = 2.0 ** -126


def groups(offsets, rows, E):
    """(first, end) row of each expert, clamped as the operators clamp them."""
    if offsets is None:
        return [(0, rows)]
    off = [min(max(int(v), 0), rows) for v in offsets.tolist()]
    return [(off[e], max(off[e], off[e + 1])) for e in range(E)]


def experts(w):
    return w if w.dim() == 3 else w[None]


def product(a, w, offsets=None, transposed=False):
    """(sum, bound) [rows, N] of each row with its expert's weights; rows of no expert are NaN."""
    w = experts(w)
    N, K = (w.shape[2], w.shape[1]) if transposed else (w.shape[1], w.shape[2])
    out = torch.full((a.shape[0], N), float("nan"), dtype=torch.float64, device=a.device)
    tol = out.clone()
    for e, (lo, hi) in enumerate(groups(offsets, a.shape[0], w.shape[0])):
        m = w[e].double() if transposed else w[e].double().t()
        x = a[lo:hi].double()
        out[lo:hi] = x @ m
        tol[lo:hi] = (x.abs() @ m.abs()) * K * 2.0 ** -23 + TINY
    return out, tol


def rounded(v, tol, dtype):
    """The bound of v (off by at most tol) after it is stored in dtype."""
    return tol + HALF[dtype] * (v.abs() + tol) + TINY


def gated(x, w_gate, w_up, offsets=None):
    """((h, bound), (g, bound), (u, bound)), all bf16 results.

    silu's slope is below 1.1, so h moves by 1.1 tg (|u| + tu) + |silu(g)| tu; exp(-g) in fp32 is off by a few units
    and 2^-22 |g| relatively, the reciprocal and products by a few more: (1 + |g|) 2^-19 of h covers them."""
    (g, tg), (u, tu) = product(x, w_gate, offsets), product(x, w_up, offsets)
    s = g * torch.sigmoid(g)
    h = s * u
    th = 1.1 * tg * (u.abs() + tu) + s.abs() * tu + 2.0 ** -19 * (1 + g.abs()) * h.abs()
    return (h, rounded(h, th, BF16)), (g, rounded(g, tg, BF16)), (u, rounded(u, tu, BF16))


def gated_grad(dy, w_down, gate, up, offsets=None):
    """((dgate, bound), (dup, bound)).  The factors are functions of the given gate and up: off by 2^-19 (1 + |g|) of
    s, once more times 1 + |g| where 1 - s is taken."""
    dh, t = product(dy, w_down, offsets, transposed=True)
    g, u = gate.double(), up.double()
    s = torch.sigmoid(g)
    fg, fu = u * (s + g * s * torch.sigmoid(-g)), g * s
    eg = 2.0 ** -19 * (1 + g.abs()) ** 2 * s * u.abs()
    eu = 2.0 ** -19 * (1 + g.abs()) * fu.abs()
    dg, du = dh * fg, dh * fu
    tg = t * (fg.abs() + eg) + dh.abs() * eg
    tu = t * (fu.abs() + eu) + dh.abs() * eu
    return (dg, rounded(dg, tg, BF16)), (du, rounded(du, tu, BF16))


def wgrad(dy, x, E, offsets=None, start=None):
    """(dw, bound) [E, N, K] (start: what is added to)."""
    N, K = dy.shape[1], x.shape[1]
    dw = torch.zeros(E, N, K, dtype=torch.float64, device=dy.device)
    tol = torch.zeros_like(dw)
    for e, (lo, hi) in enumerate(groups(offsets, dy.shape[0], E)):
        d, v = dy[lo:hi].double(), x[lo:hi].double()
        dw[e] = d.t() @ v
        tol[e] = (d.abs().t() @ v.abs()) * (hi - lo) * 2.0 ** -23
    if start is not None:
        dw, tol = dw + start.double(), tol + 2.0 ** -24 * (dw.abs() + start.double().abs())
    return dw, tol


def close(got, want, tol, what=""):
    """got within tol of want; where want is not finite, got is the same infinity or NaN."""
    got, fine = got.double(), torch.isfinite(want)
    assert got.shape == want.shape, what
    off = (got - want).abs()
    bad = fine & ~(off <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {off[bad].max():.3g} " \
                                f"at {bad.nonzero()[0].tolist()} (bound {tol[bad][off[bad].argmax()]:.3g})"
    rest = ~fine
    if bool(rest.any()):
        assert torch.equal(torch.isnan(got[rest]), torch.isnan(want[rest])), what
        n = ~torch.isnan(want[rest])
        assert torch.equal(got[rest][n], want[rest][n]), what


def offsets_of(counts, device="cuda"):
    c = torch.tensor([0] + list(counts)).cumsum(0)
    return c.to(torch.int32).to(device)


def norm(grads):
    return sum((g.double() ** 2).sum() for g in grads).sqrt() if grads else torch.zeros((), dtype=torch.float64)


def clipped(g, norm_, max_norm):
    """(value, bound) of a gradient clipped with the fp32 norm: f is two fp32 roundings off, the product one more."""
    f = min(1.0, max_norm / (float(norm_) + 1e-6))
    v = g.double() * f
    return v, (HALF[g.dtype] + 4 * 2.0 ** -24) * v.abs() + TINY * 2
