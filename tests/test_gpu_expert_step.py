"""The operators together, as a training step of bf16 experts uses them: routing and its losses, rows in expert order,
the gated block and the down projection, their input and weight gradients, and all gradients clipped to a largest norm; eager,
accumulated over two micro-batches, and captured into a graph.

Every stage is compared, in 64 bits, with the plain operation on the stage's own inputs, with expert_util's bounds; the
whole chain's gradients with those of the same function by automatic differentiation in 64 bits."""
import pytest
import torch

import expert_util as xu
from expert_util import BF16, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    import latent_mixture_experts_router_gb300 as lm
    return lm


class Step:
    """Experts y = down(silu(gate x) * up x) on routed rows; buffers kept from step to step, gradients in fp32."""

    def __init__(self, lm, T, E, k, L, I):
        self.lm, self.T, self.E, self.k, self.L, self.I, self.R = lm, T, E, k, L, I, T * k
        g = torch.Generator(device="cuda").manual_seed(T + E)
        new = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
        self.x, self.logits = new(T, L).to(BF16), 1.5 * new(T, E)
        self.wg, self.wu = new(E, I, L, std=L ** -0.5).to(BF16), new(E, I, L, std=L ** -0.5).to(BF16)
        self.wd = new(E, L, I, std=I ** -0.5).to(BF16)
        self.dy, self.gw = new(self.R, L, std=1e-2).to(BF16), new(T, k)
        self.gl = torch.tensor([0.01, 0.001], device="cuda")
        self.grads = [torch.zeros(w.shape, device="cuda") for w in (self.wg, self.wu, self.wd)] + \
            [torch.zeros(T, E, device="cuda")]
        z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")
        R = self.R
        self.h, self.gate, self.up, self.dgate, self.dup = (z(R, I) for _ in range(5))
        self.y, self.dx = z(R, L), z(R, L)
        self.norm, self.status = z(1, dtype=torch.float32), z(1, dtype=torch.int32)
        self.clipped = [torch.zeros_like(t) for t in self.grads]
        self.ws = z(lm.lmoe_grad_norm_workspace_size(4), dtype=torch.uint8)
        self.lws = z(lm.lmoe_router_losses_workspace_size(T, E), dtype=torch.uint8)
        self.counts, self.mean, self.losses = z(E + 1, dtype=torch.int32), z(E, dtype=torch.float32), z(2, dtype=torch.float32)
        self.offsets, self.row_of, self.tok = z(E + 1, dtype=torch.int32), z(T, k, dtype=torch.int32), z(R, dtype=torch.int32)
        self.idx = z(T, k, dtype=torch.int32)

    def route(self):
        """(Not capturable: the permutation looks its scratch up.)"""
        self.idx.copy_(self.logits.topk(self.k, 1).indices)
        self.lm.lmoe_permute_noalloc(self.idx, self.E, self.offsets, self.row_of, self.tok)

    def backward(self, accumulate):
        lm, o = self.lm, dict(offsets=self.offsets, status=self.status)
        lm.lmoe_router_losses(self.logits, self.idx, self.counts, self.mean, self.losses, self.lws)
        self.xr = self.x[self.tok.long()]
        lm.lmoe_gated_ffn(self.xr, self.wg, self.wu, self.h, self.gate, self.up, **o)
        lm.lmoe_matmul_bf16(self.h, self.wd, self.y, **o)
        lm.lmoe_gated_ffn_grad(self.dy, self.wd, self.gate, self.up, self.dgate, self.dup, **o)
        lm.lmoe_matmul_bf16(self.dgate, self.wg, self.dx, a2=self.dup, w2=self.wu, transposed=True, **o)
        lm.lmoe_matmul_bf16_wgrad(self.dgate, self.xr, self.grads[0], dy2=self.dup, dw2=self.grads[1], accumulate=accumulate, **o)
        lm.lmoe_matmul_bf16_wgrad(self.dy, self.h, self.grads[2], accumulate=accumulate, **o)
        lm.lmoe_router_grad(self.logits, self.idx, self.counts, self.grads[3], self.gw, self.gl)

    def __call__(self, accumulate=False):
        self.backward(accumulate)
        self.lm.lmoe_clip_grad_norm(self.grads, self.norm, 1e-2, self.ws, out=self.clipped)

    def outputs(self):
        return [self.h, self.gate, self.up, self.y, self.dgate, self.dup, self.dx, *self.grads, self.norm, *self.clipped]


def check(s, start=None):
    off, E = s.offsets, s.E
    assert int(s.status) == 0
    assert torch.equal(s.counts[:E].cumsum(0), off[1:].long())
    for got, (v, tol), name in zip((s.h, s.gate, s.up), xu.gated(s.xr, s.wg, s.wu, off), ("h", "gate", "up")):
        close(got, v, tol, name)
    v, tol = xu.product(s.h, s.wd, off)
    close(s.y, v, xu.rounded(v, tol, BF16), "y")
    for got, (v, tol), name in zip((s.dgate, s.dup), xu.gated_grad(s.dy, s.wd, s.gate, s.up, off), ("dgate", "dup")):
        close(got, v, tol, name)
    (v, tol), (v2, tol2) = xu.product(s.dgate, s.wg, off, True), xu.product(s.dup, s.wu, off, True)
    # (one sum of twice as many products)
    close(s.dx, v + v2, xu.rounded(v + v2, 2 * (tol + tol2), BF16), "dx")
    for i, (dy, x) in enumerate(((s.dgate, s.xr), (s.dup, s.xr), (s.dy, s.h))):
        v, tol = xu.wgrad(dy, x, E, off, None if start is None else start[i])
        close(s.grads[i], v, xu.rounded(v, tol, torch.float32), f"dw{i}")
    want = xu.norm(s.grads)
    assert abs(float(s.norm) - float(want)) <= 34 * 2.0 ** -24 * float(want)
    for got, g in zip(s.clipped, s.grads):
        v, tol = xu.clipped(g, s.norm, 1e-2)
        close(got, v, tol, "clipped")


SIZES = [(64, 16, 2, 256, 512), (1, 8, 2, 256, 128), (37, 5, 3, 136, 200), (600, 4, 2, 512, 264), (2000, 40, 4, 128, 136)]


@pytest.mark.parametrize("T,E,k,L,I", SIZES)
def test_a_training_step(lm, T, E, k, L, I):
    s = Step(lm, T, E, k, L, I)
    s.route()
    s()
    check(s)
    start = [g.clone() for g in s.grads]
    s(accumulate=True)
    check(s, start)


@pytest.mark.parametrize("T,E,k,L,I", SIZES[:4])
def test_the_same_step_in_a_graph(lm, T, E, k, L, I):
    s = Step(lm, T, E, k, L, I)
    s.route()
    s()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s()
    g = torch.Generator(device="cuda").manual_seed(9)
    for _ in range(2):
        s.x.copy_(torch.randn(T, L, generator=g, device="cuda"))
        s.logits.copy_(torch.randn(T, E, generator=g, device="cuda"))
        s.dy.copy_(torch.randn(s.R, L, generator=g, device="cuda") * 1e-2)
        s.route()
        graph.replay()
        got = [t.clone() for t in s.outputs()]
        for t in s.outputs():
            t.zero_()
        s()
        for a, b in zip(got, s.outputs()):
            assert torch.equal(a, b)
        check(s)


def test_gradients_are_those_of_the_chain(lm):
    """Against automatic differentiation in 64 bits of y = down(silu(gate x) * up x): each stage rounds to bf16 once, 2^-8 of
    its result, and a gradient is a sum over stages' results, so in the 2-norm it is off by a few 2^-8 (six roundings:
    gate, up, h, dgate and dup, and its own)."""
    s = Step(lm, 300, 6, 2, 256, 384)
    s.route()
    s()
    leaves = [t.double().requires_grad_(True) for t in (s.xr, s.wg, s.wu, s.wd)]
    x, wg, wu, wd = leaves
    loss = 0
    for e, (lo, hi) in enumerate(xu.groups(s.offsets, s.R, s.E)):
        g, u = x[lo:hi] @ wg[e].t(), x[lo:hi] @ wu[e].t()
        loss = loss + ((g * torch.sigmoid(g) * u) @ wd[e].t() * s.dy[lo:hi].double()).sum()
    want = torch.autograd.grad(loss, leaves)
    for got, w in zip((s.dx, *s.grads[:3]), want):
        assert float((got.double() - w).norm()) <= 6 * 2.0 ** -8 * float(w.norm())
