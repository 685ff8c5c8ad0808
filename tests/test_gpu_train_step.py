"""The operators together, as a training step of routed 8-bit experts uses them: routing and its
losses, rows into 8 bits in expert order, gate/up and down products, their input and weight
gradients, and the router's gradient; eager and captured into a graph.

Every stage is compared, in 64 bits, with the plain operation on the stage's own unquantised inputs.
An operand's value is off by at most half a step of its 8-bit type, h |v| + t s (h 2^-4 or 2^-3, t half
the smallest step, s its block's scale), so a sum of products by at most the sum of |x| ew + |w| ex +
ex ew, plus the fp32 sum's own bound."""
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


class Step:
    """Experts y = down(silu(gate x) * up x), weights in 8 bits; buffers kept from step to step."""

    def __init__(self, lm, T, E, k, D, I, dtype, pow2):
        self.lm, self.T, self.E, self.k, self.D, self.I, self.dtype, self.pow2 = lm, T, E, k, D, I, dtype, pow2
        self.R = T * k
        self.Rp = lm.lmoe_fp8_padded_rows(self.R, E)
        g = torch.Generator(device="cuda").manual_seed(T + E)
        new = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.x, self.logits = new(T, D).to(dtype), 1.5 * new(T, E)
        self.w1, self.w2 = new(E, 2 * I, D).to(dtype) * D ** -0.5, new(E, D, I).to(dtype) * I ** -0.5
        self.dy, self.gw, self.gl = (1e-3 * new(self.R, D)).to(dtype), new(T, k), torch.tensor([0.01, 0.001], device="cuda")
        self.mask = (torch.rand(T, generator=g, device="cuda") > 0.1).to(torch.uint8)
        self.b = {}

    def buf(self, name, shape, dtype=torch.float32):
        if name not in self.b:
            self.b[name] = torch.zeros(shape, dtype=torch.uint8, device="cuda").view(dtype) if dtype in tu.MAXIMUM \
                else torch.zeros(shape, dtype=dtype, device="cuda")
        return self.b[name]

    def rows(self, name, src, fmt, index=None):
        K = src.shape[1]
        q, s = self.buf(name, (self.R, K), fmt), self.buf(name + "_s", (-(-K // 128), self.R))
        self.lm.lmoe_quantize_fp8_rows(src, q, s, index, self.pow2)
        return q, s

    def cols(self, name, src, fmt, index=None):
        K = src.shape[1]
        q, s = self.buf(name, (K, self.Rp), fmt), self.buf(name + "_s", (self.Rp // 128, K))
        self.lm.lmoe_quantize_fp8_cols(src, q, s, self.offsets, index, self.pow2)
        return q, s

    def weight(self, name, src):
        E, N, K = src.shape
        c = [self.buf(name, (E, N, K), E4M3), self.buf(name + "_s", (E, -(-N // 128), -(-K // 128))),
             self.buf(name + "_t", (E, K, N), E4M3), self.buf(name + "_ts", (E, -(-K // 128), -(-N // 128)))]
        self.lm.lmoe_quantize_fp8_weight(src, *c, self.pow2)
        return c

    def route(self):
        """The experts of each token and their rows in expert order (not capturable: it looks its scratch up)."""
        E, k, R, i32 = self.E, self.k, self.R, torch.int32
        self.idx = self.buf("idx", (self.T, k), i32)
        self.idx.copy_(self.logits.topk(k, 1).indices)
        self.offsets, row_of, self.tok = self.buf("off", (E + 1,), i32), self.buf("rof", (self.T, k), i32), self.buf("tok", (R,), i32)
        self.lm.lmoe_permute_noalloc(self.idx, E, self.offsets, row_of, self.tok)

    def __call__(self):
        lm, E, k, I, D, R = self.lm, self.E, self.k, self.I, self.D, self.R
        i32 = torch.int32
        self.counts, self.mean, self.losses = self.buf("counts", (E + 1,), i32), self.buf("mean", (E,)), self.buf("loss", (2,))
        ws = self.buf("ws", (lm.lmoe_router_losses_workspace_size(self.T, E),), torch.uint8)
        lm.lmoe_router_losses(self.logits, self.idx, self.counts, self.mean, self.losses, ws, row_mask=self.mask)
        status = self.buf("status", (1,), i32)
        w1, w1s, w1t, w1ts = self.weight("w1q", self.w1)
        w2, w2s, w2t, w2ts = self.weight("w2q", self.w2)
        o = dict(offsets=self.offsets, status=status)
        # forward
        self.h = self.buf("h", (R, 2 * I), self.dtype)
        lm.lmoe_matmul_fp8(*self.rows("xq", self.x, E4M3, self.tok), w1, w1s, self.h, **o)
        gate, up = self.h.float().chunk(2, 1)
        sg = torch.sigmoid(gate)
        self.act = self.buf("act", (R, I), self.dtype)
        self.act.copy_(gate * sg * up)
        self.y = self.buf("y", (R, D), self.dtype)
        lm.lmoe_matmul_fp8(*self.rows("aq", self.act, E4M3), w2, w2s, self.y, **o)
        # backward
        self.da = self.buf("da", (R, I), self.dtype)
        lm.lmoe_matmul_fp8(*self.rows("dyq", self.dy, E5M2), w2t, w2ts, self.da, **o)
        self.dh = self.buf("dh", (R, 2 * I), self.dtype)
        self.dh[:, :I].copy_(self.da.float() * up * sg * (1 + gate * (1 - sg)))
        self.dh[:, I:].copy_(self.da.float() * gate * sg)
        self.dx = self.buf("dx", (R, D), self.dtype)
        lm.lmoe_matmul_fp8(*self.rows("dhq", self.dh, E5M2), w1t, w1ts, self.dx, **o)
        self.dw1, self.dw2 = self.buf("dw1", self.w1.shape), self.buf("dw2", self.w2.shape)
        lm.lmoe_matmul_fp8_wgrad(*self.cols("dhc", self.dh, E5M2), *self.cols("xc", self.x, E4M3, self.tok), self.dw1, **o)
        lm.lmoe_matmul_fp8_wgrad(*self.cols("dyc", self.dy, E5M2), *self.cols("ac", self.act, E4M3), self.dw2, **o)
        self.dl = self.buf("dl", (self.T, E))
        lm.lmoe_router_grad(self.logits, self.idx, self.counts, self.dl, self.gw, self.gl, row_mask=self.mask)
        self.status = status

    def outputs(self):
        return [self.losses, self.mean, self.counts, self.h, self.act, self.y, self.da, self.dh, self.dx, self.dw1,
                self.dw2, self.dl]


def off_by(v, fmt, dim, square=False):
    """Bound of a value's quantisation error, blocks along ``dim`` (square: 128 x 128 of a matrix)."""
    if v.numel() == 0:
        return v
    a = v.abs()
    b = tu.blocks(a, dim)
    if square:
        b = tu.blocks(tu.blocks(a, 1), 0)
        s = b.amax((1, 3), keepdim=True).expand(b.shape).flatten(2).flatten(0, 1)[:v.shape[0], :v.shape[1]]
    else:
        s = b.amax(dim + 1, keepdim=True).expand(b.shape).flatten(dim, dim + 1).narrow(dim, 0, v.shape[dim])
    # the scale itself may be twice as large when it is a power of two
    return tu.HALF[fmt] * a + 2 * s / tu.MAXIMUM[fmt] * (2.0 ** -10 if fmt == E4M3 else 2.0 ** -17)


def check_product(got, p, ep, q, eq, what):
    want, tol = tu.product(p, q)
    tol = tol + (p.abs() @ eq.t() + ep @ q.abs().t() + ep @ eq.t()) * (1 + 1e-4)
    assert_close(got, want, tol + tu.HALF[got.dtype] * (want.abs() + tol), what)


@pytest.mark.parametrize("T,E,k,D,I,dtype,pow2", [
    (1, 8, 2, 256, 128, torch.bfloat16, False), (50, 4, 2, 144, 208, torch.float32, True),
    (300, 8, 2, 272, 144, torch.bfloat16, False), (900, 3, 2, 512, 400, torch.bfloat16, True),
    (64, 100, 5, 128, 128, torch.float32, False)])
def test_training_step(lm, T, E, k, D, I, dtype, pow2):
    s = Step(lm, T, E, k, D, I, dtype, pow2)
    s.route()
    s()
    torch.cuda.synchronize()
    assert int(s.status) == 0
    loss, mean, counts = tu.router_losses(s.logits, s.idx, None, s.mask)
    assert torch.equal(s.counts.long(), counts)
    assert_close(s.losses, loss, loss * 1e-4)   # (bounds of the losses by themselves are tested elsewhere)
    d, tol = tu.router_grad(s.logits, s.idx, s.counts, s.gw, s.gl, None, s.mask)
    assert_close(s.dl, d, tol)
    x = s.x.double()[s.tok.long()]
    act, dy, dh = s.act.double(), s.dy.double(), s.dh.double()
    off = s.offsets.tolist()
    assert off[0] == 0 and off[-1] == s.R
    for e in range(E):
        r = slice(off[e], off[e + 1])
        w1, w2 = s.w1[e].double(), s.w2[e].double()
        e1, e2 = off_by(w1, E4M3, 1, True), off_by(w2, E4M3, 1, True)
        if off[e + 1] > off[e]:
            check_product(s.h[r], x[r], off_by(x[r], E4M3, 1), w1, e1, "gate/up")
            check_product(s.y[r], act[r], off_by(act[r], E4M3, 1), w2, e2, "down")
            check_product(s.da[r], dy[r], off_by(dy[r], E5M2, 1), w2.t(), e2.t(), "input gradient of down")
            check_product(s.dx[r], dh[r], off_by(dh[r], E5M2, 1), w1.t(), e1.t(), "input gradient of gate/up")
        xt, at, yt, ht = x[r].t(), act[r].t(), dy[r].t(), dh[r].t()
        check_product(s.dw1[e], ht, off_by(ht, E5M2, 1), xt, off_by(xt, E4M3, 1), "weight gradient of gate/up")
        check_product(s.dw2[e], yt, off_by(yt, E5M2, 1), at, off_by(at, E4M3, 1), "weight gradient of down")


def test_training_step_captured(lm):
    s = Step(lm, 200, 6, 2, 256, 144, torch.bfloat16, False)
    s.route()
    s()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s()
    for seed in (1, 2):   # other inputs, another routing
        g = torch.Generator(device="cuda").manual_seed(seed)
        s.x.copy_(torch.randn(s.x.shape, generator=g, device="cuda"))
        s.logits.copy_(torch.randn(s.logits.shape, generator=g, device="cuda"))
        s.route()
        s()
        want = [t.clone() for t in s.outputs()]
        for t in s.outputs():
            t.fill_(3)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, s.outputs()))


def test_product_gradients_against_differences(lm):
    # y = x w^T is linear: with operands and steps that 8 bits hold exactly (small integers, scales of one),
    # differences of sum(y gy) are the gradients exactly
    R, N, K = 140, 144, 160
    g = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float()
    x, w, gy = new(R, K), new(N, K), new(R, N)
    one = lambda *s: torch.ones(*s, device="cuda")

    def value(x, w):
        y = torch.zeros(R, N, device="cuda")
        lm.lmoe_matmul_fp8(x.to(E4M3), one(2, R), w.to(E4M3), one(2, 2), y)
        return float((y.double() * gy.double()).sum())
    dx = torch.zeros(R, K, device="cuda")
    lm.lmoe_matmul_fp8(gy.to(E5M2), one(2, R), w.t().contiguous().to(E4M3), one(2, 2), dx)
    P = lm.lmoe_fp8_padded_rows(R, 1)
    pad = lambda v: torch.nn.functional.pad(v, (0, 0, 0, P - R)).t().contiguous()
    dw = torch.zeros(N, K, device="cuda")
    lm.lmoe_matmul_fp8_wgrad(pad(gy).to(E5M2), one(P // 128, N), pad(x).to(E4M3), one(P // 128, K), dw)
    for r, c in ((0, 0), (R - 1, K - 1), (70, 130), (128, 5)):
        hi, lo = x.clone(), x.clone()
        hi[r, c] += 1
        lo[r, c] -= 1
        assert float(dx[r, c]) == (value(hi, w) - value(lo, w)) / 2
    for n, c in ((0, 0), (N - 1, K - 1), (129, 3), (7, 140)):
        hi, lo = w.clone(), w.clone()
        hi[n, c] += 1
        lo[n, c] -= 1
        assert float(dw[n, c]) == (value(x, hi) - value(x, lo)) / 2
