"""Backward pass and adapters against plain 64-bit forms.

Two kinds of inputs.  "Whole" inputs are small integers and powers of two for
which every product and every partial sum is exact in fp32 (also when a
factor is split into two bf16 parts of 8 bits each), so the result has to be
the exact value rounded once to the output's type: compared bit for bit.
"Drawn" inputs are normal; there an output may be off by half a step of its
type plus the error bound of an fp32 sum of n terms, in any order and with
each addition off by at most a step (2^-23 of the sum of the terms'
magnitudes S): n 2^-23 S; a factor split into two bf16 parts is off by at most
2^-17 of itself (half a step of 8 bits, twice).
"""
import pytest
import torch

from ternary_weight_linear_04_b200 import bitlinear as bl
from ternary_weight_linear_04_b200 import build as libbuild

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert bl.device_error() == 0


class Case:
    """Inputs of one layer and their 64-bit values."""

    def __init__(self, M, K, N, L=2, r=4, whole=True, seed=0, dy_dtype=BF, order="mixed"):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed * 1000003 + M * 7919 + K * 31 + N)
        ri = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda")  # noqa: E731
        rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.M, self.K, self.N, self.L, self.r = M, K, N, L, r
        self.t = ri(-1, 1, N, K)
        self.packed = pack(self.t)
        if whole:
            self.gamma = torch.full((1,), 0.125, device="cuda")
            self.xq = ri(-2, 2, M, K).to(torch.int8)
            self.eta = 127 * torch.exp2(ri(-2, 2, M).float())
            self.dy = ri(-4, 4, M, N).to(dy_dtype)
            self.A = (ri(-1, 1, L, r, K) * (ri(0, 3, L, r, K) == 0)).to(BF)
            self.B = (ri(-2, 2, L, N, r) * (ri(0, 3, L, N, r) == 0)).to(BF)
            self.scale = torch.exp2(ri(-1, 1, L).float())
        else:
            self.gamma = torch.rand(1, generator=g, device="cuda") * 0.02 + 0.01
            self.xq = (rn(M, K) * 30).round().clamp(-127, 127).to(torch.int8)
            self.eta = torch.rand(M, generator=g, device="cuda") * 4 + 0.5
            self.dy = (rn(M, N) * 0.01).to(dy_dtype)
            self.A = (rn(L, r, K) / K ** 0.5).to(BF)
            self.B = (rn(L, N, r) * 0.1).to(BF)
            self.scale = torch.rand(L, generator=g, device="cuda") + 0.5
        self.xsum = self.xq.sum(1, dtype=torch.int32)
        self.ids = ri(-1, L - 1, M).to(torch.int32)
        if order == "packed":
            self.ids = self.ids.sort()[0]

    # 64-bit values, and beside each the sum of its terms' magnitudes
    @property
    def xh(self):
        return self.xq.to(F64) * (self.eta.to(F64) / 127)[:, None]

    @property
    def W(self):
        return self.t.to(F64) * self.gamma.to(F64)

    def dx(self):
        dy = self.dy.to(F64)
        return dy @ self.W, dy.abs() @ self.W.abs()

    def dw(self):
        dy = self.dy.to(F64)
        return dy.t() @ self.xh, dy.t().abs() @ self.xh.abs()

    def per_adapter(self):
        for a in range(self.L):
            yield a, (self.ids == a).nonzero()[:, 0], self.A[a].to(F64), self.B[a].to(F64), float(self.scale[a])

    def y(self):
        xh = self.xh
        y, S = xh @ self.W.t(), xh.abs() @ self.W.t().abs()
        for a, of, A, B, s in self.per_adapter():
            y[of] += s * (xh[of] @ A.t()) @ B.t()
            S[of] += s * (xh[of].abs() @ A.t().abs()) @ B.t().abs()
        return y, S

    def adapters_grad(self):
        xh, dy = self.xh, self.dy.to(F64)
        dx, Sx = self.dx()
        dA, dB = torch.zeros_like(self.A, dtype=F64), torch.zeros_like(self.B, dtype=F64)
        SA, SB = dA.clone(), dB.clone()
        for a, of, A, B, s in self.per_adapter():
            v, Sv = s * dy[of] @ B, s * dy[of].abs() @ B.abs()
            dx[of] += v @ A
            Sx[of] += Sv @ A.abs()
            dA[a], SA[a] = v.t() @ xh[of], Sv.t() @ xh[of].abs()
            dB[a] = s * dy[of].t() @ (xh[of] @ A.t())
            SB[a] = s * dy[of].t().abs() @ (xh[of].abs() @ A.t().abs())
        return (dx, Sx), (dA, SA), (dB, SB)


def pack(t):
    N, K = t.shape
    c = torch.ones(N, (K + 3) // 4 * 4, dtype=torch.int32, device=t.device)
    c[:, :K] = t.to(torch.int32) + 1
    c = c.view(N, -1, 4)
    return (c[..., 0] | c[..., 1] << 2 | c[..., 2] << 4 | c[..., 3] << 6).to(torch.uint8)


def same(got, want):
    """Bit for bit the exact value rounded once (fp64 -> fp32 is exact for whole inputs)."""
    w = want[0] if isinstance(want, tuple) else want
    assert torch.equal(w, w.to(F32).to(F64)), "the case's values are not exact in fp32"
    assert torch.equal(got, w.to(F32).to(got.dtype))


def near(got, want, n, split=0):
    """Within half a step of the type, plus an fp32 sum of n terms, plus `split` factors in two bf16 parts."""
    val, S = want
    bound = torch.finfo(got.dtype).eps / 2 * val.abs() * (1 + 2 ** -7) + ((n + 8) * 2 ** -23 + split * 2 ** -17) * S + 1e-38
    off = (got.to(F64) - val).abs()
    assert (off <= bound).all(), float((off / bound).max())


SIZES = [(1, 1, 1), (1, 64, 64), (2, 3, 5), (5, 130, 63), (17, 64, 128), (33, 200, 257), (64, 256, 192),
         (128, 320, 64), (129, 511, 129), (200, 1000, 72), (256, 512, 264), (257, 1024, 520), (300, 77, 1001),
         (515, 640, 640)]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_grad_input_whole(M, K, N, dt, out):
    c = Case(M, K, N, dy_dtype=dt)
    same(bl.grad_input(c.dy, c.packed, c.gamma, K, out_dtype=out), c.dx())


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K,N", [(1, 3200, 640), (7, 100, 2000), (130, 1024, 1000), (300, 513, 4100)])
def test_grad_input_drawn(M, K, N, dt, out):
    c = Case(M, K, N, whole=False, dy_dtype=dt)
    near(bl.grad_input(c.dy, c.packed, c.gamma, K, out_dtype=out), c.dx(), N)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_grad_weight_whole(M, K, N, dt, out):
    c = Case(M, K, N, dy_dtype=dt)
    same(bl.grad_weight(c.dy, c.xq, c.eta, out_dtype=out), c.dw())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K,N", [(1, 320, 640), (7, 100, 200), (130, 1024, 1000), (2500, 130, 72), (4100, 64, 513)])
def test_grad_weight_drawn(M, K, N, dt):
    c = Case(M, K, N, whole=False, dy_dtype=dt)
    near(bl.grad_weight(c.dy, c.xq, c.eta), c.dw(), M, split=1)
    # bf16 results: the tokens' values are rounded to bf16 before the product, half a step (2^-8) at most
    near(bl.grad_weight(c.dy, c.xq, c.eta, out_dtype=BF), c.dw(), M, split=2 ** 9 + 1)


def test_gradients_of_no_tokens():
    c = Case(0, 96, 40)
    assert bl.grad_input(c.dy, c.packed, c.gamma, 96).shape == (0, 96)
    dw = bl.grad_weight(c.dy, c.xq, c.eta, out=torch.full((40, 96), 7.0, device="cuda"))
    assert not dw.any()
    dx, dA, dB = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids)
    assert dx.shape == (0, 96) and not dA.any() and not dB.any() and dA.shape == c.A.shape
    assert bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, 40, c.A, c.B, c.scale, c.ids).shape == (0, 40)
    assert bl.rmsnorm_grad(torch.empty(0, 96, device="cuda"), c.xq, c.eta, c.eta).shape == (0, 96)


ADAPTED = [(1, 1, 1, 1, 1), (1, 64, 64, 1, 8), (1, 3200, 640, 8, 16), (2, 65, 5, 3, 2), (3, 640, 128, 40, 128),
           (9, 256, 130, 5, 33), (16, 1024, 512, 16, 16), (17, 333, 100, 4, 7), (64, 512, 256, 64, 32),
           (130, 192, 257, 3, 5), (256, 512, 264, 7, 24), (300, 640, 200, 2, 64), (515, 128, 384, 9, 16),
           (257, 100, 1000, 300, 3)]


@pytest.mark.parametrize("order", ["mixed", "packed"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,K,N,L,r", ADAPTED)
def test_forward_adapters_whole(M, K, N, L, r, out, order):
    c = Case(M, K, N, L, r, order=order)
    same(bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, N, c.A, c.B, c.scale, c.ids, out_dtype=out), c.y())


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,K,N,L,r", [(1, 3200, 640, 4, 16), (16, 1000, 300, 8, 64), (300, 640, 260, 3, 16)])
def test_forward_adapters_drawn(M, K, N, L, r, out):
    c = Case(M, K, N, L, r, whole=False)
    y = bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, N, c.A, c.B, c.scale, c.ids, out_dtype=out)
    near(y, c.y(), K + r, split=1)


@pytest.mark.parametrize("order", ["mixed", "packed"])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K,N,L,r", ADAPTED)
def test_adapters_grad_whole(M, K, N, L, r, dt, order):
    c = Case(M, K, N, L, r, dy_dtype=dt, order=order)
    dx, dA, dB = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, grad_dtype=F32)
    want = c.adapters_grad()
    same(dx, want[0])
    same(dA, want[1])
    same(dB, want[2])


@pytest.mark.parametrize("grad", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K,N,L,r", [(1, 320, 640, 4, 16), (48, 1000, 300, 8, 64), (700, 640, 264, 3, 16)])
def test_adapters_grad_drawn(M, K, N, L, r, dt, grad):
    c = Case(M, K, N, L, r, whole=False, dy_dtype=dt)
    dx, dA, dB = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, out_dtype=F32,
                                  grad_dtype=grad)
    want = c.adapters_grad()
    near(dx, want[0], N + r, split=1)
    near(dA, want[1], M + N, split=1)
    near(dB, want[2], M + K, split=1)


def test_adapters_grad_parts():
    c = Case(70, 256, 136, 3, 8)
    args = (c.dy, c.xq, c.eta)
    ad = (c.A, c.B, c.scale, c.ids)
    dx, dA, dB = bl.adapters_grad(*args, c.packed, c.gamma, *ad)
    x2, a2, b2 = bl.adapters_grad(*args, c.packed, c.gamma, *ad, want_dab=False)
    assert a2 is None and b2 is None and torch.equal(x2, dx)
    x3, a3, b3 = bl.adapters_grad(*args, None, None, *ad, want_dx=False)
    assert x3 is None and torch.equal(a3, dA) and torch.equal(b3, dB)


@pytest.mark.parametrize("ids", ["none", "out of range", "one for all"])
def test_adapter_ids(ids):
    c = Case(70, 256, 136, 3, 8)
    c.ids[:] = {"none": -1, "out of range": 3, "one for all": 1}[ids]
    if ids == "out of range":
        c.ids[::2] = -2 ** 31
        c.ids[1::2] = 2 ** 31 - 1
        c.ids[::5] = 3
    y = bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, 136, c.A, c.B, c.scale, c.ids)
    same(y, c.y())
    if ids != "one for all":
        assert torch.equal(y, bl.forward(c.xq, c.eta, c.xsum, c.packed, c.gamma, 136))
    dx, dA, dB = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids)
    want = c.adapters_grad()
    same(dx, want[0])
    assert torch.equal(dA, want[1][0].to(F32).to(BF)) and torch.equal(dB, want[2][0].to(F32).to(BF))


def norm_case(M, K, dt=BF, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + M * 131 + K)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF)
    dn = (torch.randn(M, K, generator=g, device="cuda") * 0.01).to(dt)
    return x, dn


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 7), (2, 64), (3, 1000), (5, 3200), (17, 4096), (300, 520), (2, 8640),
                                 (1, 60001), (2, 65536)])
def test_rmsnorm_grad(M, K, dt, out):
    x, dn = norm_case(M, K, dt)
    xq, eta, xsum, rstd = bl.rmsnorm_quant_act(x, want_rstd=True)
    for a, b in zip((xq, eta, xsum), bl.rmsnorm_quant_act(x)):
        assert torch.equal(a, b)
    r = 1 / torch.sqrt(x.to(F64).square().mean(1) + 1e-6)
    assert ((rstd.to(F64) - r).abs() <= 4 * 2 ** -24 * r).all()  # four fp32 roundings
    dx = bl.rmsnorm_grad(dn, xq, eta, rstd, out_dtype=out)
    n = xq.to(F64) * (eta.to(F64) / 127)[:, None]
    p, S = (n * dn.to(F64)).mean(1, keepdim=True), (n * dn.to(F64)).abs().mean(1, keepdim=True)
    want = rstd.to(F64)[:, None] * (dn.to(F64) - n * p)
    # the sum over K (K 2^-23 of S), then a handful of fp32 roundings of each term
    size = rstd.to(F64)[:, None] * (dn.to(F64).abs() + n.abs() * S * (1 + K / 8))
    near(dx, (want, size), 0)


def test_rmsnorm_grad_in_place_and_misaligned():
    x, dn = norm_case(9, 1001)
    xq, eta, _, rstd = bl.rmsnorm_quant_act(x, want_rstd=True)
    want = bl.rmsnorm_grad(dn, xq, eta, rstd)
    part = bl.rmsnorm_grad(dn[1:], xq[1:], eta[1:], rstd[1:])  # rows that start on odd addresses
    assert torch.equal(part, want[1:])
    bl.rmsnorm_grad(dn, xq, eta, rstd, out=dn)
    assert torch.equal(dn, want)


def test_rows_behind_the_last_token_stay_as_they_were():
    c = Case(33, 200, 72, 3, 8)
    for make, rows, cols in [(lambda o: bl.grad_input(c.dy, c.packed, c.gamma, 200, out=o), 33, 200),
                             (lambda o: bl.grad_weight(c.dy, c.xq, c.eta, out=o), 72, 200),
                             (lambda o: bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, 72, c.A, c.B,
                                                            c.scale, c.ids, out=o), 33, 72)]:
        big = torch.full((rows * cols + 4096,), 5.0, device="cuda", dtype=BF)
        make(big[:rows * cols].view(rows, cols))
        assert (big[rows * cols:] == 5).all() and not (big[:rows * cols] == 5).all()


def test_another_stream_and_a_captured_graph():
    c = Case(70, 256, 136, 3, 8)

    def step(stream=None):
        y = bl.linear_adapters(c.x, c.packed, c.gamma, 136, c.A, c.B, c.scale, c.ids, stream=stream)
        return (y, *bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, stream=stream),
                bl.grad_weight(c.dy, c.xq, c.eta, stream=stream), bl.grad_input(c.dy, c.packed, c.gamma, 256, stream=stream))

    c.x = torch.randn(70, 256, device="cuda").to(BF)
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(2):
        for t in held:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)
    c.ids.fill_(-1)  # a replay reads the ids as they are then
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], bl.linear(c.x, c.packed, c.gamma, 136))
    assert not held[2].any() and not held[3].any()


def test_a_training_step_by_differences():
    """The gradients of a loss through linear + adapters against central differences of the 64-bit function."""
    c = Case(6, 24, 10, 2, 3, whole=False)
    c.dy = torch.randn(6, 10, device="cuda").to(BF)
    dx, dA, dB = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, out_dtype=F32,
                                  grad_dtype=F32)
    dw = bl.grad_weight(c.dy, c.xq, c.eta)
    dy = c.dy.to(F64)

    def loss(xh, W, A, B):
        y = xh @ W.t()
        for a in range(c.L):
            of = c.ids == a
            y = y + of[:, None] * float(c.scale[a]) * (xh @ A[a].t()) @ B[a].t()
        return float((dy * y).sum())

    at = [c.xh, c.W, c.A.to(F64), c.B.to(F64)]
    for i, grad in enumerate((dx, dw, dA, dB)):
        for j in range(0, at[i].numel(), max(1, at[i].numel() // 17)):
            hi, lo = [t.clone() for t in at], [t.clone() for t in at]
            hi[i].view(-1)[j] += 1e-3
            lo[i].view(-1)[j] -= 1e-3
            diff = (loss(*hi) - loss(*lo)) / 2e-3  # the loss is linear in each: exact but for rounding
            assert abs(diff - float(grad.reshape(-1)[j])) <= 1e-5 * (1 + abs(diff))
