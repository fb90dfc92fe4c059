"""Adapters and gradients where they can go wrong: factors of other adapters
that are not finite, more shapes of the adapter operators, splits over
clusters.  Inputs, 64-bit forms and tolerances as in test_gpu_train.py."""
import pytest
import torch

from ternary_weight_linear_04_b200 import bitlinear as bl
from ternary_weight_linear_04_b200 import build as libbuild
from test_gpu_train import BF, F32, F64, Case, near, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert bl.device_error() == 0


def forward(c, out, A=None, B=None):
    return bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, c.N, c.A if A is None else A,
                               c.B if B is None else B, c.scale, c.ids, out_dtype=out)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,K,N,r", [(3, 256, 96, 8), (12, 256, 96, 5), (40, 200, 130, 8), (70, 256, 136, 3),
                                     (300, 320, 264, 16), (600, 128, 96, 40)])
def test_a_factor_that_is_not_finite_stays_with_its_tokens(M, K, N, r, out, bad):
    c = Case(M, K, N, 3, r)
    c.ids[:3] = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")[:M]
    others = c.ids != 1
    y = forward(c, out)
    args = lambda A, B: (c.dy, c.xq, c.eta, c.packed, c.gamma, A, B, c.scale, c.ids)  # noqa: E731
    grads = bl.adapters_grad(*args(c.A, c.B), out_dtype=out, grad_dtype=out)
    for which in "AB":
        A, B = c.A.clone(), c.B.clone()
        t = A if which == "A" else B
        t[1].view(-1)[::7] = bad
        got = forward(c, out, A, B)
        assert torch.equal(got[others], y[others])
        assert not got[~others].isfinite().all()
        dx, dA, dB = bl.adapters_grad(*args(A, B), out_dtype=out, grad_dtype=out)
        assert torch.equal(dx[others], grads[0][others])
        assert not dx[~others].isfinite().all()
        for a in (0, 2):
            assert torch.equal(dA[a], grads[1][a]) and torch.equal(dB[a], grads[2][a])


def test_values_beside_one_that_is_not_finite():
    """dx of the adapter's own tokens: infinite where the infinity is, exact elsewhere."""
    c = Case(40, 256, 64, 2, 4)
    c.B.clamp_(min=1)  # v is not zero where dy's row does not cancel
    c.dy.abs_()
    c.dy[:, 0] = 1
    want = c.adapters_grad()[0][0]
    c.A[1, 2, 100] = float("inf")
    dx = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, out_dtype=F32,
                          want_dab=False)[0]
    own = c.ids == 1
    assert (dx[own, 100] == float("inf")).all()
    keep = torch.ones_like(dx, dtype=torch.bool)
    keep[own, 100] = False
    assert torch.equal(dx[keep], want.to(F32)[keep])


@pytest.mark.parametrize("order", ["mixed", "packed"])
@pytest.mark.parametrize("M,K,N,L,r", [(1, 16, 8, 1, 128), (16, 8, 100, 2, 127), (15, 16384, 33, 3, 9), (4, 16392, 70, 2, 3),
                                       (513, 192, 200, 2, 32), (700, 66, 129, 33, 65), (1030, 256, 64, 1, 1),
                                       (2100, 64, 72, 5, 20), (4500, 40, 24, 2, 8)])
def test_adapter_shapes(M, K, N, L, r, order):
    c = Case(M, K, N, L, r, order=order)
    same(forward(c, F32), c.y())
    got = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, out_dtype=F32, grad_dtype=F32)
    for g, w in zip(got, c.adapters_grad()):
        same(g, w)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K,N", [(1, 64, 8640), (77, 2048, 3200), (100, 1500, 5000), (128, 256, 16384), (129, 256, 9000),
                                   (333, 1000, 4097), (200, 8640, 700)])
def test_grad_input_split(M, K, N, dt):
    c = Case(M, K, N, dy_dtype=dt)
    same(bl.grad_input(c.dy, c.packed, c.gamma, K, out_dtype=F32), c.dx())


@pytest.mark.parametrize("M", [1, 2, 5, 16, 17, 200])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("K", [320, 333])
def test_linear_adapters_is_quantiser_and_forward(M, K, norm, dt):
    """The one call and its parts: the same tokens, so the same results but for the order of the adapter's sums."""
    if norm and dt == F32:
        pytest.skip("the normalisation takes bf16")
    c = Case(M, K, 200, 3, 8, whole=False)
    x = torch.randn(M, K, device="cuda").to(dt)
    x[:, 0] = 0.5
    if M > 2:
        x[2] = 0  # eta at its floor
    c.xq, c.eta, c.xsum = (bl.rmsnorm_quant_act if norm else bl.quant_act)(x)
    for out in (BF, F32):
        y = bl.linear_adapters(x, c.packed, c.gamma, 200, c.A, c.B, c.scale, c.ids, out_dtype=out, rmsnorm=norm)
        near(y, c.y(), K + 8, split=1)
        none = bl.linear_adapters(x, c.packed, c.gamma, 200, c.A, c.B, c.scale, torch.full_like(c.ids, -1), out_dtype=out,
                                  rmsnorm=norm)
        assert torch.equal(none, bl.forward(c.xq, c.eta, c.xsum, c.packed, c.gamma, 200, out_dtype=out))


def step(c, x):
    """Forward and backward pass of one layer with adapters."""
    y = bl.linear_adapters(x, c.packed, c.gamma, c.N, c.A, c.B, c.scale, c.ids)
    return (y, *bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids),
            bl.grad_weight(c.dy, c.xq, c.eta), bl.grad_input(c.dy, c.packed, c.gamma, c.K))


@pytest.mark.parametrize("M", [2, 40, 600])
def test_two_streams_and_two_graphs_at_once(M):
    """Calls that overlap on the GPU have scratch of their own."""
    cases = [Case(M, 320, 520, 3, 8, seed=i) for i in range(2)]
    xs = [torch.randn(M, 320, device="cuda").to(BF) for _ in cases]
    want = [step(c, x) for c, x in zip(cases, xs)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for c, x, s in zip(cases, xs, streams):
            with torch.cuda.stream(s):
                got.append(step(c, x))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    graphs, held = [], []
    for c, x in zip(cases, xs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(step(c, x))
        graphs.append(graph)
    for _ in range(3):
        for t in held[0] + held[1]:
            t.fill_(3)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(held, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


FRESH = """
import torch
from ternary_weight_linear_04_b200 import bitlinear as bl
from test_gpu_adapters import BF, Case, step
c = Case(70, 320, 520, 3, 8)
x = torch.randn(70, 320, device="cuda").to(BF)
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    held = step(c, x)
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(held, step(c, x)))
print("the same")
"""


def test_the_first_call_of_a_process_can_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([root, os.path.join(root, "tests")]))
    done = subprocess.run([sys.executable, "-c", FRESH], cwd=root, env=env, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "the same" in done.stdout, done.stderr[-2000:]


@pytest.mark.parametrize("M", [1, 9, 40])
def test_tokens_that_start_anywhere(M):
    """A slice of a ragged batch: x, dy and xq off 16 bytes."""
    c = Case(M + 1, 321, 203, 2, 5)
    x = torch.randn(M + 1, 321, device="cuda").to(BF)
    ids = c.ids[1:].clone()
    y = bl.linear_adapters(x[1:], c.packed, c.gamma, 203, c.A, c.B, c.scale, ids)
    assert torch.equal(y, bl.linear_adapters(x[1:].clone(), c.packed, c.gamma, 203, c.A, c.B, c.scale, ids))
    args = lambda f: (f(c.dy[1:]), f(c.xq[1:]), c.eta[1:].clone(), c.packed, c.gamma, c.A, c.B, c.scale, ids)  # noqa: E731
    for a, b in zip(bl.adapters_grad(*args(lambda t: t)), bl.adapters_grad(*args(torch.clone))):
        assert torch.equal(a, b)
    dy, xq, eta = c.dy[1:], c.xq[1:], c.eta[1:].clone()
    assert torch.equal(bl.grad_weight(dy, xq, eta), bl.grad_weight(dy.clone(), xq.clone(), eta))


def test_offsets_past_32_bits():
    """dy of more than 2^31 values: the rows behind that, and their share of the weights' gradients."""
    M, K, N, L, r = 66000, 64, 33000, 2, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    ri = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    c = Case(4, K, N, L, r)
    dy = torch.zeros(M, N, device="cuda", dtype=BF)
    rows = torch.tensor([0, 1, 40000, 65500, 65999], device="cuda")
    dy[rows] = ri(-4, 4, 5, N).to(BF)
    xq, eta, ids = ri(-2, 2, M, K).to(torch.int8), torch.full((M,), 127.0, device="cuda"), ri(-1, 1, M)
    dx, dA, dB = bl.adapters_grad(dy, xq, eta, c.packed, c.gamma, c.A, c.B, c.scale, ids, out_dtype=F32, grad_dtype=F32)
    c.M, c.dy, c.xq, c.eta, c.ids = 5, dy[rows], xq[rows], eta[rows], ids[rows]
    want = c.adapters_grad()
    assert torch.equal(dx[rows], want[0][0].to(F32))
    assert not dx[2:40000].any() and not dx[65501:65999].any()
    same(dA, want[1])
    same(dB, want[2])
    same(bl.grad_weight(dy, xq, eta), c.dw())
    assert torch.equal(bl.grad_input(dy, c.packed, c.gamma, K, out_dtype=F32)[rows], c.dx()[0].to(F32))


def test_a_large_gradient_does_not_wipe_out_the_others():
    """One token's gradients 2^10 times the others': the columns of dW where that token is zero keep the precision the
    fixed point promises (half a unit of 2^-22 of the column's largest for each of the other tokens)."""
    M, K, N = 700, 96, 40
    c = Case(M, K, N, whole=False)
    c.dy[3] = (c.dy[3].float() * 1024).to(BF)
    c.xq[3, ::2] = 0
    top = (c.dy.to(F64).abs() * (c.eta.to(F64) / 127)[:, None]).amax(0)  # of each output n
    val, S = c.dw()
    for out, bits in ((F32, 22), (BF, 14)):
        got = bl.grad_weight(c.dy, c.xq, c.eta, out_dtype=out).to(F64)
        # each g is off by at most half a unit; a unit is at most 2^-bits of the largest (2^-(bits-1) where its power
        # of two had to be halved), and fp32 rounds g itself and the sums of the chunk
        off = top[:, None] * 2.0 ** -bits * c.xq.to(F64).abs().sum(0)[None, :] + S * 2 ** -22 + val.abs() * torch.finfo(out).eps
        assert ((got - val).abs() <= off).all()


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dt", [BF, F32])
def test_gradients_that_are_not_finite_stay_in_their_rows(dt, bad):
    c = Case(1100, 200, 70, 2, 4, dy_dtype=dt)
    clean = [bl.grad_weight(c.dy, c.xq, c.eta, out_dtype=o) for o in (F32, BF)]
    dx = bl.grad_input(c.dy, c.packed, c.gamma, 200)
    grads = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids)
    c.ids[1030] = -1
    without = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids)
    c.dy[1030, 33] = bad
    for o, w in zip((F32, BF), clean):
        got = bl.grad_weight(c.dy, c.xq, c.eta, out_dtype=o)
        assert got[33].isnan().all()
        assert torch.equal(got[torch.arange(70, device="cuda") != 33], w[torch.arange(70, device="cuda") != 33])
    others = torch.arange(1100, device="cuda") != 1030
    assert torch.equal(bl.grad_input(c.dy, c.packed, c.gamma, 200)[others], dx[others])
    # the token has no adapter: dA and dB do not meet it
    got = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids)
    assert torch.equal(got[0][others], grads[0][others])
    assert torch.equal(got[1], without[1]) and torch.equal(got[2], without[2])
