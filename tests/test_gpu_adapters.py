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
