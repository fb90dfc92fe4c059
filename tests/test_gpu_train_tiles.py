"""Every tile of the tensor-core kernels of the adapters and of the input
gradient: exact inputs at sizes that take it, ragged widths among them.
Inputs, 64-bit forms and tolerances as in test_gpu_train.py."""
import pytest
import torch

from ternary_weight_linear_04_b200 import bitlinear as bl
from ternary_weight_linear_04_b200 import build as libbuild
from test_gpu_train import BF, F32, Case, near, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert bl.device_error() == 0


# tokens of the tile, M, K, N; K of 4096 and more is split over a cluster where the tiles leave room
FORWARD = [(32, 20, 320, 200), (64, 40, 320, 200), (32, 17, 4160, 200), (64, 64, 8192, 130), (64, 600, 4160, 264),
           (128, 100, 130, 14400), (128, 128, 256, 14331), (256, 300, 130, 11003), (256, 700, 192, 8192),
           (256, 2048, 64, 2500), (256, 300, 4160, 11008)]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("order", ["mixed", "packed"])
@pytest.mark.parametrize("L,r", [(1, 16), (3, 5), (4, 40), (40, 3)])
@pytest.mark.parametrize("tile,M,K,N", FORWARD)
def test_projection_with_adapters(tile, M, K, N, L, r, order, out):
    assert bl.tile_tokens(M, K, N, sms=148) == tile
    c = Case(M, K, N, L, r, order=order)
    same(bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, N, c.A, c.B, c.scale, c.ids, out_dtype=out), c.y())


@pytest.mark.parametrize("tile,M,K,N", FORWARD)
def test_projection_with_adapters_drawn(tile, M, K, N):
    """Additions of an output: K / 64 steps of u, 16 warps' and 8 CTAs' sums, four MMAs in a step, and as few for y."""
    c = Case(M, K, N, 3, 12, whole=False)
    for out in (BF, F32):
        near(bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, N, c.A, c.B, c.scale, c.ids, out_dtype=out), c.y(), K // 64 + 48)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("tile,M,K,N", [t for t in FORWARD if t[0] >= 128])
def test_a_large_tile_keeps_what_is_not_finite_apart(tile, M, K, N, out):
    c = Case(M, K, N, 3, 5)
    y = bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, N, c.A, c.B, c.scale, c.ids, out_dtype=out)
    for t in (c.A, c.B):
        keep = t.clone()
        t[1].view(-1)[::7] = float("inf")
        got = bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, N, c.A, c.B, c.scale, c.ids, out_dtype=out)
        assert torch.equal(got[c.ids != 1], y[c.ids != 1]) and not got[c.ids == 1].isfinite().all()
        t.copy_(keep)


# tokens of the tile, M, K, N
GRAD = [(128, 300, 3200, 70), (256, 1100, 7000, 70), (256, 1100, 7001, 72), (256, 1030, 7168, 200), (256, 300, 14592, 33),
        (256, 2048, 4096, 130)]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("tile,M,K,N", GRAD)
def test_input_gradient(tile, M, K, N, dt, out):
    assert bl.tile_tokens(M, K, N, grad=True, sms=148) == tile
    c = Case(M, K, N, dy_dtype=dt)
    same(bl.grad_input(c.dy, c.packed, c.gamma, K, out_dtype=out), c.dx())


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("L,r", [(1, 16), (3, 5), (4, 40), (40, 3)])
@pytest.mark.parametrize("tile,M,K,N", GRAD)
def test_input_gradient_with_adapters(tile, M, K, N, L, r, dt, out):
    c = Case(M, K, N, L, r, dy_dtype=dt)
    dx = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, out_dtype=out, want_dab=False)[0]
    same(dx, c.adapters_grad()[0])


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("tile,M,K,N", GRAD)
def test_input_gradient_keeps_what_is_not_finite_apart(tile, M, K, N, out, bad):
    c = Case(M, K, N, 3, 5)
    args = lambda: (c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids)  # noqa: E731
    dx = bl.adapters_grad(*args(), out_dtype=out, want_dab=False)[0]
    c.A[1, 2, K - 3] = bad
    got = bl.adapters_grad(*args(), out_dtype=out, want_dab=False)[0]
    own = c.ids == 1
    assert torch.equal(got[~own], dx[~own])
    rest = torch.arange(K, device="cuda") != K - 3
    assert torch.equal(got[:, rest], dx[:, rest])
    assert not got[own, K - 3].isfinite().any()


@pytest.mark.parametrize("M", [1, 2, 8, 9, 16])
@pytest.mark.parametrize("K,N,L,r", [(64, 40001, 3, 8), (4096, 11008, 2, 16), (256, 100000, 5, 5), (8192, 9000, 1, 40)])
def test_few_tokens_on_the_tensor_cores(M, K, N, L, r):
    """Layers that the register-resident kernels do not take: tiles of 16 tokens."""
    assert bl.decode_regm_shape(max(M, 2), K, N, sms=148) is None and bl.decode_mma_shape(M, K, N, sms=148) is None
    assert bl.tile_tokens(M, K, N, sms=148) == 16
    c = Case(M, K, N, L, r)
    for out in (BF, F32):
        same(bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, N, c.A, c.B, c.scale, c.ids, out_dtype=out), c.y())
    x = torch.randn(M, K, device="cuda").to(BF)
    c.xq, c.eta, c.xsum = bl.quant_act(x)
    y = bl.linear_adapters(x, c.packed, c.gamma, N, c.A, c.B, c.scale, c.ids, out_dtype=F32)
    near(y, c.y(), K // 64 + 48)


@pytest.mark.parametrize("M", [1, 5, 12])
def test_the_register_kernels_switched_off(M):
    c = Case(M, 320, 200, 3, 8)
    args = (c.xq, c.eta, c.xsum, c.packed, c.gamma, 200, c.A, c.B, c.scale, c.ids)
    try:
        bl.set_decode_reg(False)
        bl.set_decode_mma(False)
        same(bl.forward_adapters(*args, out_dtype=F32), c.y())
        x = torch.randn(M, 320, device="cuda").to(BF)
        off = bl.linear_adapters(x, *args[3:5], 200, *args[6:], out_dtype=F32)
    finally:
        bl.set_decode_reg(True)
        bl.set_decode_mma(True)
    c.xq, c.eta, c.xsum = bl.quant_act(x)
    near(off, c.y(), 320 // 8 + 48)
