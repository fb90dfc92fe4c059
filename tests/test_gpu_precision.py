"""What the sums of the backward pass and the adapters hold.

Inputs for which every term and every partial sum is exact, built so that a
value with fewer bits than fp32's, or a sum that is cut off instead of
rounded, gives another result than the formula's.
"""
import pytest
import torch

from ternary_weight_linear_04_b200 import bitlinear as bl
from ternary_weight_linear_04_b200 import build as libbuild
from test_gpu_train import BF, F32, F64, Case, pack  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert bl.device_error() == 0


def still(M, K, N, L=1, r=2):
    """A case whose every input is zero, of unit scales."""
    c = Case(M, K, N, L, r)
    for t in (c.xq, c.xsum, c.dy, c.A, c.B, c.t):
        t.zero_()
    c.packed = pack(c.t)
    c.gamma.fill_(1)
    c.eta.fill_(127)
    c.scale.fill_(1)
    c.ids.zero_()
    return c


# 1 + 2^-10 + 2^-20 has 21 bits in three groups: no two bf16 values hold it
LONG = (1.0, 2.0 ** -10, 2.0 ** -20)
SHORT = (1.0, 2.0 ** -10, 0.0)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,K,N", [(1, 64, 64), (16, 64, 64), (17, 64, 64), (40, 70, 33), (300, 64, 9000), (600, 64, 72)])
def test_u_enters_y_whole(M, K, N, out):
    """u = (1 + 2^-10 + 2^-20, -1 - 2^-10) against B = (1, 1): 2^-20 is left."""
    c = still(M, K, N)
    c.xq[:, :3] = 1
    c.xsum[:] = 3
    c.A[0, 0, :3] = torch.tensor(LONG).to(BF)
    c.A[0, 1, :3] = -torch.tensor(SHORT).to(BF)
    c.B.fill_(1)
    y = bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, N, c.A, c.B, c.scale, c.ids, out_dtype=out)
    assert (y == 2.0 ** -20).all()


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,K,N", [(1, 64, 64), (40, 70, 33), (300, 9000, 64), (1800, 4096, 64)])
def test_v_enters_dx_whole(M, K, N, dt, out):
    c = still(M, K, N)
    c.dy = c.dy.to(dt)
    c.dy[:, :3] = torch.tensor(LONG).to(dt)
    c.B[0, :3, 0] = 1
    c.B[0, :2, 1] = -1
    c.A.fill_(1)
    dx = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, out_dtype=out, want_dab=False)[0]
    assert (dx == 2.0 ** -20).all()


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M", [2, 32, 128, 1024])
@pytest.mark.parametrize("r", [2, 40, 128])
def test_u_and_v_enter_the_factors_gradients_whole(M, r, out):
    """Every other token's u and v are -(1 + 2^-10): M / 2 times 2^-20 are left."""
    c = still(M, 64, 72, 1, r)
    c.xq[0::2, :3] = 1
    c.xq[1::2, :2] = -1
    c.A[0, 0, :3] = torch.tensor(LONG).to(BF)
    c.dy[:, 5] = 1
    dB = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, grad_dtype=out, want_dx=False)[2]
    assert (dB[0, 5, 0] == M / 2 * 2.0 ** -20) and dB.count_nonzero() == 1
    c = still(M, 64, 72, 1, r)
    c.dy[0::2, :3] = torch.tensor(LONG).to(BF)
    c.dy[1::2, :3] = -torch.tensor(SHORT).to(BF)
    c.B[0, :3, 0] = 1
    c.xq[:, 7] = 1
    dA = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, grad_dtype=out, want_dx=False)[1]
    assert (dA[0, 0, 7] == M / 2 * 2.0 ** -20) and dA.count_nonzero() == 1


TOP = torch.finfo(F32).max  # rounds to infinity in bf16


@pytest.mark.parametrize("M,K,N", [(3, 64, 64), (40, 130, 70), (300, 9000, 72)])
@pytest.mark.parametrize("big", [float("inf"), -float("inf"), TOP, -TOP])
def test_an_fp32_gradient_past_bf16(M, K, N, big):
    """Infinities and the largest numbers of an fp32 dy stay what they are in dx, v and dA, and large numbers in dB."""
    c = still(M, K, N, 1, 3)
    c.dy = c.dy.float()
    c.dy[2, 5] = big
    c.t[5, 0::2] = 1
    c.t[5, 1::2] = -1
    c.packed = pack(c.t)
    c.gamma.fill_(0.125)
    want = torch.full((K,), big * 0.125, device="cuda")
    want[1::2] *= -1
    if abs(big) == float("inf"):  # the sum of a row meets no zero of another output's weights
        c.t[c.t == 0] = 1
        c.packed = pack(c.t)
    for out in (F32, BF):
        dx = bl.grad_input(c.dy, c.packed, c.gamma, K, out_dtype=out)
        assert torch.equal(dx[2], want.to(out))
        assert not dx[:2].any() and not dx[3:].any()
    c.xq[2, 7] = 16
    c.eta.fill_(127)
    c.A[0, 0, 7] = 2.0 ** -7  # u = 1 / 8
    dB = bl.adapters_grad(c.dy, c.xq, c.eta, None, None, c.A, c.B, c.scale, c.ids, grad_dtype=F32, want_dx=False)[2]
    if abs(big) == float("inf"):  # times the empty parts of u: an infinity here may come out as NaN
        assert not dB[0, 5, 0].isfinite()
    else:
        assert float(dB[0, 5, 0]) == big * 0.125
    assert not dB[0, :5].any() and not dB[0, 6:].any()
    c.eta.fill_(127 / 1024.)  # x^ = 16 / 1024
    c.B[0, 5, 1] = 1
    dA = bl.adapters_grad(c.dy, c.xq, c.eta, None, None, c.A, c.B, c.scale, c.ids, grad_dtype=F32, want_dx=False)[1]
    assert float(dA[0, 1, 7]) == big / 64


# A sum in fp32 that rounds to nearest is off by at most half a step for each
# addition; one that cuts off, by a whole one.  Here a running sum of 2^24
# (steps of 2) takes 63/32 once for each further 16 tokens: cut off, none of
# them arrives.

def additions(M):
    return (M + 15) // 16


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("r", [2, 40, 128])
def test_factors_gradients_round_to_nearest(dt, r):
    M = 240  # one CTA's chain: clusters split 256 tokens and more
    c = still(M, 64, 72, 1, r)
    c.dy = c.dy.to(dt)
    c.B[0, 3, 0] = 1
    c.dy[0, 3] = 2.0 ** 24
    c.dy[16::16, 3] = 63 / 32
    c.xq[:, 7] = 1
    want = 2.0 ** 24 + (additions(M) - 1) * 63 / 32
    dA = bl.adapters_grad(c.dy, c.xq, c.eta, None, None, c.A, c.B, c.scale, c.ids, grad_dtype=F32, want_dx=False)[1]
    assert abs(float(dA[0, 0, 7]) - want) <= additions(M) and dA.count_nonzero() == 1
    c = still(M, 64, 72, 1, r)
    c.dy = c.dy.to(dt)
    c.A[0, 0, 5] = 1
    c.xq[0, 5] = 1
    c.xq[16::16, 5] = 63
    c.eta[0] = 127 * 2.0 ** 24
    c.eta[1:] = 127 / 32
    c.dy[:, 3] = 1
    dB = bl.adapters_grad(c.dy, c.xq, c.eta, None, None, c.A, c.B, c.scale, c.ids, grad_dtype=F32, want_dx=False)[2]
    assert abs(float(dB[0, 3, 0]) - want) <= additions(M) and dB.count_nonzero() == 1


@pytest.mark.parametrize("dt", [BF, F32])
def test_v_rounds_to_nearest(dt):
    """Steps of 64 outputs, 12 of them a warp: within the first step three MMAs may cut off (2 each), then eleven
    additions of steps and fifteen of warps round (1 each)."""
    M, K, N = 4800, 64, 64 * 16 * 12
    c = still(M, K, N)
    c.A[0, 0] = 1
    c.B[0, :, 0] = 1
    c.dy = c.dy.to(dt)
    c.dy[:, 16::16] = 63 / 32
    c.dy[:, 0] = 2.0 ** 24
    want = 2.0 ** 24 + (N // 16 - 1) * 63 / 32
    dx = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, out_dtype=F32, want_dab=False)[0]
    assert float((dx.to(F64) - want).abs().max()) <= 3 * 2 + 11 + 15


def test_u_rounds_to_nearest():
    M, K, N = 4800, 64 * 16 * 12, 64
    c = still(M, K, N)
    for i in range(0, 16, 4):  # one for each MMA of a step: MMA i takes the codes 16 q + 4 i .. + 3 (q < 4)
        c.A[0, 0, i::64] = 63 / 32
    c.A[0, 0, 0] = 2.0 ** 24
    c.xq.fill_(1)
    c.xsum.fill_(K)
    c.B[0, :, 0] = 1
    want = 2.0 ** 24 + (K // 16 - 1) * 63 / 32
    y = bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, N, c.A, c.B, c.scale, c.ids, out_dtype=F32)
    assert float((y.to(F64) - want).abs().max()) <= 3 * 2 + 11 + 15


@pytest.mark.parametrize("M,K,N", [(100, 320, 4096), (1800, 4096, 4096), (300, 9000, 2048)])
def test_the_low_planes_of_an_fp32_dy_are_not_cut_off(M, K, N):
    """dy = 1 + 2^-22: the last bits add up to N 2^-22, which a running sum of the tops would lose."""
    c = still(M, K, N)
    c.dy = torch.full((M, N), 1 + 2.0 ** -22, device="cuda")
    c.t.fill_(1)
    c.packed = pack(c.t)
    want = N + N * 2.0 ** -22
    assert float(torch.tensor(want, dtype=F32)) == want
    dx = bl.grad_input(c.dy, c.packed, c.gamma, K, out_dtype=F32)
    assert (dx == want).all()


@pytest.mark.parametrize("out", [BF, F32])
def test_weight_gradients_keep_all_of_a_column(out):
    """dy eta / 127 of 1 + 2^-20 and -1: 2^-20 of the codes is left."""
    c = still(70, 96, 40)
    c.dy[3, :] = 1
    c.dy[50, :] = -1
    c.eta[3] = 127 * (1 + 2.0 ** -20)
    c.xq[3] = c.xq[50] = torch.arange(-48, 48, device="cuda", dtype=torch.int8)
    assert float(c.eta[3] / 127) == 1 + 2.0 ** -20
    dw = bl.grad_weight(c.dy, c.xq, c.eta, out_dtype=out)
    assert torch.equal(dw.float(), (c.xq[3].float() * 2.0 ** -20).expand(40, 96))


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("power", [6, 10, 14, 20, 26])
@pytest.mark.parametrize("M,K,N", [(5, 40, 10), (700, 130, 300), (1100, 64, 70), (2500, 200, 513), (3000, 2100, 2500)])
def test_a_column_with_one_large_token(M, K, N, power, dt, out):
    """One token 2^power times the others, in some columns and one chunk: where its codes are zero the others' sum is
    exact, as are the columns beside it."""
    c = Case(M, K, N, dy_dtype=dt)
    big = M - 2
    cols = torch.arange(N, device="cuda") % 130 == 5
    c.dy[big, cols] = 2.0 ** power
    c.eta[big] = 127
    c.xq[big, 1::2] = 0
    val = c.dw()[0]
    got = bl.grad_weight(c.dy, c.xq, c.eta, out_dtype=out)
    assert torch.equal(val[:, 1::2], val[:, 1::2].to(F32).to(F64)) and torch.equal(val[~cols], val[~cols].to(F32).to(F64))
    assert torch.equal(got[:, 1::2], val[:, 1::2].to(F32).to(out))
    assert torch.equal(got[~cols], val[~cols].to(F32).to(out))


def promised(c, out):
    """Largest error the fixed point promises: in each chunk of 1024 tokens half a unit of the last digit for each
    token's g: the largest is below 2^5 times the geometric mean for the digits taken (2^4, and the exponents' floors),
    and half a unit at most 2^-22.99 of it (2^22 units, or half of 8355711); g
    itself is rounded once (2^-24) and its factor once; each chunk adds up to five digits' sums in fp32."""
    g = c.dy.to(F64).abs() * (c.eta.to(F64) / 127)[:, None]
    bound, S = 0, g.t() @ c.xq.to(F64).abs()
    for m in range(0, c.M, 1024):
        part = g[m:m + 1024]
        some = part > 0
        mean = torch.exp2((torch.where(some, part, 1.0).log2().sum(0) / some.sum(0).clamp(min=1)))
        bound = bound + (2.0 ** -17.9 * mean)[:, None] * c.xq[m:m + 1024].to(F64).abs().sum(0)[None, :]
    adds = 5 * ((c.M + 1023) // 1024)
    return bound + (2 + adds) * 2.0 ** -24 * S


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("kind", ["normal", "heavy", "tokens", "outlier"])
@pytest.mark.parametrize("M,K,N", [(3, 64, 70), (200, 96, 300), (1024, 64, 64), (2500, 130, 72), (4100, 64, 513)])
def test_weight_gradients_of_any_spread(M, K, N, kind, dt):
    c = Case(M, K, N, whole=False)
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    z = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    dy = z(M, N)
    if kind == "heavy":
        dy = dy.sign() * torch.exp(2 * z(M, N))
    elif kind == "tokens":
        dy = dy * torch.exp(3 * z(M, 1))
    elif kind == "outlier":
        c.eta[1] *= 2 ** 13
        c.xq[1, 1:] = 0
    c.dy = dy.to(dt)
    val = c.dw()[0]
    off = (bl.grad_weight(c.dy, c.xq, c.eta).to(F64) - val).abs()
    assert (off <= promised(c, F32)).all(), float((off / promised(c, F32)).max())
    off = (bl.grad_weight(c.dy, c.xq, c.eta, out_dtype=BF).to(F64) - val).abs()
    assert (off <= promised(c, BF) + 2.0 ** -8 * (val.abs() + promised(c, BF))).all()
