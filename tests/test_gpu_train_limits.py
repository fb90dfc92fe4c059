"""The backward pass and the adapters at the ends of their ranges: outputs past
2^31 values, as many adapters as there may be, codes of every size, calls of
several host threads.  Inputs and 64-bit forms as in test_gpu_train.py."""
import threading

import pytest
import torch

from ternary_weight_linear_04_b200 import bitlinear as bl
from ternary_weight_linear_04_b200 import build as libbuild
from test_gpu_train import BF, F32, Case, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert bl.device_error() == 0


def rows_of(c, rows):
    """The case's tokens at `rows` alone, for the 64-bit forms."""
    c.M, c.xq, c.eta, c.ids, c.dy = len(rows), c.xq[rows], c.eta[rows], c.ids[rows], c.dy[rows]
    return c


ROWS = [0, 1, 32768, 65074, 65075, 65999]


def test_outputs_past_32_bits():
    """y and dx of more than 2^31 values."""
    c = Case(66000, 64, 33000, 3, 8)
    y = bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, c.N, c.A, c.B, c.scale, c.ids)[ROWS]
    same(y, rows_of(c, ROWS).y())
    c = Case(66000, 33000, 64, 3, 8)
    ad = (c.A, c.B, c.scale, c.ids)
    dx = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, *ad, want_dab=False)[0][ROWS]
    plain = bl.grad_input(c.dy, c.packed, c.gamma, c.K)[ROWS]
    c = rows_of(c, ROWS)
    same(dx, c.adapters_grad()[0])
    same(plain, c.dx())


@pytest.mark.parametrize("dt,out", [(BF, BF), (F32, F32)])
def test_a_weight_gradient_past_32_bits(dt, out):
    c = Case(40, 40000, 54000, dy_dtype=dt)
    dw = bl.grad_weight(c.dy, c.xq, c.eta, out_dtype=out)
    for n in (0, 53687, 53999):
        same(dw[n], (c.dy[:, n].double() @ c.xh,))


@pytest.mark.parametrize("M", [1, 40, 700])
def test_as_many_adapters_as_there_may_be(M):
    c = Case(M, 24, 16, 65535, 1)
    c.ids[0] = 65534
    same(bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, 16, c.A, c.B, c.scale, c.ids), c.y())
    dx, dA, dB = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, grad_dtype=F32)
    used = c.ids.unique()
    used = used[used >= 0].long()
    c.scale, c.A, c.B = c.scale[used], c.A[used], c.B[used]
    c.ids = torch.where(c.ids >= 0, torch.searchsorted(used, c.ids.long()), -1).int()
    c.L = len(used)
    want = c.adapters_grad()
    same(dx, want[0])
    same(dA[used], want[1])
    same(dB[used], want[2])
    rest = torch.ones(65535, dtype=torch.bool, device="cuda")
    rest[used] = False
    assert not dA[rest].any() and not dB[rest].any()


@pytest.mark.parametrize("M", [5, 300])
def test_codes_of_every_size(M):
    """127 and -127 everywhere, and -128, which no quantiser writes."""
    c = Case(M, 200, 72, 2, 4)
    for codes in ((-127, 127), (-128, 127), (-128, -128)):
        c.xq[:, 0::2], c.xq[:, 1::2] = codes
        c.xsum = c.xq.sum(1, dtype=torch.int32)
        same(bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, 72, c.A, c.B, c.scale, c.ids, out_dtype=F32), c.y())
        same(bl.grad_weight(c.dy, c.xq, c.eta), c.dw())
        got = bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, c.A, c.B, c.scale, c.ids, out_dtype=F32, grad_dtype=F32)
        for g, w in zip(got, c.adapters_grad()):
            same(g, w)


def test_calls_of_several_host_threads():
    cases = [Case(M, 320, 520, 3, 8, seed=M) for M in (3, 40, 300, 600)]

    def step(c):
        ad = (c.A, c.B, c.scale, c.ids)
        return (bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, 520, *ad),
                *bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, *ad), bl.grad_weight(c.dy, c.xq, c.eta))

    want = [step(c) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def run(c, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    if not all(torch.equal(a, b) for a, b in zip(step(c), w)):
                        wrong.append(c.M)
        except Exception as e:  # pragma: no cover
            wrong.append(e)

    threads = [threading.Thread(target=run, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
