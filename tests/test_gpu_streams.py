"""Outputs and scratch belong to the stream that a call runs on."""
import pytest
import torch

from ternary_weight_linear_04_b200 import bitlinear as bl
from ternary_weight_linear_04_b200 import build as libbuild
from test_gpu_train import BF, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert bl.device_error() == 0


def calls(c, x):
    ad = (c.A, c.B, c.scale, c.ids)
    return {
        "rmsnorm_quant_act": lambda s=None: bl.rmsnorm_quant_act(x, want_rstd=True, stream=s),
        "grad_input": lambda s=None: bl.grad_input(c.dy, c.packed, c.gamma, c.K, stream=s),
        "grad_weight": lambda s=None: bl.grad_weight(c.dy, c.xq, c.eta, stream=s),
        "rmsnorm_grad": lambda s=None: bl.rmsnorm_grad(x, c.xq, c.eta, c.eta, stream=s),
        "forward_adapters": lambda s=None: bl.forward_adapters(c.xq, c.eta, c.xsum, c.packed, c.gamma, c.N, *ad, stream=s),
        "linear_adapters": lambda s=None: bl.linear_adapters(x, c.packed, c.gamma, c.N, *ad, stream=s),
        "adapters_grad": lambda s=None: bl.adapters_grad(c.dy, c.xq, c.eta, c.packed, c.gamma, *ad, stream=s),
    }


@pytest.mark.parametrize("name", [
    "rmsnorm_quant_act", "grad_input", "grad_weight", "rmsnorm_grad", "forward_adapters", "linear_adapters", "adapters_grad"])
def test_memory_that_another_stream_still_writes(name):
    """Blocks freed on the current stream, their last writes not run yet: a call on another stream does not take them."""
    c = Case(70, 256, 136, 3, 8)
    x = torch.randn(70, 256, device="cuda").to(BF)
    call = calls(c, x)[name]
    want = call()
    want = want if isinstance(want, tuple) else (want,)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.empty_like(t) for t in want for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    for t in freed:
        t.fill_(7)
    del freed, t
    got = call(side)
    got = got if isinstance(got, tuple) else (got,)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
