"""Bounded waits of the backward pass and of the adapters' steps.

As test_gpu_timeout.py: the separate build (BL_TEST_HOOKS) withholds one
arrival, a wait runs out after 1 ms, the kernel records BL_ERR_TIMEOUT, lets
what it issued finish, frees its tensor memory and returns without writing
its output; the next call on the same context is exact.  Every wait is
bounded: nothing traps, faults or hangs.
"""
import ctypes

import pytest
import torch

from ternary_weight_linear_04_b200 import _lib
from ternary_weight_linear_04_b200 import build as libbuild
from test_gpu_train import Case, same

pytestmark = pytest.mark.gpu
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def hooks():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    L = ctypes.CDLL(libbuild.build_test_hooks())
    for name, (res, args) in _lib.SIGNATURES.items():
        getattr(L, name).restype, getattr(L, name).argtypes = res, args
    L.bitlinear_test_set_fault.argtypes = [ctypes.c_int]
    yield L
    L.bitlinear_test_set_fault(0)
    L.bitlinear_set_tc_split(0)


def p(t):
    return P(t.data_ptr())


def ran_out(L, fault, run, out, want):
    """`run` with the arrival withheld, then without."""
    def error():
        code = ctypes.c_int32(-1)
        assert L.bitlinear_device_error(ctypes.byref(code), None) == _lib.BL_OK
        return code.value

    assert error() == _lib.BL_OK
    for value, status in ((fault, _lib.BL_ERR_TIMEOUT), (0, _lib.BL_OK)):
        out.fill_(7)
        assert L.bitlinear_test_set_fault(value) == _lib.BL_OK
        torch.cuda.synchronize()
        assert run() == _lib.BL_OK
        torch.cuda.synchronize()
        assert error() == status
        if value:
            assert (out == 7).all(), "an aborted kernel must not write its output"
    same(out, want)


@pytest.mark.parametrize("fault", [1, 2, 3])
@pytest.mark.parametrize("M,K,N", [(40, 1024, 100), (40, 128, 100)])
def test_adapter_steps_of_the_projection(hooks, fault, M, K, N):
    L, c = hooks, Case(M, K, N, 3, 16)
    assert L.bitlinear_set_tc_split(1) == _lib.BL_OK  # one CTA a tile
    y = torch.empty(M, N, device="cuda")
    n = L.bitlinear_forward_adapters_workspace_bytes(M, K, N, 3, 16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ran_out(L, fault, lambda: L.bitlinear_forward_adapters(
        p(c.xq), p(c.eta), p(c.xsum), M, K, p(c.packed), p(c.gamma), N, p(c.A), p(c.B), p(c.scale), p(c.ids), 3, 16,
        p(y), _lib.BL_F32, p(ws), n, 0, None), y, c.y())


@pytest.mark.parametrize("M,K,N", [(40, 256, 448), (1800, 4096, 448)])
def test_input_gradient(hooks, M, K, N):
    """Seven steps: one CTA a tile (few tokens), and two tiles of tokens a CTA (many)."""
    L, c = hooks, Case(M, K, N)
    dx = torch.empty(M, K, device="cuda")
    n = L.bitlinear_grad_input_workspace_bytes(M, N, K, _lib.BL_BF16)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    ran_out(L, 4, lambda: L.bitlinear_grad_input(p(c.dy), _lib.BL_BF16, M, N, p(c.packed), p(c.gamma), K, p(dx),
                                                 _lib.BL_F32, p(ws), n, None), dx, c.dx())


@pytest.mark.parametrize("fault", [5, 6])
@pytest.mark.parametrize("M,K,N", [(300, 256, 200), (1100, 500, 300)])
def test_weight_gradient(hooks, fault, M, K, N):
    L, c = hooks, Case(M, K, N)
    dw = torch.empty(N, K, device="cuda")
    n = L.bitlinear_grad_weight_workspace_bytes(M, N, K, _lib.BL_BF16, _lib.BL_F32)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ran_out(L, fault, lambda: L.bitlinear_grad_weight(p(c.dy), _lib.BL_BF16, p(c.xq), p(c.eta), M, N, K, p(dw),
                                                      _lib.BL_F32, p(ws), n, None), dw, c.dw())
