"""Backward-pass and adapter entry points: refusals before any launch (no GPU)
and the binding's checks of shapes and types."""
import ctypes

import pytest
import torch

from ternary_weight_linear_04_b200 import _lib
from ternary_weight_linear_04_b200 import bitlinear as bl
from ternary_weight_linear_04_b200 import build as libbuild

P = ctypes.c_void_p
F = 4096  # a fake, aligned address: validation fails before it is read
BAD, UNS, ALN, OK = (_lib.BL_ERR_INVALID_ARG, _lib.BL_ERR_UNSUPPORTED, _lib.BL_ERR_ALIGNMENT, _lib.BL_OK)
BIG = 1 << 40  # a workspace size that is never too small


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return _lib.lib()


def call(fn, base, **change):
    args = dict(base, **change)
    return fn(*[P(v) if v is not None and k.startswith("p_") else v for k, v in args.items()])


GI = dict(p_dy=F, dydt=1, M=4, N=64, p_packed=F, p_gamma=F, K=64, p_dx=F, dxdt=1, p_ws=F, nws=BIG, p_s=None)
GW = dict(p_dy=F, dydt=1, p_xq=F, p_eta=F, M=4, N=64, K=64, p_dw=F, dwdt=0, p_ws=F, nws=BIG, p_s=None)
RN = dict(p_dn=F, dndt=1, p_xq=F, p_eta=F, p_rstd=F, M=4, K=64, p_dx=F, dxdt=1, p_s=None)
FA = dict(p_xq=F, p_eta=F, p_xsum=F, M=4, K=64, p_packed=F, p_gamma=F, N=64, p_A=F, p_B=F, p_scale=F, p_ids=F,
          L=2, r=8, p_y=F, ydt=1, p_ws=F, nws=BIG, flags=0, p_s=None)
AG = dict(p_dy=F, dydt=1, p_xq=F, p_eta=F, M=4, N=64, K=64, p_packed=F, p_gamma=F, p_A=F, p_B=F, p_scale=F,
          p_ids=F, L=2, r=8, p_dx=F, dxdt=1, p_dA=F, p_dB=F, dabdt=1, p_ws=F, nws=BIG, p_s=None)

REFUSED = [
    ("grad_input", GI, BAD, [dict(p_dy=None), dict(p_packed=None), dict(p_gamma=None), dict(p_dx=None),
                             dict(dydt=2), dict(dxdt=7), dict(M=-1), dict(N=0), dict(K=0)]),
    ("grad_input", GI, UNS, [dict(M=1 << 30), dict(N=1 << 30), dict(K=1 << 25), dict(M=1 << 29, K=1 << 12)]),
    ("grad_input", GI, ALN, [dict(p_dy=F + 8), dict(p_packed=F + 4), dict(p_dx=F + 8), dict(p_gamma=F + 2),
                             dict(p_ws=F + 16)]),
    ("grad_weight", GW, BAD, [dict(p_dy=None), dict(p_xq=None), dict(p_eta=None), dict(p_dw=None), dict(dydt=3),
                              dict(dwdt=-1), dict(M=-1), dict(N=0), dict(K=-5)]),
    ("grad_weight", GW, UNS, [dict(M=1 << 30), dict(N=1 << 30), dict(K=1 << 25)]),
    ("grad_weight", GW, ALN, [dict(p_dy=F + 2), dict(p_xq=F + 1), dict(p_dw=F + 4), dict(p_eta=F + 2),
                              dict(p_ws=F + 128)]),
    ("rmsnorm_grad", RN, BAD, [dict(p_dn=None), dict(p_xq=None), dict(p_eta=None), dict(p_rstd=None),
                               dict(p_dx=None), dict(dndt=2), dict(dxdt=2), dict(M=-1), dict(K=0)]),
    ("rmsnorm_grad", RN, UNS, [dict(K=(1 << 24) + 1), dict(M=1 << 39)]),
    ("rmsnorm_grad", RN, ALN, [dict(p_dn=F + 1), dict(p_dx=F + 1), dict(p_eta=F + 2), dict(p_rstd=F + 1)]),
    ("forward_adapters", FA, BAD, [dict(p_xq=None), dict(p_eta=None), dict(p_xsum=None), dict(p_packed=None),
                                   dict(p_gamma=None), dict(p_A=None), dict(p_B=None), dict(p_scale=None),
                                   dict(p_ids=None), dict(p_y=None), dict(p_ws=None), dict(ydt=2), dict(L=0),
                                   dict(r=0), dict(M=-1), dict(N=0), dict(K=0), dict(nws=0)]),
    ("forward_adapters", FA, UNS, [dict(L=65536), dict(r=129), dict(M=1 << 30), dict(K=1 << 25)]),
    ("forward_adapters", FA, ALN, [dict(p_xq=F + 8), dict(p_packed=F + 8), dict(p_A=F + 2), dict(p_B=F + 8),
                                   dict(p_y=F + 2), dict(p_ids=F + 2), dict(p_scale=F + 2), dict(p_ws=F + 8)]),
    ("adapters_grad", AG, BAD, [dict(p_dy=None), dict(p_xq=None), dict(p_eta=None), dict(p_packed=None),
                                dict(p_gamma=None), dict(p_A=None), dict(p_B=None), dict(p_scale=None),
                                dict(p_ids=None), dict(p_dA=None), dict(p_dB=None), dict(p_ws=None),
                                dict(p_dx=None, p_dA=None, p_dB=None), dict(dydt=2), dict(dxdt=2), dict(dabdt=2),
                                dict(L=0), dict(r=0), dict(M=-1), dict(N=0), dict(K=0), dict(nws=0)]),
    ("adapters_grad", AG, UNS, [dict(L=65536), dict(r=129), dict(N=1 << 30), dict(K=1 << 25)]),
    ("adapters_grad", AG, ALN, [dict(p_dy=F + 2), dict(p_xq=F + 4), dict(p_packed=F + 8), dict(p_A=F + 8),
                                dict(p_B=F + 8), dict(p_dx=F + 8), dict(p_dA=F + 8), dict(p_dB=F + 2),
                                dict(p_ids=F + 1), dict(p_ws=F + 64)]),
]


@pytest.mark.parametrize("name,base,status,changes", REFUSED)
def test_refused_before_a_launch(L, name, base, status, changes):
    fn = getattr(L, "bitlinear_" + name)
    for change in changes:
        assert call(fn, base, **change) == status, change


def test_no_tokens_is_no_work(L):
    assert call(L.bitlinear_grad_input, GI, M=0, p_dy=None, p_dx=None, p_ws=None, nws=0) == OK
    assert call(L.bitlinear_rmsnorm_grad, RN, M=0, p_dn=None, p_dx=None, p_xq=None) == OK
    assert call(L.bitlinear_forward_adapters, FA, M=0, p_xq=None, p_ids=None, p_y=None, p_ws=None, nws=0) == OK
    rq = L.bitlinear_rmsnorm_quant_act_rstd
    assert rq(None, 1, 0, 64, None, None, None, None, None) == OK
    assert rq(P(F), 1, 1, 64, P(F), P(F), P(F), None, None) == BAD
    assert rq(P(F), 1, 1, 64, P(F), P(F), P(F), P(F + 2), None) == ALN
    assert rq(P(F), 0, 1, 64, P(F), P(F), P(F), P(F), None) == UNS  # fp32 input


def test_a_small_workspace_is_refused(L):
    for fn, base, need in [
            (L.bitlinear_grad_input, GI, L.bitlinear_grad_input_workspace_bytes(4, 63, 61, 0)),
            (L.bitlinear_grad_weight, GW, L.bitlinear_grad_weight_workspace_bytes(4, 63, 61, 0, 0)),
            (L.bitlinear_forward_adapters, FA, L.bitlinear_forward_adapters_workspace_bytes(4, 61, 63, 2, 8)),
            (L.bitlinear_adapters_grad, AG, L.bitlinear_adapters_grad_workspace_bytes(4, 63, 61, 2, 8, 0))]:
        if need:
            change = dict(K=61, N=63, nws=need - 1)
            if "dydt" in base:
                change["dydt"] = 0
            assert call(fn, base, **change) == BAD


def test_workspace_queries_of_refused_sizes_are_zero(L):
    assert L.bitlinear_grad_input_workspace_bytes(4, 0, 64, 1) == 0
    assert L.bitlinear_grad_weight_workspace_bytes(4, 64, 64, 9, 0) == 0
    assert L.bitlinear_forward_adapters_workspace_bytes(4, 64, 64, 2, 129) == 0
    assert L.bitlinear_adapters_grad_workspace_bytes(-1, 64, 64, 2, 8, 1) == 0


def test_binding_checks_shapes_and_types():
    bf, f32 = torch.bfloat16, torch.float32
    dy, xq, eta = torch.zeros(4, 6, dtype=bf), torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    packed, gamma = torch.zeros(6, 2, dtype=torch.uint8), torch.ones(1)
    A, B = torch.zeros(2, 3, 8, dtype=bf), torch.zeros(2, 6, 3, dtype=bf)
    scale, ids = torch.ones(2), torch.zeros(4, dtype=torch.int32)
    bad = [
        lambda: bl.grad_input(dy.half(), packed, gamma, 8),
        lambda: bl.grad_input(dy, packed, gamma, 9),
        lambda: bl.grad_input(dy[0], packed, gamma, 8),
        lambda: bl.grad_input(dy, packed, gamma.double(), 8),
        lambda: bl.grad_weight(dy, xq[:3], eta),
        lambda: bl.grad_weight(dy, xq.to(torch.uint8), eta),
        lambda: bl.grad_weight(dy, xq, eta[:3]),
        lambda: bl.rmsnorm_grad(dy, xq, eta, eta),
        lambda: bl.rmsnorm_grad(torch.zeros(4, 8), xq, eta, eta[:2]),
        lambda: bl.forward_adapters(xq, eta, ids, packed, gamma, 6, A.float(), B, scale, ids),
        lambda: bl.forward_adapters(xq, eta, ids, packed, gamma, 6, A, B.transpose(1, 2), scale, ids),
        lambda: bl.forward_adapters(xq, eta, ids, packed, gamma, 6, A, B, scale[:1], ids),
        lambda: bl.forward_adapters(xq, eta, ids, packed, gamma, 6, A, B, scale, ids.long()),
        lambda: bl.forward_adapters(xq, eta, ids, packed, gamma, 6, A[0], B[0], scale, ids),
        lambda: bl.forward_adapters(xq, eta, ids, packed, gamma, 7, A, B, scale, ids),
        lambda: bl.adapters_grad(dy, xq, eta, packed, gamma, A, B[:1], scale, ids),
        lambda: bl.adapters_grad(dy, xq, eta, packed, gamma, A, B, scale, ids, want_dx=False, want_dab=False),
        # right shapes, but not on a GPU
        lambda: bl.grad_input(dy, packed, gamma, 8),
        lambda: bl.grad_weight(dy, xq, eta),
        lambda: bl.linear_adapters(dy, packed, gamma, 6, A, B, scale, ids),
        lambda: bl.adapters_grad(dy, xq, eta, packed, gamma, A, B, scale, ids),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was taken" % i)


class FakeTensor:
    """Enough of a CUDA tensor for the checks before a launch."""
    is_cuda = True

    def __init__(self, index, contiguous=True):
        self.index, self.contiguous = index, contiguous

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous


def test_tensors_of_two_devices_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert bl._place(None, FakeTensor(0), None, FakeTensor(0)) is bl._HERE
    with pytest.raises(ValueError, match="one device"):
        bl._place(None, FakeTensor(0), FakeTensor(1))
    with pytest.raises(ValueError, match="contiguous"):
        bl._place(None, FakeTensor(0), FakeTensor(0, contiguous=False))
    guard = bl._place(None, FakeTensor(1), FakeTensor(1))  # not the current device
    assert isinstance(guard, torch.cuda.device) and guard.idx == 1

    class Stream:
        device = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="stream"):
        bl._place(Stream(), FakeTensor(1))


LA = dict(p_x=F, xdt=1, M=4, K=64, p_packed=F, p_gamma=F, N=64, p_A=F, p_B=F, p_scale=F, p_ids=F, L=2, r=8, p_y=F,
          ydt=1, p_ws=F, nws=BIG, flags=0, p_s=None)


@pytest.mark.parametrize("status,changes", [
    (BAD, [dict(p_x=None), dict(p_packed=None), dict(p_gamma=None), dict(p_A=None), dict(p_B=None), dict(p_scale=None),
           dict(p_ids=None), dict(p_y=None), dict(p_ws=None), dict(xdt=2), dict(ydt=5), dict(L=0), dict(r=0), dict(M=-1),
           dict(N=0), dict(K=0), dict(nws=0)]),
    (UNS, [dict(L=65536), dict(r=129), dict(M=1 << 30), dict(K=1 << 25), dict(xdt=0, flags=2),
           dict(K=((1 << 31) - 1) // 127)]),
    (ALN, [dict(p_x=F + 1), dict(p_packed=F + 8), dict(p_A=F + 2), dict(p_B=F + 8), dict(p_y=F + 2), dict(p_ids=F + 2),
           dict(p_scale=F + 2), dict(p_gamma=F + 2), dict(p_ws=F + 8)])])
def test_linear_adapters_refused_before_a_launch(L, status, changes):
    for change in changes:
        assert call(L.bitlinear_linear_adapters, LA, **change) == status, change


def test_linear_adapters_of_no_tokens_and_its_workspace(L):
    assert call(L.bitlinear_linear_adapters, LA, M=0, p_x=None, p_ids=None, p_y=None, p_ws=None, nws=0) == OK
    for K in (64, 61):
        fwd = L.bitlinear_forward_adapters_workspace_bytes(40, K, 63, 2, 8)
        need = L.bitlinear_linear_adapters_workspace_bytes(40, K, 63, 2, 8)
        assert need >= fwd + 40 * K + 2 * 4 * 40
        assert call(L.bitlinear_linear_adapters, LA, M=40, K=K, N=63, nws=need - 1) == BAD
    assert L.bitlinear_linear_adapters_workspace_bytes(4, 64, 64, 2, 129) == 0


def test_adapter_gradients_of_no_tokens_still_need_the_workspace(L):
    need = L.bitlinear_adapters_grad_workspace_bytes(0, 64, 64, 2, 8, 1)
    assert need > 0
    assert call(L.bitlinear_adapters_grad, AG, M=0, p_ws=None) == BAD
    assert call(L.bitlinear_adapters_grad, AG, M=0, nws=need - 1) == BAD
