"""Calls that the backward pass and the adapters refuse before anything is launched (no GPU)."""
import pytest

from ternary_weight_linear_04_b200 import _lib
from ternary_weight_linear_04_b200 import build as libbuild
from test_train_abi import AG, BAD, F, FA, GI, GW, LA, RN, UNS, call


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return _lib.lib()


def test_more_tokens_than_the_projection_takes(L):
    """Its grid holds 65535 tiles of 256 tokens: refused before u is launched, and by the queries."""
    most = 65535 * 256
    for change in (dict(M=most + 1, K=16, N=8), dict(M=(1 << 30) - 1, K=16, N=8), dict(M=4, K=((1 << 31) - 1) // 127)):
        assert call(L.bitlinear_forward_adapters, FA, **change) == UNS
        assert call(L.bitlinear_linear_adapters, LA, **change) == UNS
        sizes = change["M"], change["K"], change.get("N", 64), 2, 8
        assert L.bitlinear_forward_adapters_workspace_bytes(*sizes) == 0
        assert L.bitlinear_linear_adapters_workspace_bytes(*sizes) == 0
    assert L.bitlinear_forward_adapters_workspace_bytes(most, 16, 8, 2, 8) > 0


G = 1 << 30  # far from F


@pytest.mark.parametrize("name,base,out,inputs", [
    ("grad_input", GI, "p_dx", ["p_dy", "p_packed", "p_gamma"]),
    ("grad_weight", GW, "p_dw", ["p_dy", "p_xq", "p_eta"]),
    ("rmsnorm_grad", RN, "p_dx", ["p_dn", "p_xq", "p_eta", "p_rstd"]),
    ("forward_adapters", FA, "p_y", ["p_xq", "p_eta", "p_xsum", "p_packed", "p_gamma", "p_A", "p_B", "p_scale", "p_ids"]),
    ("linear_adapters", LA, "p_y", ["p_x", "p_packed", "p_gamma", "p_A", "p_B", "p_scale", "p_ids"]),
    ("adapters_grad", AG, "p_dx", ["p_dy", "p_xq", "p_eta", "p_packed", "p_gamma", "p_A", "p_B", "p_scale", "p_ids"]),
    ("adapters_grad", AG, "p_dA", ["p_dy", "p_A", "p_B"]),
    ("adapters_grad", AG, "p_dB", ["p_dy", "p_A", "p_B"])])
def test_an_output_on_an_input_is_refused(L, name, base, out, inputs):
    """Whether it begins at the input, inside it, or ends inside it."""
    fn = getattr(L, "bitlinear_" + name)
    spread = {k: (i + 2) * G if v == F else v for i, (k, v) in enumerate(base.items())}
    for p in inputs:
        for off in (0, 16, -16) if p != "p_gamma" else (0, -16):
            if name == "rmsnorm_grad" and p == "p_dn" and off == 0:
                continue  # in place
            at = spread[p] + (off if p not in ("p_eta", "p_rstd", "p_xsum", "p_ids", "p_scale") else min(off, 0))
            assert call(fn, spread, **{out: at}) == BAD, (p, off)
    if name == "rmsnorm_grad":
        assert call(fn, spread, p_dx=spread["p_dn"], dxdt=0) == BAD  # of another type
        assert call(fn, spread, p_dx=spread["p_dn"] + 2) == BAD


def test_tiles_of_refused_sizes(L):
    tile = L.bitlinear_tile_tokens
    assert tile(0, 300, 130, 11003, 148) == 256 and tile(1, 300, 3200, 70, 148) == 128
    assert tile(0, 0, 64, 64, 148) == tile(0, 65535 * 256 + 1, 16, 8, 148) == tile(0, 4, 64, 64, 0) == 0
    assert tile(1, 0, 64, 64, 148) == tile(1, 1 << 30, 64, 64, 148) == tile(1, 4, 0, 64, 148) == 0
