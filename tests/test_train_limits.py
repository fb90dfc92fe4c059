"""Calls that the backward pass and the adapters refuse before anything is launched (no GPU)."""
import pytest

from ternary_weight_linear_04_b200 import _lib
from ternary_weight_linear_04_b200 import build as libbuild
from test_train_abi import BAD, F, FA, LA, OK, UNS, call  # noqa: F401


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
