"""The package's own names are the binding's."""
import pytest

import ternary_weight_linear_04_b200 as pkg
from ternary_weight_linear_04_b200 import bitlinear as bl


@pytest.mark.parametrize("name", ["pack_weights", "quant_act", "rmsnorm_quant_act", "forward", "linear", "grad_input",
                                  "grad_weight", "rmsnorm_grad", "forward_adapters", "linear_adapters", "adapters_grad",
                                  "BitLinear"])
def test_name(name):
    assert getattr(pkg, name) is getattr(bl, name)


def test_an_unknown_name():
    with pytest.raises(AttributeError):
        pkg.backward
