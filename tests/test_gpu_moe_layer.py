"""The operators together: the example's MoE layer, forward and backward,
against the same layer in 64 bits.

The difference is e4m3 rounding.  A rounding to three mantissa bits is off by
at most 2^-4 of a value, about 2^-4 / sqrt(3) / sqrt(2) = 2.6 % in the root mean square
over a binade; a product of two rounded operands by sqrt(2) times that, 3.6 %
of its norm, as the errors of its terms are independent.  Two products in a
row (out) give 1.4 times that again and the gate's derivatives at most another
factor of two: 0.11 bounds every result.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location(
        "moe_layer_example", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,top_k,experts,hidden,width,local", [
    (300, 4, 8, 512, 256, None),     # ordinary
    (1, 2, 8, 256, 144, None),       # one token
    (513, 3, 16, 272, 400, 5),       # most slots belong to experts held elsewhere
    (2000, 2, 4, 640, 1040, None),   # groups of a thousand rows
])
def test_moe_layer(example, tokens, top_k, experts, hidden, width, local):
    errors = example.relative_errors(
        example.make_inputs(tokens, top_k, experts, hidden, width, seed=tokens, local=local))
    assert all(e <= 0.11 for e in errors.values()), errors
