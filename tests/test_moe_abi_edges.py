"""Host-side checks of the MoE-layer operators that empty extents could let
through: every refusal comes before any CUDA call (CPU only)."""
import pytest

# Fake device addresses: never dereferenced.
A16 = 0x10000


@pytest.fixture(scope="module")
def gq():
    import __graft_entry__

    __graft_entry__.build()
    import fp8_quantization_moe_gb300 as m

    return m


@pytest.mark.parametrize("args,status", [
    # g, y, dtype, rows, H, pos, weights, tokens, top_k, dy, dweights
    ((None, None, 0, 0, 64, A16, A16, 4, 2, None, A16), 1),  # no rows: g is read all the same
    ((None, A16, 1, 0, 64, A16, A16, 4, 2, A16, A16), 1),
    ((A16, None, 0, 1, 64, A16, A16, 4, 2, A16, A16), 1),
    ((A16, A16, 0, 1, 64, A16, A16, 4, 2, None, A16), 1),
    ((None, None, 0, 0, 64, None, None, 0, 2, None, None), 0),  # no tokens: nothing is read
])
def test_combine_backward_refuses_a_missing_gradient(gq, args, status):
    assert gq.lib().gq_moe_combine_backward(*args, None) == status
