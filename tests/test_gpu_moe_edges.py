"""The MoE-layer operators at their edges: what the plain sizes do not reach."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def gq():
    import __graft_entry__

    __graft_entry__.build()
    import fp8_quantization_moe_gb300 as m

    return m


def randn(seed, *shape, dtype=torch.bfloat16):
    r = np.random.default_rng(seed)
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(DEV).to(dtype)


# ------------------------------------------------------------------ slots --

def test_dispatch_block_refuses_tokens_without_slots(gq):
    """An empty position array has no address; it must not be taken for the
    call without positions, which writes a row per token."""
    x = randn(1, 4, 64)
    pos = torch.empty(4, 0, dtype=torch.int32, device=DEV)
    out = torch.full((4, 64), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((4, 1), -3.0, device=DEV)
    with pytest.raises(ValueError):
        gq.dispatch_block(x, pos, out=out, scales=scales)
    assert (out == 0x5A).all() and (scales == -3.0).all()
    with pytest.raises(ValueError):
        gq.dispatch_block(x, pos)
    q, s = gq.dispatch_block(x[:0], pos[:0])  # no tokens either: nothing to do
    assert q.shape == (0, 64) and s.shape == (0, 1)
