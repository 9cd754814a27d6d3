"""Host-side checks of the MoE-layer operators: every refusal comes before
any CUDA call (CPU only)."""
import pytest
import torch

# Fake device addresses: never dereferenced.
A16 = 0x10000
BAD = 0x10008
ODD = 0x10002


@pytest.fixture(scope="module")
def gq():
    import __graft_entry__

    __graft_entry__.build()
    import fp8_quantization_moe_gb300 as m

    return m


@pytest.mark.parametrize("args,status", [
    # ids, id_bytes, tokens, top_k, n_experts, offs, pos, token
    ((A16, 4, -1, 2, 4, A16, A16, A16), 1),
    ((A16, 4, 8, 0, 4, A16, A16, A16), 1),
    ((A16, 2, 8, 2, 4, A16, A16, A16), 1),
    ((A16, 4, 8, 2, 0, A16, A16, A16), 1),
    ((A16, 4, 8, 2, 1025, A16, A16, A16), 2),
    ((A16, 4, 1 << 30, 2, 4, A16, A16, A16), 2),
    ((None, 4, 8, 2, 4, A16, A16, A16), 1),
    ((A16, 4, 8, 2, 4, None, A16, A16), 1),
    ((A16, 4, 8, 2, 4, A16, None, A16), 1),
    ((A16, 4, 8, 2, 4, A16, A16, None), 1),
    ((A16 + 4, 8, 8, 2, 4, A16, A16, A16), 1),
    ((A16, 4, 8, 2, 4, A16, ODD, A16), 1),
])
def test_sort_refusals(gq, args, status):
    assert gq.lib().gq_moe_sort(*args, None) == status
    assert gq.lib().gq_last_error() != b""


@pytest.mark.parametrize("args,status", [
    # x, tokens, row_bytes, ld_bytes, pos, top_k, out_rows, out
    ((A16, -1, 64, 64, A16, 2, 8, A16), 1),
    ((A16, 4, 64, 64, A16, 0, 8, A16), 1),
    ((A16, 4, -64, 64, A16, 2, 8, A16), 1),
    ((A16, 4, 64, 48, A16, 2, 8, A16), 1),
    ((A16, 4, 64, 72, A16, 2, 8, A16), 1),
    ((A16, 4, 72, 80, A16, 2, 8, A16), 2),
    ((A16, 4, 1 << 23, 1 << 23, A16, 2, 8, A16), 2),
    ((A16, 4, 64, 64, A16, 2, -1, A16), 1),
    ((None, 4, 64, 64, A16, 2, 8, A16), 1),
    ((A16, 4, 64, 64, None, 2, 8, A16), 1),
    ((A16, 4, 64, 64, A16, 2, 8, None), 1),
    ((BAD, 4, 64, 64, A16, 2, 8, A16), 1),
    ((A16, 4, 64, 64, A16, 2, 8, BAD), 1),
    ((None, 0, 64, 64, None, 2, 0, None), 0),
])
def test_dispatch_refusals(gq, args, status):
    assert gq.lib().gq_moe_dispatch(*args, None) == status


@pytest.mark.parametrize("args,status", [
    # y, dtype, rows, H, pos, weights, tokens, top_k, out
    ((A16, 2, 8, 64, A16, A16, 4, 2, A16), 1),
    ((A16, 0, -8, 64, A16, A16, 4, 2, A16), 1),
    ((A16, 0, 8, 60, A16, A16, 4, 2, A16), 2),
    ((A16, 1, 8, 6, A16, A16, 4, 2, A16), 2),
    ((A16, 0, 8, 64, A16, A16, 4, 0, A16), 1),
    ((None, 0, 8, 64, A16, A16, 4, 2, A16), 1),
    ((A16, 0, 8, 64, None, A16, 4, 2, A16), 1),
    ((A16, 0, 8, 64, A16, A16, 4, 2, None), 1),
    ((BAD, 0, 8, 64, A16, A16, 4, 2, A16), 1),
    ((A16, 0, 8, 64, A16, ODD, 4, 2, A16), 1),
    ((None, 0, 0, 64, None, None, 0, 2, None), 0),
])
def test_combine_refusals(gq, args, status):
    assert gq.lib().gq_moe_combine(*args, None) == status


@pytest.mark.parametrize("args,status", [
    # g, y, dtype, rows, H, pos, weights, tokens, top_k, dy, dweights
    ((A16, A16, 3, 8, 64, A16, A16, 4, 2, A16, A16), 1),
    ((A16, A16, 0, 8, 68, A16, A16, 4, 2, A16, A16), 2),
    ((A16, A16, 0, 8, 64, A16, None, 4, 2, A16, A16), 1),
    ((A16, A16, 0, 8, 64, A16, A16, 4, 2, A16, None), 1),
    ((None, A16, 0, 8, 64, A16, A16, 4, 2, A16, A16), 1),
    ((A16, A16, 0, 8, 64, A16, A16, 4, 2, None, A16), 1),
    ((A16, BAD, 0, 8, 64, A16, A16, 4, 2, A16, A16), 1),
    ((A16, A16, 0, 8, 64, A16, A16, 1 << 31, 1, A16, A16), 2),
    ((None, None, 0, 0, 64, None, None, 0, 2, None, None), 0),
])
def test_combine_backward_refusals(gq, args, status):
    assert gq.lib().gq_moe_combine_backward(*args, None) == status


@pytest.mark.parametrize("args,status", [
    # x, dtype, rows, K, ld, pos, top_k, out_rows, out, scales, flags
    ((A16, 0, 4, 64, 64, None, 1, 4, A16, A16, 2), 1),
    ((A16, 2, 4, 64, 64, None, 1, 4, A16, A16, 0), 1),
    ((A16, 0, 4, 72, 72, None, 1, 4, A16, A16, 0), 2),
    ((A16, 0, 4, 64, 48, None, 1, 4, A16, A16, 0), 1),
    ((A16, 0, 4, 64, 68, None, 1, 4, A16, A16, 0), 1),
    ((A16, 0, 4, 64, 64, A16, 0, 4, A16, A16, 0), 1),
    ((A16, 0, 4, 64, 64, A16, 2, -1, A16, A16, 0), 1),
    ((A16, 0, 4, 64, 64, ODD, 2, 8, A16, A16, 0), 1),
    ((None, 0, 4, 64, 64, None, 1, 4, A16, A16, 0), 1),
    ((A16, 0, 4, 64, 64, None, 1, 4, None, A16, 0), 1),
    ((A16, 0, 4, 64, 64, None, 1, 4, A16, None, 0), 1),
    ((BAD, 0, 4, 64, 64, None, 1, 4, A16, A16, 0), 1),
    ((None, 0, 0, 64, 64, None, 1, 0, None, None, 0), 0),
])
def test_block_rows_refusals(gq, args, status):
    assert gq.lib().gq_fp8_block_rows(*args, None) == status


@pytest.mark.parametrize("args,status", [
    # w, dtype, E, N, K, out, scales, flags
    ((A16, 0, 0, 64, 64, A16, A16, 0), 1),
    ((A16, 0, 2, -1, 64, A16, A16, 0), 1),
    ((A16, 0, 2, 64, 40, A16, A16, 0), 2),
    ((A16, 9, 2, 64, 64, A16, A16, 0), 1),
    ((A16, 0, 2, 64, 64, A16, A16, 4), 1),
    ((A16, 0, 2, 1 << 31, 64, A16, A16, 0), 2),
    ((A16, 0, 1 << 20, 1 << 20, 1 << 10, A16, A16, 0), 2),
    ((A16, 0, 2, 64, 64, BAD, A16, 0), 1),
    ((None, 0, 2, 64, 64, A16, A16, 0), 1),
    ((None, 0, 2, 0, 64, None, None, 0), 0),
])
def test_block_tiles_refusals(gq, args, status):
    assert gq.lib().gq_fp8_block_tiles(*args, None) == status


@pytest.mark.parametrize("args,status", [
    # qa, sa, M, qb, sb, N, K, transpose_b, offs, n_groups, out
    ((A16, A16, -1, A16, A16, 64, 64, 0, A16, 2, A16), 1),
    ((A16, A16, 8, A16, A16, 64, 64, 2, A16, 2, A16), 1),
    ((A16, A16, 8, A16, A16, 64, 64, 0, A16, 0, A16), 1),
    ((A16, A16, 8, A16, A16, 64, 64, 0, A16, 1025, A16), 2),
    ((A16, A16, 8, A16, A16, 72, 64, 0, A16, 2, A16), 2),
    ((A16, A16, 8, A16, A16, 64, 40, 0, A16, 2, A16), 2),
    ((A16, A16, 8, A16, A16, 1 << 23, 64, 0, A16, 2, A16), 2),
    ((A16, A16, 8, A16, A16, 1 << 22, 64, 0, A16, 1024, A16), 2),
    ((A16, A16, 8, A16, A16, 64, 0, 0, A16, 2, A16), 2),
    ((None, A16, 8, A16, A16, 64, 64, 0, A16, 2, A16), 1),
    ((A16, None, 8, A16, A16, 64, 64, 0, A16, 2, A16), 1),
    ((A16, A16, 8, BAD, A16, 64, 64, 0, A16, 2, A16), 1),
    ((A16, A16, 8, A16, ODD, 64, 64, 0, A16, 2, A16), 1),
    ((A16, A16, 8, A16, A16, 64, 64, 0, None, 2, A16), 1),
    ((A16, A16, 8, A16, A16, 64, 64, 0, A16, 2, None), 1),
    ((None, None, 0, None, None, 64, 64, 0, None, 2, None), 0),
    ((None, None, 8, None, None, 0, 64, 0, None, 2, None), 0),
])
def test_grouped_mm_refusals(gq, args, status):
    assert gq.lib().gq_grouped_mm(*args, None) == status


def test_binding_refuses_host_tensors(gq):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    w = torch.zeros((4, 2))
    for call in (lambda: gq.sort_tokens(ids, 4), lambda: gq.dispatch(x, ids),
                 lambda: gq.dispatch_block(x, ids), lambda: gq.block_rows(x),
                 lambda: gq.block_tiles(x[None]), lambda: gq.combine(x, ids, w),
                 lambda: gq.combine_backward(x, x, ids, w),
                 lambda: gq.grouped_mm(x, w, x[None], w[None], ids[:, 0])):
        with pytest.raises(ValueError):
            call()
