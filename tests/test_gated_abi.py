"""Host-side checks of the gated block and of the gradient norm: every refusal
comes before any CUDA call (CPU only)."""
import ctypes
import math

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


def mm(**kw):
    a = dict(qa=A16, sa=A16, M=4, qb=A16, sb=A16, N=32, K=64, act=0, offs=A16, E=2, out=A16, q=A16, scales=A16,
             pre=A16, flags=0)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 1), (dict(N=-16), 1), (dict(K=-16), 1), (dict(act=2), 1), (dict(act=-1), 1), (dict(E=0), 1),
    (dict(E=1025), 2), (dict(M=1 << 31), 2), (dict(N=(1 << 22) + 16), 2), (dict(K=(1 << 22) + 16), 2),
    (dict(N=1 << 21, E=512), 2), (dict(N=40), 2), (dict(K=40), 2), (dict(K=0), 2), (dict(flags=2), 1),
    (dict(qa=None), 1), (dict(sa=None), 1), (dict(qb=None), 1), (dict(sb=None), 1), (dict(offs=None), 1),
    (dict(out=None, q=None), 1), (dict(scales=None), 1), (dict(qa=BAD), 1), (dict(qb=BAD), 1), (dict(out=BAD), 1),
    (dict(q=BAD), 1), (dict(pre=BAD), 1), (dict(sa=ODD), 1), (dict(sb=ODD), 1), (dict(scales=ODD), 1),
    (dict(offs=ODD), 1),
    (dict(M=0, qa=None, sa=None, out=None, q=None, scales=None, pre=None), 0), (dict(N=0, qb=None), 0),
])
def test_grouped_gated_mm(gq, kw, status):
    assert gq.lib().gq_grouped_gated_mm(*mm(**kw), None) == status


def grad(**kw):
    a = dict(qd=A16, sd=A16, M=4, qb=A16, sb=A16, N=32, K=64, offs=A16, E=2, out=A16)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 1), (dict(E=0), 1), (dict(E=1025), 2), (dict(M=1 << 31), 2), (dict(N=(1 << 22) + 16), 2),
    (dict(N=1 << 21, E=512), 2), (dict(N=40), 2), (dict(K=40), 2), (dict(N=0), 2), (dict(qd=None), 1),
    (dict(sd=None), 1), (dict(qb=None), 1), (dict(sb=None), 1), (dict(offs=None), 1), (dict(out=None), 1),
    (dict(qd=BAD), 1), (dict(qb=BAD), 1), (dict(out=BAD), 1), (dict(sd=ODD), 1), (dict(sb=ODD), 1),
    (dict(offs=ODD), 1), (dict(M=0, qd=None, out=None), 0), (dict(K=0, qb=None, out=None), 0),
])
def test_grouped_gated_grad(gq, kw, status):
    assert gq.lib().gq_grouped_gated_grad(*grad(**kw), None) == status


def backward(**kw):
    a = dict(g=A16, pre=A16, dtype=0, rows=4, N=32, ld=32, act=0, out=A16, q=A16, scales=A16, flags=0)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 1), (dict(rows=-1), 1), (dict(N=-16), 1), (dict(act=2), 1), (dict(flags=4), 1), (dict(N=24, ld=24), 2),
    (dict(ld=16), 1), (dict(ld=36), 1), (dict(rows=1 << 31), 2), (dict(N=(1 << 22) + 16, ld=(1 << 22) + 16), 2),
    (dict(g=None), 1), (dict(pre=None), 1), (dict(out=None, q=None), 1), (dict(scales=None), 1), (dict(g=BAD), 1),
    (dict(pre=BAD), 1), (dict(out=BAD), 1), (dict(q=BAD), 1), (dict(scales=ODD), 1),
    (dict(rows=0, g=None, pre=None, out=None), 0), (dict(N=0, ld=0, g=None), 0),
])
def test_gated_backward(gq, kw, status):
    assert gq.lib().gq_gated_backward(*backward(**kw), None) == status


def lists(ptrs, sizes, dtypes):
    n = len(ptrs)
    return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*dtypes), n


TENSORS = [
    (([A16], [-1], [0]), 1), (([A16], [4], [2]), 1), (([None], [4], [0]), 1), (([A16 + 1], [4], [0]), 1),
    (([ODD], [4], [1]), 1), (([A16], [(1 << 42) + 1], [0]), 2), (([A16, A16], [1 << 41, (1 << 41) + 1], [0, 0]), 2),
    (([A16], [1 << 62], [1]), 2),
]


@pytest.mark.parametrize("t,status", TENSORS)
def test_grad_norm_lists(gq, t, status):
    p, s, d, n = lists(*t)
    size = 1 << 20
    assert gq.lib().gq_grad_norm(p, s, d, n, A16, A16, size, None) == status
    assert gq.lib().gq_clip_grads(p, None, s, d, n, 1.0, None, A16, A16, size, None) == status


def test_grad_norm_refusals(gq):
    L = gq.lib()
    p, s, d, n = lists([A16], [1 << 20], [0])
    bytes_of = L.gq_grad_norm_workspace_bytes
    size = bytes_of(s, d, n)
    assert size > 0 and size % 8 == 0
    assert bytes_of(s, d, 0) == 0 and bytes_of(s, d, -1) == 0 and bytes_of(s, d, (1 << 20) + 1) == 0
    assert bytes_of(None, d, n) == 0 and bytes_of(s, None, n) == 0
    # one cluster: 16 tensors, 1 MiB in chunks of 16 KB
    few = lists([A16] * 16, [1 << 13] * 16, [1] * 16)
    assert bytes_of(few[1], few[2], 16) == 0
    assert bytes_of(*lists([A16], [1 << 19], [0])[1:]) == 0 and bytes_of(*lists([A16], [(1 << 19) + 1], [0])[1:]) > 0
    assert bytes_of(*lists([A16] * 17, [1] * 17, [1] * 17)[1:]) > 0
    assert bytes_of(*lists([A16], [0], [0])[1:]) > 0
    assert L.gq_grad_norm(p, s, d, -1, A16, A16, size, None) == 1
    assert L.gq_grad_norm(None, s, d, n, A16, A16, size, None) == 1
    assert L.gq_grad_norm(p, None, d, n, A16, A16, size, None) == 1
    assert L.gq_grad_norm(p, s, None, n, A16, A16, size, None) == 1
    assert L.gq_grad_norm(p, s, d, (1 << 20) + 1, A16, A16, size, None) == 2
    assert L.gq_grad_norm(p, s, d, n, None, A16, size, None) == 1
    assert L.gq_grad_norm(p, s, d, n, ODD, A16, size, None) == 1
    assert L.gq_grad_norm(p, s, d, n, A16, None, size, None) == 1
    assert L.gq_grad_norm(p, s, d, n, A16, A16 + 16, size, None) == 1
    assert L.gq_grad_norm(p, s, d, n, A16, A16, size - 1, None) == 1
    for most in (-1.0, math.nan):
        assert L.gq_clip_grads(p, None, s, d, n, most, None, A16, A16, size, None) == 1
    assert L.gq_clip_grads(p, None, s, d, n, 1.0, None, None, A16, size, None) == 1
    assert L.gq_clip_grads(p, None, s, d, n, 1.0, ODD, None, None, 0, None) == 1
    assert L.gq_clip_grads(p, lists([ODD + 1], [4], [0])[0], s, d, n, 1.0, None, A16, A16, size, None) == 1
    assert L.gq_clip_grads(p, lists([None], [4], [0])[0], s, d, n, 1.0, None, A16, A16, size, None) == 1


@pytest.mark.parametrize("grads,outs,sizes", [
    ([A16, A16], None, [8, 8]),                             # twice the same
    ([A16, A16 + 14], None, [8, 8]),                        # the last element is the other's first
    ([A16 + 14, A16], None, [8, 8]),
    ([A16, A16 + 64], [A16 + 128, A16 + 130], [8, 8]),      # two outputs
    ([A16], [A16 + 2], [8]),                                # an output over a part of its own tensor
    ([A16, A16 + 64], [A16 + 128, A16], [8, 8]),            # over another tensor
    ([A16, A16 + 16, A16 + 32], [A16, A16 + 64, A16 + 20], [8, 8, 8]),
])
def test_overlaps(gq, grads, outs, sizes):
    n = len(grads)
    p, s, d, _ = lists(grads, sizes, [0] * n)
    o = None if outs is None else (ctypes.c_void_p * n)(*outs)
    size = 1 << 20
    assert gq.lib().gq_clip_grads(p, o, s, d, n, 1.0, None, A16, A16, size, None) == 1
    assert b"overlap" in gq.lib().gq_last_error()


def test_python_refusals_without_a_gpu(gq):
    t = torch.zeros(4, 4)
    for call in (lambda: gq.grad_norm([t]), lambda: gq.clip_grads([t], 1.0), lambda: gq.gated_backward(t, t),
                 lambda: gq.grouped_gated_mm(t, t, t, t, t), lambda: gq.grouped_gated_grad(t, t, t, t, t)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
