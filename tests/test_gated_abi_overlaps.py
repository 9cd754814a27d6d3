"""Host-side refusals of buffers of the gated block's calls and of clipping that
overlap (CPU only: every refusal comes before any CUDA call)."""
import ctypes

import pytest

# Fake device addresses: never dereferenced.
A = 0x100000
INVALID = 1


@pytest.fixture(scope="module")
def gq():
    import __graft_entry__

    __graft_entry__.build()
    import fp8_quantization_moe_gb300 as m

    return m


def refused(gq, status):
    assert status == INVALID
    assert b"overlap" in gq.lib().gq_last_error()


def clip(gq, grads, outs, sizes, dtypes, given, norm):
    n = len(grads)
    p = (ctypes.c_void_p * n)(*grads)
    o = None if outs is None else (ctypes.c_void_p * n)(*outs)
    s, d = (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*dtypes)
    return gq.lib().gq_clip_grads(p, o, s, d, n, 1.0, given, norm, 0x800000, 1 << 20, None)


@pytest.mark.parametrize("grads,outs,sizes,dtypes,given,norm", [
    ([A], None, [8], [1], A, None),                                # a given norm inside a tensor that is written
    ([A], None, [8], [1], A + 28, None),                           # its last element
    ([A, A + 0x1000], None, [8, 7], [1, 0], A + 0x100C, None),     # half of it over a bf16 tensor's last element
    ([A], [A + 0x1000], [8], [1], A + 0x1004, None),               # inside an output
    ([A], [A], [8], [1], A + 4, None),
    ([A], None, [8], [1], None, A + 4),                            # the norm written into a tensor
    ([A], [A + 0x1000], [8], [1], None, A + 4),                    # that is only read
    ([A], [A + 0x1000], [8], [1], None, A + 0x1000),               # and into an output
    ([A + 0x1000, A], [A + 0x2000, A + 0x3000], [8, 1 << 20], [1, 1], None, A + 4 * ((1 << 20) - 1)),
])
def test_norm_inside_a_tensor(gq, grads, outs, sizes, dtypes, given, norm):
    refused(gq, clip(gq, grads, outs, sizes, dtypes, given, norm))
