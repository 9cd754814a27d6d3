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


def spread(sizes, start=A):
    """Addresses of buffers of those sizes, one behind the other without a gap
    (all of them multiples of 16 here)."""
    out = {}
    for name, size in sizes.items():
        out[name] = start
        start += size
    return out, start


def backward(gq, dtype=0, rows=6, N=144, ld=None, **at):
    size = 4 if dtype else 2
    ld = N if ld is None else ld
    sizes = dict(g=((rows - 1) * ld + N) * size, pre=rows * 2 * N * size, out=rows * 2 * N * size, q=rows * 2 * N,
                 scales=rows * 2 * -(-N // 128) * 4)
    p, _ = spread(sizes)
    p.update({k: v(p, sizes) if callable(v) else v for k, v in at.items()})
    return gq.lib().gq_gated_backward(p["g"], p["pre"], dtype, rows, N, ld, 0, p["out"], p["q"], p["scales"], 0, None)


BACKWARD = [
    dict(out=lambda p, s: p["g"]),
    dict(out=lambda p, s: p["pre"] + 16), dict(out=lambda p, s: p["pre"] + s["pre"] - 16),
    dict(out=lambda p, s: p["g"] + s["g"] - 16),
    dict(out=lambda p, s: p["g"] - s["out"] + 16),
    dict(q=lambda p, s: p["pre"]), dict(q=lambda p, s: p["g"] + 16), dict(q=lambda p, s: p["out"] + s["out"] - 16),
    dict(out=None, q=lambda p, s: p["pre"]),
    dict(scales=lambda p, s: p["g"] + 4), dict(scales=lambda p, s: p["pre"] + s["pre"] - 4),
    dict(scales=lambda p, s: p["out"] + 8), dict(scales=lambda p, s: p["q"] + s["q"] - 4),
    # g with a pitch: an output over its last row, and the gradient of the first half in pre, written in place
    dict(ld=4096, q=lambda p, s: p["g"] + 5 * 4096 * 2 + 272),
    dict(ld=288, g=lambda p, s: p["pre"], out=lambda p, s: p["pre"]),
    dict(dtype=1, out=lambda p, s: p["g"] + 16),
]


@pytest.mark.parametrize("kw", BACKWARD, ids=range(len(BACKWARD)))
def test_gated_backward(gq, kw):
    refused(gq, backward(gq, **kw))


def test_gated_backward_takes_what_does_not_overlap(gq):
    """Buffers right behind one another, out in pre's place, and outputs between
    the rows of g get past the checks (to the missing GPU here, so not on one)."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("addresses are made up")
    for kw in (dict(), dict(out=lambda p, s: p["pre"]), dict(dtype=1), dict(rows=1), dict(q=None, scales=lambda p, s: p["pre"]),
               dict(ld=4096, q=lambda p, s: p["g"] + 4 * 4096 * 2 + 288, scales=lambda p, s: p["g"] + 288),
               dict(out=lambda p, s: p["g"] - s["out"])):
        status = backward(gq, **kw)
        assert status not in (0, INVALID), kw
