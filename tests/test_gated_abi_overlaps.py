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


def product(gq, form, M=5, N=144, K=272, E=3, **at):
    n, k = -(-N // 128), -(-K // 128)
    weights = dict(qb=E * 2 * N * K, sb=E * 2 * n * k * 4, offs=E * 4 + 4)
    if form == "mm":
        sizes = dict(qa=M * K, sa=M * k * 4 + 4, **weights, out=M * N * 2, q=M * N, scales=M * n * 4, pre=M * 2 * N * 2)
    else:
        sizes = dict(qa=M * 2 * N, sa=M * 2 * n * 4, **weights, out=M * K * 2)
    sizes = {name: -(-size // 16) * 16 for name, size in sizes.items()}
    p, _ = spread(sizes)
    p.update({name: v(p, sizes) if callable(v) else v for name, v in at.items()})
    a = p["qa"], p["sa"], M, p["qb"], p["sb"], N, K
    if form == "mm":
        return gq.lib().gq_grouped_gated_mm(*a, 0, p["offs"], E, p["out"], p["q"], p["scales"], p["pre"], 0, None)
    return gq.lib().gq_grouped_gated_grad(*a, p["offs"], E, p["out"], None)


@pytest.mark.parametrize("which", ["qa", "sa", "qb", "sb", "offs"])
def test_products_refuse_outputs_over_inputs(gq, which):
    for form in ("mm", "grad"):
        for name in ("out", "q", "scales", "pre") if form == "mm" else ("out",):
            refused(gq, product(gq, form, **{name: lambda p, s: p[which]}))
            refused(gq, product(gq, form, **{name: lambda p, s: p[which] - s[name] + 16}))


def test_products_refuse_outputs_over_outputs(gq):
    names = ("out", "q", "scales", "pre")
    for a in names:
        for b in names:
            if a != b:
                refused(gq, product(gq, "mm", **{a: lambda p, s: p[b]}))
                refused(gq, product(gq, "mm", **{a: lambda p, s: p[b] + s[b] // 32 * 16}))


def test_products_take_what_does_not_overlap(gq):
    import torch

    if torch.cuda.is_available():
        pytest.skip("addresses are made up")
    for form, kw in (("mm", {}), ("grad", {}), ("mm", dict(out=None)), ("mm", dict(pre=None)),
                     ("mm", dict(q=None, scales=lambda p, s: p["out"]))):  # scales of no rows are not written
        assert product(gq, form, **kw) not in (0, INVALID)
