"""The norm of a list of tensors and clipping against 64 bits.

A thread's partial sums are of eight squares each, four of them added in fp32:
at most 13 roundings of 2^-24 of a sum of non-negative terms, fp64 beyond; the
root halves that and is rounded to fp32 once: 7.5 * 2^-24 of the norm.  The
factor max_norm / norm adds one rounding, the product one (2^-24 each), then
the rounding to the tensor's type (bf16 2^-8, or half of its smallest step).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
NORM_TOL = 8 * 2.0 ** -24


@pytest.fixture(scope="module")
def gq():
    import __graft_entry__

    __graft_entry__.build()
    import fp8_quantization_moe_gb300 as m

    return m


def norm64(tensors):
    return math.sqrt(sum(float(t.double().square().sum()) for t in tensors))


def draw(gen, n, dtype, shift=0, scale=1.0):
    """n elements, the first `shift` elements behind a 16-byte boundary."""
    t = (scale * torch.randn(n + shift, device=DEV, generator=gen, dtype=torch.float64)).to(dtype)
    return t[shift:]


def like(t):
    """A copy that lies as t does in its 16 bytes: the order of the sum, and with
    it the norm's last bit, goes by the sizes and by that."""
    size = t.element_size()
    c = torch.empty(t.numel() + 16, dtype=t.dtype, device=DEV)
    at = (t.data_ptr() - c.data_ptr()) % 16 // size
    c = c[at:at + t.numel()]
    assert t.numel() == 0 or c.data_ptr() % 16 == t.data_ptr() % 16
    return c.copy_(t)


LISTS = [
    [(1, torch.float32, 0)],
    [(1, torch.bfloat16, 3)],
    [(0, torch.float32, 0), (7, torch.bfloat16, 1), (0, torch.bfloat16, 0)],
    [(8191, torch.bfloat16, 0), (8192, torch.bfloat16, 5), (8193, torch.bfloat16, 7)],
    [(8191, torch.float32, 1), (8192, torch.float32, 2), (8193, torch.float32, 3)],
    [(100003, torch.float32, 1), (5, torch.bfloat16, 2), (70001, torch.bfloat16, 3), (16, torch.float32, 0)],
    [(i * 37 % 1000 + 1, torch.float32 if i % 3 else torch.bfloat16, i % 4) for i in range(17)],
    [(i * 7919 % 5000, torch.float32 if i % 3 else torch.bfloat16, i % 4) for i in range(1025)],
    [(3, torch.bfloat16, i % 8) for i in range(2100)],
    [(40_000_003, torch.bfloat16, 1), (11_000_001, torch.float32, 1)],
    # the largest lists of one cluster, and just past them
    [(262144, torch.float32, 0)],
    [(262144, torch.float32, 3), (1, torch.bfloat16, 0)],
    [(32768, torch.bfloat16, i % 8) for i in range(16)],
    [(30000, torch.bfloat16, i % 8) for i in range(17)],
    [(70000, torch.float32, 1), (70001, torch.bfloat16, 3)],
]


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{s[0][0]}")
def test_norm_and_clip(gq, sizes):
    gen = torch.Generator(device=DEV).manual_seed(len(sizes))
    ts = [draw(gen, *s) for s in sizes]
    want = norm64(ts)
    norm = gq.grad_norm(ts)
    assert norm.dtype == torch.float32 and norm.dim() == 0
    assert abs(float(norm) - want) <= NORM_TOL * want
    for ratio in (0.37, 1.5):  # clipped, and left alone
        most = ratio * want
        factor = min(1.0, float(torch.tensor(most).float()) / want)
        outs = [torch.full((t.numel() + 16,), 7.0, dtype=t.dtype, device=DEV) for t in ts]
        views = [o[i % 3:i % 3 + t.numel()] for i, (o, t) in enumerate(zip(outs, ts))]
        before = [t.clone() for t in ts]
        got = gq.clip_grads(ts, most, out=views)
        assert torch.equal(got, norm)
        placed = [like(t) for t in ts]  # and in place
        assert torch.equal(gq.clip_grads(placed, most), norm)
        for i, (t, b, v, o, p) in enumerate(zip(ts, before, views, outs, placed)):
            assert torch.equal(t, b)  # the inputs of a call with outputs stay
            y = t.double() * factor
            step = 2.0 ** -8 if t.dtype == torch.bfloat16 else 2.0 ** -24
            off = (v.double() - y).abs() - ((1 + step) * 11 * 2.0 ** -24 + step) * y.abs()
            assert t.numel() == 0 or float(off.max()) <= 2.0 ** -134
            assert bool((o[:i % 3] == 7).all()) and bool((o[i % 3 + t.numel():] == 7).all())
            assert torch.equal(p, v)
            if ratio > 1:
                assert torch.equal(p, t)


def test_past_2_31_elements(gq):
    n = 2 ** 31 + 12_345
    t = torch.zeros(n + 1, dtype=torch.bfloat16, device=DEV)[1:]
    at = [0, 5, 2 ** 30, 2 ** 31 - 1, 2 ** 31, n - 1]
    t[at] = 2.0
    want = 2.0 * math.sqrt(len(at))
    assert abs(float(gq.grad_norm([t])) - want) <= NORM_TOL * want
    o = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    gq.clip_grads([t], want / 2, out=[o])  # a factor of a half
    assert o[at].tolist() == [1.0] * len(at) and int((o != 0).sum()) == len(at)
    gq.clip_grads([t], want / 2)
    assert torch.equal(t, o)


def test_norm_is_the_same_every_time(gq):
    gen = torch.Generator(device=DEV).manual_seed(3)
    ts = [draw(gen, 3_000_001, torch.bfloat16, 1), draw(gen, 777_777, torch.float32, 2)]
    first = gq.grad_norm(ts)
    for _ in range(20):
        assert torch.equal(gq.grad_norm(ts), first)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-12, 1.0, 1e18, 1e30, 2e37])
def test_ranges(gq, dtype, scale):
    """No square overflows or vanishes between the tensors' type and the norm."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    ts = [draw(gen, 50, dtype, 1, scale), draw(gen, 20000, dtype, 0, scale * 1e-3)]
    want = norm64(ts)
    norm = gq.grad_norm(ts)
    assert abs(float(norm) - want) <= NORM_TOL * want + 2.0 ** -149
    gq.clip_grads(ts, 1.0)
    after = norm64(ts)
    # each element off by half a step of its type: the norm by no more than that
    assert abs(after - min(1.0, want)) <= (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20) * after + 1e-40


def test_mixed_magnitudes(gq):
    """Neighbouring threads on both sides of the range that squares in fp32."""
    t = torch.zeros(20000, device=DEV)
    t[0], t[5], t[9000], t[19999] = 3e30, 4e30, 1e-30, 1e5
    assert abs(float(gq.grad_norm([t])) - 5e30) <= NORM_TOL * 5e30
    assert float(gq.grad_norm([torch.zeros(100, device=DEV)])) == 0.0
    u = torch.tensor([3e-30, 4e-30], device=DEV)
    assert abs(float(gq.grad_norm([u, torch.zeros(9, device=DEV)])) - 5e-30) <= NORM_TOL * 5e-30


def test_not_finite(gq):
    def clipped(v, most=1.0):
        t = torch.tensor([3.0, v, 4.0] + [0.5] * 30, device=DEV)
        return gq.clip_grads([t], most), t

    norm, t = clipped(float("nan"))
    assert math.isnan(float(norm)) and bool(t.isnan().all())
    norm, t = clipped(float("inf"))
    assert float(norm) == math.inf and math.isnan(float(t[1]))
    assert bool((t[torch.arange(33) != 1] == 0).all())
    norm, t = clipped(0.0, math.inf)
    assert bool((t[[0, 2]] == torch.tensor([3.0, 4.0], device=DEV)).all())
    t = torch.tensor([3.0, 4.0], device=DEV)
    gq.clip_grads([t], 0.0)
    assert t.tolist() == [0.0, 0.0]
    z = torch.zeros(5, device=DEV)
    assert float(gq.clip_grads([z], 0.0)) == 0.0 and bool((z == 0).all())
    assert float(gq.grad_norm([torch.zeros(0, device=DEV)])) == 0.0


def test_given_norm(gq):
    t = torch.arange(1.0, 101.0, device=DEV)
    norm = torch.tensor(50.0, device=DEV)
    u = t.clone()
    assert gq.clip_grads([u], 25.0, norm=norm) is norm
    assert torch.equal(u, t * 0.5)
    gq.clip_grads([u], 50.0, norm=norm)
    assert torch.equal(u, t * 0.5)
    gq.clip_grads([torch.zeros(0, device=DEV)], 1.0, norm=norm)
    assert float(norm) == 50.0


def test_no_tensors(gq):
    """The C call takes an empty list: its norm is 0."""
    norm = torch.full((), 7.0, device=DEV)
    assert gq.lib().gq_grad_norm(None, None, None, 0, norm.data_ptr(), None, 0, None) == 0
    assert gq.lib().gq_clip_grads(None, None, None, None, 0, 1.0, None, norm.data_ptr(), None, 0, None) == 0
    torch.cuda.synchronize()
    assert float(norm) == 0.0


def test_norm_counts_a_tensor_as_often_as_it_comes(gq):
    t = torch.full((1000,), 2.0, device=DEV)
    assert abs(float(gq.grad_norm([t, t, t[10:20]])) - math.sqrt(4 * 2010)) <= NORM_TOL * 90


def test_overlaps_are_refused(gq):
    t = torch.ones(1000, device=DEV)
    o = torch.ones(1000, device=DEV)
    for grads, out in [([t, t], None), ([t[:600], t[500:]], None), ([t[:500], t[500:]], [o[:500], o[499:999]]),
                       ([t[:500]], [t[1:501]]), ([t[:500], t[500:]], [o[:500], t[:500]])]:
        with pytest.raises(gq.GQError, match="overlap"):
            gq.clip_grads(grads, 0.5, out=out)
    assert bool((t == 1).all())
    half = t[:500], t[500:]
    gq.clip_grads(list(half), 0.5, out=[half[0], o[:500]])
    assert not bool((half[0] == 1).any()) and bool((half[1] == 1).all()) and torch.equal(o[:500], half[0])


def test_refusals(gq):
    t = torch.ones(10, device=DEV)
    for bad, match in [(t, "list"), ([], "no tensors"), ([t.cpu()], "CUDA"), ([t.half()], "bfloat16 or float32"),
                       ([torch.ones(4, 4, device=DEV).t()], "contiguous"), ([t, None], "CUDA")]:
        with pytest.raises(ValueError, match=match):
            gq.grad_norm(bad)
        with pytest.raises(ValueError, match=match):
            gq.clip_grads(bad, 1.0)
    for most in (-1.0, math.nan):
        with pytest.raises(ValueError, match="max_norm"):
            gq.clip_grads([t], most)
    for out in ([], [t[:9]], [t.bfloat16()], [t, t]):
        with pytest.raises(ValueError, match="types and sizes"):
            gq.clip_grads([t], 1.0, out=out)
    with pytest.raises(ValueError, match="norm"):
        gq.clip_grads([t], 1.0, norm=torch.ones(1, device=DEV))


def test_streams_and_graphs(gq):
    gen = torch.Generator(device=DEV).manual_seed(8)
    ts = [draw(gen, 300_001, torch.bfloat16, 1), draw(gen, 5000, torch.float32)]
    want = [like(t) for t in ts]
    norm = gq.clip_grads(want, 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [like(t) for t in ts]
    side.wait_stream(torch.cuda.current_stream())
    n1 = gq.clip_grads(got, 1.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(n1, norm) and all(torch.equal(a, b) for a, b in zip(got, want))
    work, outs = [like(t) for t in ts], [torch.empty_like(t) for t in ts]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n2 = gq.clip_grads(work, 1.0, out=outs)
    with torch.cuda.graph(other):
        n3 = gq.grad_norm(work)
    for k in (1.0, 0.25):  # new values in the same tensors
        for w, t in zip(work, ts):
            w.copy_(t * k)
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        assert torch.equal(n2, n3)
        if k == 1.0:
            assert torch.equal(n2, norm) and all(torch.equal(a, b) for a, b in zip(outs, want))
        else:
            assert abs(float(n2) - 0.25 * float(norm)) <= 2.0 ** -7 * float(norm)
