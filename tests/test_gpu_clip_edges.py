"""Clipping at the ends of fp32's range.

Bounds: the norm is within 7.5 * 2^-24 and fp32, max_norm is given as fp32, the
factor and the product add a rounding each, 2^-24: 11 * 2^-24 of the value.  The
result is rounded to its type once more, by half a step at most: 2^-24 (fp32) or 2^-8
(bf16) of the value, and below the type's normal values half of its smallest step,
2^-150 or 2^-134.
"""
import math

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


def norm64(tensors):
    return math.sqrt(sum(float(t.double().square().sum()) for t in tensors))


def tensors(dtype, scale, long):
    """A few elements of that size, all tensors in one cluster's launch or in many blocks'."""
    gen = torch.Generator(device=DEV).manual_seed(7)
    head = scale * (0.5 + torch.rand(5, device=DEV, generator=gen, dtype=torch.float64))
    n = 600_000 if long else 3000
    rest = 1e-3 * scale * torch.randn(n, device=DEV, generator=gen, dtype=torch.float64)
    return [torch.cat([head, rest]).to(dtype)[1:], (-head[:3]).to(dtype)]


def check_scaled(got, before, most, norm):
    factor = min(1.0, float(torch.tensor(most)) / norm)
    for y, x in zip(got, before):
        want = x.double() * factor
        step, least = (2.0 ** -8, 2.0 ** -134) if x.dtype == torch.bfloat16 else (2.0 ** -24, 2.0 ** -150)
        tol = ((1 + step) * 11 * 2.0 ** -24 + step) * want.abs() + least * 1.01
        assert bool(((y.double() - want).abs() <= tol).all()), (most, float((y.double() - want).abs().max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("scale,most", [(1e38, 1e-6), (1e38, 1e-7), (1e38, 1e-8), (1e38, 1e-30), (1e30, 1e-12), (1e20, 1e-18),
                                        (1.0, 1e-37), (1.0, 3e-38), (1.0, 1e-40), (1e-10, 1e-44), (1e10, 1e-27), (1e10, 1.2e-28)])
def test_factors_below_fp32(gq, dtype, long, scale, most):
    """max_norm / norm may lie below fp32's normal values, or below all of them,
    where the scaled tensors do not."""
    ts = tensors(dtype, scale, long)
    norm = norm64(ts)
    outs = [torch.full_like(t, 7.0) for t in ts]
    own = gq.clip_grads(ts, most, out=outs)
    assert abs(float(own) - norm) <= 8 * 2.0 ** -24 * norm
    check_scaled(outs, ts, most, norm)
    outs = [torch.full_like(t, 7.0) for t in ts]
    gq.clip_grads(ts, most, norm=own, out=outs)
    check_scaled(outs, ts, most, norm)
    placed = [t.clone() for t in ts]
    gq.clip_grads(placed, most)
    check_scaled(placed, ts, most, norm)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("scale,most", [(1.0, 0.5), (1e-20, 3e-22), (1e38, 1e-8), (1e30, 2e29), (2.2e38, 1.0), (2.2e38, 1e38), (1.0, 1e9)])
def test_one_meaning_of_the_norm(gq, dtype, long, scale, most):
    """The tensors' own norm and the same norm handed in: the same bits, also where
    the norm of finite elements is past fp32 (2.2e38: 3.8e38 and more)."""
    ts = tensors(dtype, scale, long)
    norm = gq.grad_norm(ts)
    a, b = ([torch.full_like(t, 7.0) for t in ts] for _ in range(2))
    assert torch.equal(gq.clip_grads(ts, most, out=a), norm)
    gq.clip_grads(ts, most, norm=norm, out=b)
    placed = [t.clone() for t in ts]
    gq.clip_grads(placed, most, norm=norm)
    for x, y, z in zip(a, b, placed):
        assert torch.equal(x, y) and torch.equal(x, z)
    past = norm64(ts) > torch.finfo(torch.float32).max * (1 + 2.0 ** -20)
    assert past == (scale > 2e38) and bool(torch.isinf(norm)) == past
    if past:
        assert all(bool((x == 0).all()) for x in a)


def test_given_norm_and_the_tensors(gq):
    """A given norm may lie in a tensor that is only read, and right beside one
    that is written; in one that is written it is refused."""
    t = torch.arange(1.0, 1001.0, device=DEV)
    out = torch.zeros_like(t)
    gq.clip_grads([t], 50.0, norm=t[99], out=[out])  # 100
    assert torch.equal(out, t * 0.5)
    u = t.clone()
    gq.clip_grads([u[:99], u[100:]], 50.0, norm=u[99])
    assert torch.equal(u[:99], t[:99] * 0.5) and torch.equal(u[100:], t[100:] * 0.5) and float(u[99]) == 100.0
    for grads, out in (([u], None), ([u[99:]], None), ([t], [u])):
        with pytest.raises(gq.GQError, match="overlap"):
            gq.clip_grads(grads, 50.0, norm=u[99], out=out)
    assert float(u[99]) == 100.0
