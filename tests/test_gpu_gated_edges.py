"""The gated block's calls at their edges: rows that are alike, and values at
the ends of the range."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gq():
    import __graft_entry__

    __graft_entry__.build()
    import fp8_quantization_moe_gb300 as m

    return m


def blocks(n):
    return -(-n // 128)


def codes(gen, *shape):
    return (100 * torch.randn(*shape, device=DEV, generator=gen)).clamp(-448, 448).to(E4M3)


def scales(gen, *shape):
    return 300 + 300 * torch.rand(*shape, device=DEV, generator=gen)


# M, inner, outer, offs: few tiles, whose contraction two, four (and for few rows eight)
# blocks share, and many, that one block or a pair takes
ALIKE = [
    (16, 2064, 272, [16]), (23, 4112, 128, [3, 23]), (128, 2704, 272, [128]), (140, 7184, 768, [9, 140]),
    (300, 2704, 1040, [1, 300]), (700, 2800, 528, [257, 300, 300, 700]), (6200, 144, 2576, [3000, 3001, 6200]),
    (2000, 1024, 512, [130, 2000]),
]


def same_rows(t, offs):
    flat = t.flatten(1).view(torch.uint8)
    start = 0
    for end in offs:
        if end > start:
            assert torch.equal(flat[start:end], flat[start:start + 1].expand(end - start, -1))
        start = end


@pytest.mark.parametrize("M,inner,outer,offs", ALIKE)
def test_rows_that_are_alike(gq, M, inner, outer, offs):
    """Equal rows of a group get equal bits, wherever in their tile they are."""
    gen = torch.Generator(device=DEV).manual_seed(M)
    E = len(offs)
    ends = torch.tensor(offs, dtype=torch.int32, device=DEV)
    qa = codes(gen, 1, inner).view(torch.uint8).expand(M, -1).contiguous().view(E4M3)
    sa = scales(gen, 1, blocks(inner)).expand(M, -1).contiguous()
    qb, sb = codes(gen, E, 2, outer, inner), scales(gen, E, 2, blocks(outer), blocks(inner))
    r = gq.grouped_gated_mm(qa, sa, qb, sb, ends, fp8=True, keep=True)
    gq.check_device_error()
    for t in r:
        same_rows(t, offs)
    qd = codes(gen, 1, 2, inner).view(torch.uint8).expand(M, -1, -1).contiguous().view(E4M3)
    sd = scales(gen, 1, 2, blocks(inner)).expand(M, -1, -1).contiguous()
    qb, sb = codes(gen, E, 2, inner, outer), scales(gen, E, 2, blocks(inner), blocks(outer))
    out = gq.grouped_gated_grad(qd, sd, qb, sb, ends)
    gq.check_device_error()
    same_rows(out, offs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slope_at_zero(gq, dtype, act):
    """act'(0) = sigma(0) = 1/2 for both activations, within a unit in the last place
    of the approximate reciprocal (2^-24 here) and the rounding of the result."""
    x = torch.tensor([0.0, -0.0, 1e-30, -1e-30] * 4, device=DEV).to(dtype)
    pre = torch.stack([x, torch.ones_like(x)])[None].contiguous()
    out = gq.gated_backward(torch.ones(1, 16, device=DEV, dtype=dtype), pre, activation=act).out
    assert bool(((out[0, 0].double() - 0.5).abs() <= 2.0 ** -23).all())
    assert bool((out[0, 1].double() - 0.5 * x.double()).abs().max() <= 2.0 ** -120)


def cycle(values, n):
    return torch.tensor(values, device=DEV, dtype=torch.float64).repeat(-(-n // len(values)))[:n]


# every kernel of the forward product
EXTREMES = [(16, 256, 272, [7, 16]), (16, 2064, 272, [16]), (300, 256, 272, [140, 300]), (300, 2704, 272, [300]),
            (6200, 144, 2576, [3000, 6200])]


@pytest.mark.parametrize("M,K,N,offs", EXTREMES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward_extremes(gq, M, K, N, offs, act):
    """Projections of up to an infinity with finite factors beside them.  One
    product each makes x and u: x = v 2^k, u = w 2^(k - 100), or 2^(k - 126) for the
    odd 128-columns, k by the row, so that with |x| >= 128 sigma is 0 or 1 and h
    exact: no NaN, and q and scales those that block_rows gives.  Where |x| is
    smaller, h is off by (14 |z| + 16) 2^-24 of itself: four roundings of x and one of
    its square, cube and exponent each."""
    E, nb = len(offs), blocks(N)
    k = cycle([0, 3, 7, 33, 100, 120, 126], M)
    odd = torch.arange(N, device=DEV) // 128 % 2 == 1
    v = torch.where(odd, cycle([1, -1, 0.5, -0.5, 0, 2 ** -6], N), cycle([1, -1, 448, -448, 2, -2, 0, 16], N))
    w = cycle([1, -1.5, 0.5, 1.25, -1], N)
    qa = torch.zeros(M, K, device=DEV)
    qa[:, :2] = 1
    sa = torch.ones(M, blocks(K), device=DEV)
    sa[:, 0] = torch.exp2(-k).float()
    qb = torch.zeros(E, 2, N, K, device=DEV)
    qb[:, 0, :, 0], qb[:, 1, :, 1] = v.float(), w.float()
    sb = torch.ones(E, 2, nb, blocks(K), device=DEV)
    e = torch.where(torch.arange(nb, device=DEV) % 2 == 1, 126.0, 100.0)
    sb[:, 1, :, 0] = torch.exp2(e)
    r = gq.grouped_gated_mm(qa.to(E4M3), sa, qb.to(E4M3), sb, torch.tensor(offs, dtype=torch.int32, device=DEV),
                            activation=act, fp8=True, keep=True)
    gq.check_device_error()
    most = torch.finfo(torch.float32).max
    # 448 2^120 and 448 2^126 are past fp32: infinities there
    x, u = v * torch.exp2(k)[:, None], w * torch.exp2(k[:, None] - e.double().repeat_interleave(128)[:N])
    x = torch.where(x.abs() > most, torch.copysign(torch.full_like(x, float("inf")), x), x)
    assert bool(x.isinf().any()) and bool(u.isfinite().all())
    assert torch.equal(r.pre, torch.stack([x, u], 1).float().to(torch.bfloat16))
    far = (x.abs() >= 128) | (x == 0)
    z = x if act == "silu" else 1.5957691216057308 * (x + 0.044715 * x ** 3)
    act_x = torch.where(far, x.clamp_min(0), x * torch.sigmoid(z))
    h = act_x * u
    assert not bool(h.isnan().any())
    h32 = h.float()  # exact where far, infinities where past fp32
    tol = torch.where(far, torch.zeros_like(h), (14 * z.abs() + 16) * 2.0 ** -24 * h.abs())
    assert not bool(r.out.isnan().any())
    fine = h32.to(torch.bfloat16).isfinite()
    assert torch.equal(r.out[~fine], h32.to(torch.bfloat16)[~fine]) and bool(r.out[fine].isfinite().all())
    off = (r.out.double() - h).abs() - tol * (1 + 2.0 ** -8) - 2.0 ** -8 * h.abs()
    assert bool((off[fine] <= 2.0 ** -133).all())
    q, s = gq.block_rows(h32)
    full = torch.nn.functional.pad(far, (0, nb * 128 - N), value=True).view(M, nb, 128).all(2)
    assert bool(full.any()) and bool((s[full] == 0).any()) and bool((s[full] > 0).any())
    assert torch.equal(r.scales[full], s[full])
    cols = full.repeat_interleave(128, 1)[:, :N]
    a, b = r.q.float(), q.float()
    assert torch.equal(a.isnan()[cols], b.isnan()[cols])
    assert torch.equal(a.nan_to_num(7.0)[cols], b.nan_to_num(7.0)[cols])
