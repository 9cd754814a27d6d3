"""The gated feed-forward block and its backward pass against plain
implementations in 64 bits.

Bounds, all from the formulas; a rounding to bf16 is off by at most 2^-8 of
the value, to fp32 by 2^-24, to e4m3 by 2^-4 or half its smallest step, 2^-10:
* the projections x, u in fp32: e = 2^-12 S, S = the sum of |products|: an
  fp32 accumulation of up to 2^11 partial sums in any order, each rounding at
  most 2^-24 of a partial sum no larger than S, and the factors' few 2^-24;
* sigma(z) in fp32: exp's argument is off by at most four roundings, 4 |z|
  2^-24, exp itself and the reciprocal by a few units in the last place, so
  r = (|z| + 8) 2^-22 of sigma; past exp's overflow it is 0 instead of less
  than 2^-126;
* h = x sigma u: |act'| <= 1.13 for both activations, so
  1.13 e_x (|u| + e_u) + |act| e_u + (r + 3 2^-24) |h| + 2^-126 |x u|;
* act' = sigma + x sigma (1 - sigma) z': r of the sum of both terms' sizes,
  and the absolute error of 1 - sigma, 2^-23, times |x z' sigma|;
* quantized values divided by their scale: the value's own bound, 2^-4 of the
  value, and 2^-10 / scale; a scale is 448 / amax of values within their bounds.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
ACTS = ["silu", "gelu"]


@pytest.fixture(scope="module")
def gq():
    import __graft_entry__

    __graft_entry__.build()
    import fp8_quantization_moe_gb300 as m

    return m


# ------------------------------------------------------------ plain forms --

def blocks(n):
    return -(-n // 128)


def normal(gen, *shape):
    return torch.randn(*shape, device=DEV, generator=gen, dtype=torch.float64)


def codes(gen, *shape, width=2.0):
    """e4m3 values of a normal distribution, as quantized rows hold them."""
    return (normal(gen, *shape) * 448 / width / 3).clamp(-448, 448).float().to(E4M3)


def scales(gen, *shape):
    return torch.exp(0.7 * normal(gen, *shape)).float() * 300


def wide(q, s, tall):
    """The values that q (..., R, C) with one scale per tall x 128 stands for."""
    s = s.double()
    if tall > 1:
        s = s.repeat_interleave(tall, -2)[..., :q.shape[-2], :]
    return q.double() / s.repeat_interleave(128, -1)[..., :q.shape[-1]]


def z_of(x, act):
    """z and dz/dx."""
    if act == "silu":
        return x, torch.ones_like(x)
    a = 2 * math.sqrt(2 / math.pi)
    return a * (x + 0.044715 * x ** 3), a * (1 + 3 * 0.044715 * x * x)


def starts(offs, M):
    """Group bounds as the calls read them: running maximum, clamped."""
    ends = np.clip(np.maximum.accumulate(np.maximum(np.asarray(offs), 0)), 0, M)
    return list(zip(np.concatenate([[0], ends[:-1]]).tolist(), ends.tolist()))


class Case:
    def __init__(self, M, N, K, offs, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed + M + 3 * N + 7 * K)
        E = len(offs)
        self.M, self.N, self.K, self.E = M, N, K, E
        self.qa, self.sa = codes(g, M, K), scales(g, M, blocks(K))
        self.qb, self.sb = codes(g, E, 2, N, K), scales(g, E, 2, blocks(N), blocks(K)) * K ** 0.5
        self.qd, self.sd = codes(g, M, 2, N), scales(g, M, 2, blocks(N))
        self.offs = torch.tensor(offs, dtype=torch.int32, device=DEV)
        self.bounds = starts(offs, M)
        self.end = self.bounds[-1][1]

    def args(self):
        return self.qa, self.sa, self.qb, self.sb, self.offs

    def forward(self, act):
        """x, u, h and their bounds."""
        a = wide(self.qa, self.sa, 1)
        pre = torch.zeros(2, self.M, self.N, device=DEV, dtype=torch.float64)
        S = torch.zeros_like(pre)
        for e, (s, t) in enumerate(self.bounds):
            for j in range(2):
                w = wide(self.qb[e, j], self.sb[e, j], 128)
                pre[j, s:t] = a[s:t] @ w.T
                S[j, s:t] = a[s:t].abs() @ w.T.abs()
        (x, u), (ex, eu) = pre, 2.0 ** -12 * S
        z, _ = z_of(x, act)
        sig = torch.sigmoid(z)
        h = x * sig * u
        r = (z.abs() + 8) * 2.0 ** -22
        eh = (1.13 * ex * (u.abs() + eu) + (x * sig).abs() * eu + (r + 3 * 2.0 ** -24) * h.abs()
              + 2.0 ** -126 * (x * u).abs())
        return pre.transpose(0, 1), 2.0 ** -12 * S.transpose(0, 1), h, eh

    def grad(self):
        d = wide(self.qd, self.sd, 1)
        out = torch.zeros(self.M, self.K, device=DEV, dtype=torch.float64)
        S = torch.zeros_like(out)
        for e, (s, t) in enumerate(self.bounds):
            for j in range(2):
                w = wide(self.qb[e, j], self.sb[e, j], 128)
                out[s:t] += d[s:t, j] @ w
                S[s:t] += d[s:t, j].abs() @ w.abs()
        return out, S


def check_bf16(got, want, err):
    assert got.dtype == torch.bfloat16
    off = (got.double() - want).abs() - (1 + 2.0 ** -8) * err - 2.0 ** -8 * want.abs()
    assert bool((off <= 2.0 ** -134).all()), float(off.max())  # half of bf16's smallest step


def check_quantized(q, s, want, err, pow2=False):
    """q (R, C), s (R, blocks) against values known to within err."""
    assert q.dtype == E4M3 and s.dtype == torch.float32
    C = want.shape[1]
    for b in range(s.shape[1]):
        at = slice(128 * b, min(C, 128 * b + 128))
        w, e, k = want[:, at], err[:, at], s[:, b].double()
        most, least = ((w.abs() + e).amax(1), (w.abs() - e).clamp_min(0).amax(1))
        lo, hi = 448 / most.clamp_min(1e-12), 448 / least.clamp_min(1e-12)
        lo, hi = lo * (1 - 2.0 ** -22), hi * (1 + 2.0 ** -22)
        if pow2:
            assert bool((torch.frexp(k)[0] == 0.5).all())
            lo = torch.exp2(torch.floor(torch.log2(lo)))
        assert bool(((lo <= k) & (k <= hi)).all())
        v = q[:, at].double() / k[:, None]
        off = (v - w).abs() - (1 + 2.0 ** -4) * e - 2.0 ** -4 * w.abs() - 2.0 ** -10 / k[:, None]
        assert bool((off <= 0).all()), float(off.max())


def sentinel(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    t.view(torch.uint8).fill_(0x5A)
    return t


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == 0x5A).all())


SHAPES = [
    # M, N, K, offs
    (1, 16, 16, [1]),
    (1, 128, 128, [0, 1, 1]),
    (3, 48, 32, [1, 1, 3]),
    (5, 2064, 144, [0, 2, 2, 5]),
    (17, 144, 272, [17]),
    (64, 272, 1040, [10, 20, 64, 64]),
    (97, 400, 656, [33, 96]),                 # a row behind the last end
    (128, 128, 128, [128]),
    (129, 256, 400, [0, 129]),
    (300, 1040, 528, [0, 60, 60, 200, 290]),  # ragged everywhere, rows behind the last end
    (300, 144, 2064, [200, 100, 250, 10]),    # ends that decrease
    (700, 368, 240, [-5, 257, 999]),          # and that lie outside
    (1000, 16, 4112, [500, 1000]),
    (2500, 640, 384, [1, 2, 1300, 2500]),
]


@pytest.mark.parametrize("M,N,K,offs", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_forward(gq, M, N, K, offs, act):
    c = Case(M, N, K, offs)
    pre, epre, h, eh = c.forward(act)
    out, q, s, kept = (sentinel((M, N), torch.bfloat16), sentinel((M, N), E4M3),
                       sentinel((M, blocks(N)), torch.float32), sentinel((M, 2, N), torch.bfloat16))
    r = gq.grouped_gated_mm(*c.args(), activation=act, out=out, q=q, scales=s, pre=kept)
    gq.check_device_error()
    assert r.out is out and r.q is q and r.scales is s and r.pre is kept
    n = c.end
    check_bf16(out[:n], h[:n], eh[:n])
    check_bf16(kept[:n], pre[:n], epre[:n])
    check_quantized(q[:n], s[:n], h[:n], eh[:n])
    for t in (out, q, s, kept):
        assert untouched(t[n:])


@pytest.mark.parametrize("M,N,K,offs", [SHAPES[2], SHAPES[6], SHAPES[9], SHAPES[13]])
def test_forward_forms_agree(gq, M, N, K, offs):
    """Each output has the same bits whichever others are written with it."""
    c = Case(M, N, K, offs, seed=1)
    n = c.end
    every = gq.grouped_gated_mm(*c.args(), plain=True, fp8=True, keep=True)
    only = gq.grouped_gated_mm(*c.args())
    assert only.q is None and only.scales is None and only.pre is None
    assert torch.equal(only.out[:n].view(torch.int16), every.out[:n].view(torch.int16))
    only = gq.grouped_gated_mm(*c.args(), plain=False, fp8=True)
    assert only.out is None and only.pre is None
    assert torch.equal(only.q[:n].view(torch.uint8), every.q[:n].view(torch.uint8))
    assert torch.equal(only.scales[:n], every.scales[:n])
    only = gq.grouped_gated_mm(*c.args(), keep=True)
    assert torch.equal(only.pre[:n].view(torch.int16), every.pre[:n].view(torch.int16))
    p = gq.grouped_gated_mm(*c.args(), plain=False, fp8=True, pow2_scales=True)
    _, _, h, eh = c.forward("silu")
    check_quantized(p.q[:n], p.scales[:n], h[:n], eh[:n], pow2=True)


@pytest.mark.parametrize("M,offs", [(40, [8, 24, 40]), (400, [130, 400, 400])])
def test_forward_quantizes_exactly(gq, M, offs):
    """Gates of at least 32, whose sigma is 1 in fp32, and whole numbers all
    along: h is known exactly, and q and its scales are block_rows' of it."""
    N, K, E = 272, 128, 3
    g = torch.Generator(device=DEV).manual_seed(M)
    a = torch.randint(0, 2, (M, K), device=DEV, generator=g).double()
    a[:, :40] = 1.0
    w = torch.randint(-1, 2, (E, 2, N, K), device=DEV, generator=g).double()
    w[:, 0, :, :40] = 1.0
    w[:, 0] = w[:, 0].abs()
    one = torch.ones(M, 1, device=DEV)
    r = gq.grouped_gated_mm(a.float().to(E4M3), one, w.float().to(E4M3),
                            torch.ones(E, 2, blocks(N), 1, device=DEV),
                            torch.tensor(offs, dtype=torch.int32, device=DEV), fp8=True, keep=True)
    h = torch.empty(M, N, device=DEV)
    for e, (s, t) in enumerate(starts(offs, M)):
        x, u = (a[s:t] @ w[e, j].T for j in range(2))
        assert bool((x >= 32).all())
        assert torch.equal(r.pre[s:t, 0].double(), x) and torch.equal(r.pre[s:t, 1].double(), u)
        h[s:t] = (x * u).float()
    assert torch.equal(r.out, h.to(torch.bfloat16))
    q, s = gq.block_rows(h)
    assert torch.equal(r.q.view(torch.uint8), q.view(torch.uint8)) and torch.equal(r.scales, s)


@pytest.mark.parametrize("M,N,K,offs", SHAPES)
def test_grad(gq, M, N, K, offs):
    c = Case(M, N, K, offs, seed=2)
    out = sentinel((M, K), torch.bfloat16)
    assert gq.grouped_gated_grad(c.qd, c.sd, c.qb, c.sb, c.offs, out=out) is out
    gq.check_device_error()
    want, S = c.grad()
    n = c.end
    check_bf16(out[:n], want[:n], 2.0 ** -12 * S[:n])
    assert untouched(out[n:])


def test_grad_halves_are_apart(gq):
    """A NaN in one half of a row, or behind the ragged end of one expert's
    matrix, reaches what it belongs to only."""
    M, N, K = 300, 144, 272
    c = Case(M, N, K, [100, 200, 300], seed=3)
    want = gq.grouped_gated_grad(c.qd, c.sd, c.qb, c.sb, c.offs)
    bad = c.qd.clone()
    bad.view(torch.uint8)[7, 1, 3] = 0x7F
    bad.view(torch.uint8)[150, 0, N - 1] = 0x7F
    w = c.qb.clone()
    w.view(torch.uint8)[2, 0, 5, 17] = 0x7F  # column 17 of expert 2's rows
    got = gq.grouped_gated_grad(bad, c.sd, w, c.sb, c.offs)
    assert bool(got[7].isnan().all()) and bool(got[150].isnan().all())
    assert bool(got[200:, 17].isnan().all())
    hit = torch.zeros(M, K, dtype=torch.bool, device=DEV)
    hit[7] = hit[150] = True
    hit[200:, 17] = True
    assert torch.equal(got[~hit], want[~hit])


def test_forward_contains_nan(gq):
    M, N, K = 300, 144, 272
    c = Case(M, N, K, [100, 200, 300], seed=4)
    want = gq.grouped_gated_mm(*c.args(), fp8=True, keep=True)
    qa, qb = c.qa.clone(), c.qb.clone()
    qa.view(torch.uint8)[7, K - 1] = 0x7F
    qb.view(torch.uint8)[1, 1, N - 1, 0] = 0x7F  # u of column N - 1 of expert 1
    got = gq.grouped_gated_mm(qa, c.sa, qb, c.sb, c.offs, fp8=True, keep=True)
    hit = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    hit[7] = True
    hit[100:200, N - 1] = True
    assert torch.equal(got.out.isnan(), hit)
    assert torch.equal(got.q.float().isnan(), hit)
    assert torch.equal(got.out[~hit], want.out[~hit])
    assert bool(got.pre[7].isnan().all()) and not bool(got.pre[100:200, 0].isnan().any())
    # blocks without a NaN are as they were; one with a NaN among others does not count it
    assert torch.equal(got.scales[:7], want.scales[:7]) and torch.equal(got.scales[8:, 0], want.scales[8:, 0])
    assert bool(got.scales.isfinite().all())


# Rows that are no multiple of 64 bytes, 100 of them per group and more, and
# hundreds of tiles: the products of block pairs.
PAIRS = [
    # M, inner, outer, offs: groups that end within a pair's first and second block, a single
    # row, an empty group, rows behind the last end
    (6200, 144, 2576, [3000, 3001, 3001, 5200, 6100]),
    (7424, 400, 2320, [256, 384, 640, 7400]),
    (6144, 16, 4368, [6144]),
    (9000, 1104, 1424, [90, 300, 5000, 9000]),
]


@pytest.mark.parametrize("M,inner,outer,offs", PAIRS)
def test_pairs_of_blocks(gq, M, inner, outer, offs):
    c = Case(M, outer, inner, offs, seed=10)
    n = c.end
    pre, epre, h, eh = c.forward("silu")
    r = gq.grouped_gated_mm(*c.args(), fp8=True, keep=True)
    gq.check_device_error()
    check_bf16(r.out[:n], h[:n], eh[:n])
    check_bf16(r.pre[:n], pre[:n], epre[:n])
    check_quantized(r.q[:n], r.scales[:n], h[:n], eh[:n])
    # the same projections by the plain product
    w, sw = c.qb[:, 0].contiguous(), c.sb[:, 0].contiguous()
    out = sentinel((M, outer), torch.bfloat16)
    gq.grouped_mm(c.qa, c.sa, w, sw, c.offs, out=out)
    check_bf16(out[:n], pre[:n, 0], epre[:n, 0])
    assert untouched(out[n:])
    again = gq.grouped_gated_mm(*c.args(), fp8=True, keep=True)
    for a, b in zip(r, again):
        assert torch.equal(a[:n].view(torch.uint8), b[:n].view(torch.uint8))


@pytest.mark.parametrize("M,inner,outer,offs", PAIRS)
def test_pairs_of_blocks_transposed(gq, M, inner, outer, offs):
    c = Case(M, inner, outer, offs, seed=11)
    n = c.end
    out = sentinel((M, outer), torch.bfloat16)
    gq.grouped_gated_grad(c.qd, c.sd, c.qb, c.sb, c.offs, out=out)
    gq.check_device_error()
    want, S = c.grad()
    check_bf16(out[:n], want[:n], 2.0 ** -12 * S[:n])
    assert untouched(out[n:])
    w, sw = c.qb[:, 1].contiguous(), c.sb[:, 1].contiguous()
    d, sd = c.qd[:, 1].contiguous(), c.sd[:, 1].contiguous()
    out = gq.grouped_mm(d, sd, w, sw, c.offs, transpose_b=True)
    for e, (s, t) in enumerate(c.bounds):
        a, b = wide(d[s:t], sd[s:t], 1), wide(w[e], sw[e], 128)
        check_bf16(out[s:t], a @ b, 2.0 ** -12 * (a.abs() @ b.abs()))


# Few rows, long contractions and few tiles: two, four and eight blocks share a tile.
SPLIT = [
    # M, inner, outer, offs
    (1, 1040, 272, [1]),
    (3, 2064, 144, [0, 1, 1, 3]),
    (13, 4112, 128, [13]),
    (40, 4096, 16, [9, 40]),
    (30, 2000, 1040, [10, 28]),       # rows behind the last end
    (16, 6160, 400, [16, 3, 16, 20]),
    # more rows: the kernel for many, two and four blocks
    (128, 4096, 1040, [128]),
    (300, 2704, 272, [1, 300]),
    (700, 2800, 528, [257, 300, 300, 650]),
    (129, 7184, 48, [129]),
]


@pytest.mark.parametrize("M,inner,outer,offs", SPLIT)
def test_blocks_that_share_a_tile(gq, M, inner, outer, offs):
    c, t = Case(M, outer, inner, offs, seed=16), Case(M, inner, outer, offs, seed=17)
    n = c.end
    pre, epre, h, eh = c.forward("gelu")
    out = sentinel((M, outer), torch.bfloat16)
    r = gq.grouped_gated_mm(*c.args(), activation="gelu", out=out, fp8=True, keep=True)
    gq.check_device_error()
    check_bf16(out[:n], h[:n], eh[:n])
    check_bf16(r.pre[:n], pre[:n], epre[:n])
    check_quantized(r.q[:n], r.scales[:n], h[:n], eh[:n])
    assert untouched(out[n:])
    w, sw = c.qb[:, 0].contiguous(), c.sb[:, 0].contiguous()
    check_bf16(gq.grouped_mm(c.qa, c.sa, w, sw, c.offs)[:n], pre[:n, 0], epre[:n, 0])
    want, S = t.grad()
    got = gq.grouped_gated_grad(t.qd, t.sd, t.qb, t.sb, t.offs)
    check_bf16(got[:n], want[:n], 2.0 ** -12 * S[:n])
    w, sw = t.qb[:, 1].contiguous(), t.sb[:, 1].contiguous()
    d, sd = t.qd[:, 1].contiguous(), t.sd[:, 1].contiguous()
    back = gq.grouped_mm(d, sd, w, sw, t.offs, transpose_b=True)
    for e, (a, b) in enumerate(t.bounds):
        v, x = wide(d[a:b], sd[a:b], 1), wide(w[e], sw[e], 128)
        check_bf16(back[a:b], v @ x, 2.0 ** -12 * (v.abs() @ x.abs()))
    for _ in range(20):  # the same bits whichever block comes first
        again = gq.grouped_gated_mm(*c.args(), activation="gelu", fp8=True, keep=True)
        assert torch.equal(again.q[:n].view(torch.uint8), r.q[:n].view(torch.uint8))
        assert torch.equal(again.pre[:n], r.pre[:n])
        assert torch.equal(gq.grouped_gated_grad(t.qd, t.sd, t.qb, t.sb, t.offs)[:n], got[:n])


def test_pairs_contain_nan(gq):
    M, inner, outer, offs = PAIRS[0]
    c = Case(M, outer, inner, offs, seed=12)
    n = c.end
    want = gq.grouped_gated_mm(*c.args(), keep=True)
    qa, qb = c.qa.clone(), c.qb.clone()
    qa.view(torch.uint8)[[5, 200, 3000]] = 0x7F
    qa.view(torch.uint8)[6100:] = 0x7F  # behind the last end
    qb.view(torch.uint8)[0, 1, outer - 1, 0] = 0x7F
    got = gq.grouped_gated_mm(qa, c.sa, qb, c.sb, c.offs, keep=True)
    hit = torch.zeros(M, outer, dtype=torch.bool, device=DEV)
    hit[[5, 200, 3000]] = True
    hit[:3000, outer - 1] = True
    assert torch.equal(got.out[:n].isnan(), hit[:n])
    assert torch.equal(got.out[:n][~hit[:n]], want.out[:n][~hit[:n]])


# ---------------------------------------------------------------- backward --

def backward_plain(g, pre, act):
    """dx, du (M, 2, N) and their bounds before the rounding to the output."""
    g, x, u = g.double(), pre[:, 0].double(), pre[:, 1].double()
    z, dz = z_of(x, act)
    s, c = torch.sigmoid(z), torch.sigmoid(-z)
    # float64's own limits: sigma underflows to 0 while x is still finite
    term = torch.where(s * c == 0, torch.zeros_like(x), x * s * c * dz)
    r = (z.abs().clamp_max(200) + 8) * 2.0 ** -22
    slope = s + term
    es = r * (s + term.abs()) + 2.0 ** -23 * torch.where(s > 1e-30, x * dz * s, torch.zeros_like(x)).abs().nan_to_num(posinf=0)
    act_x = torch.where(s == 0, torch.zeros_like(x), x * s)
    want = torch.stack([g * u * slope, g * act_x], 1)
    tiny = 2.0 ** -126 * (1 + x.abs()) * (1 + dz.abs())
    err = torch.stack([(g * u).abs() * (es + tiny) + 3 * 2.0 ** -24 * want[:, 0].abs(),
                       g.abs() * (r * act_x.abs() + tiny) + 3 * 2.0 ** -24 * want[:, 1].abs()], 1)
    return want, err + 2.0 ** -148


@pytest.mark.parametrize("M,N", [(1, 16), (1, 128), (2, 144), (7, 400), (33, 112), (129, 1040), (3, 16400), (1025, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ACTS)
def test_backward(gq, M, N, dtype, act):
    gen = torch.Generator(device=DEV).manual_seed(M + N)
    g = (1e-3 * normal(gen, M, N)).to(dtype)
    pre = (3 * normal(gen, M, 2, N)).to(dtype)
    want, err = backward_plain(g, pre, act)
    r = gq.gated_backward(g, pre, activation=act, fp8=True)
    assert r.out.dtype == dtype and r.pre is None
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    off = (r.out.double() - want).abs() - (1 + step) * err - step * want.abs()
    # results below 2^-126 are multiples of their type's smallest step, 2^-133 in bf16 and 2^-149
    # in fp32 (8 and 24 bits of precision from 2^-126 down): rounding them is off by half of it,
    # however small the value
    least = 2.0 ** -134 if dtype == torch.bfloat16 else 2.0 ** -150
    assert bool((off <= least).all()), float(off.max())
    check_quantized(r.q.view(2 * M, N), r.scales.view(2 * M, -1), want.reshape(2 * M, N), err.reshape(2 * M, N))
    if dtype == torch.float32:  # the rows before any rounding: block_rows' bits
        for pow2 in (False, True):
            q, s = gq.block_rows(r.out.view(2 * M, N), pow2_scales=pow2)
            p = gq.gated_backward(g, pre, activation=act, plain=False, fp8=True, pow2_scales=pow2)
            assert p.out is None
            assert torch.equal(p.q.view(2 * M, N).view(torch.uint8), q.view(torch.uint8))
            assert torch.equal(p.scales.view(2 * M, -1), s)
    only = gq.gated_backward(g, pre, activation=act)
    assert only.q is None and only.scales is None and torch.equal(only.out, r.out)


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(gq, act):
    """The gradient of sum(g * act(x) u) by central differences in 64 bits:
    their error is step^2 / 6 of a third derivative (below 2 for both
    activations), 1e-9 here, and the rounding's 2^-52 / step."""
    gen = torch.Generator(device=DEV).manual_seed(9)
    g, pre = normal(gen, 40, 64).float(), (2 * normal(gen, 40, 2, 64)).float()
    out = gq.gated_backward(g, pre, activation=act).out.double()

    def loss(x, u):
        z, _ = z_of(x, act)
        return g.double() * x * torch.sigmoid(z) * u

    x, u, t = pre[:, 0].double(), pre[:, 1].double(), 5e-5
    dx = (loss(x + t, u) - loss(x - t, u)) / (2 * t)
    du = (loss(x, u + t) - loss(x, u - t)) / (2 * t)
    _, err = backward_plain(g, pre, act)
    tol = 1e-8 * (1 + g.double().abs() * (1 + u.abs()))
    assert bool(((out[:, 0] - dx).abs() <= tol + err[:, 0] + 2.0 ** -24 * dx.abs()).all())
    assert bool(((out[:, 1] - du).abs() <= tol + err[:, 1] + 2.0 ** -24 * du.abs()).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ACTS)
def test_backward_extremes(gq, dtype, act):
    """Projections at the ends of the range: the slope is 0 or 1 there, never
    a NaN from an infinity times a zero."""
    big = torch.finfo(dtype).max
    x = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 90.0, -90.0, 200.0, -200.0, 1e10, -1e10,
                      big, -big, float("inf"), float("-inf")], device=DEV).to(dtype)
    pre = torch.stack([x, torch.ones_like(x)])[None].contiguous()
    g = torch.ones(1, 16, device=DEV, dtype=dtype)
    out = gq.gated_backward(g, pre, activation=act).out.float()[0]
    assert bool(out[0].isfinite().all())
    assert bool((out[0][x >= 200] == 1).all()) and bool((out[0][x <= -200] == 0).all())
    assert bool((out[0][:4] == 0.5 * (1.0 if act == "silu" else 1.5957691)).all()) or act == "gelu"
    pos = x >= 200
    assert torch.equal(out[1][pos], x.float()[pos]) and bool((out[1][x <= -200] == 0).all())
    nan = torch.full_like(pre, float("nan"))
    assert bool(gq.gated_backward(g, nan, activation=act).out.isnan().all())


def test_backward_order_of_factors(gq):
    """A product of g and u past fp32's range beside a slope that makes up for it."""
    pre = torch.tensor([[[-100.0] * 8 + [-50.0] * 8, [1e30] * 16]], device=DEV)
    g = torch.full((1, 16), 1e30, device=DEV)
    out = gq.gated_backward(g, pre).out[0]
    x = pre[0, 0].double()
    sig = torch.sigmoid(x)
    want = 1e30 * sig * (1 + x * (1 - sig)) * 1e30  # -50: -9e39, past the range; -100: 0 in fp32
    assert bool((out[0, :8] == 0).all()) and bool((want[8:] < -3.5e38).all())
    assert bool((out[0, 8:] == float("-inf")).all())


def test_backward_blocks_with_nan_and_inf(gq):
    """As block_rows: a NaN does not count, an infinity makes the scale 0."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    g, pre = normal(gen, 6, 400).float(), normal(gen, 6, 2, 400).float()
    g[1, 5] = float("nan")
    g[2, 300] = float("inf")
    g[3, :128] = 0.0
    pre[4, 1, 399] = float("nan")
    r = gq.gated_backward(g, pre, fp8=True)
    q, s = gq.block_rows(r.out.view(12, 400))
    assert torch.equal(r.q.view(12, 400).view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(r.scales.view(12, -1), s)
    assert bool(r.out[1, :, 5].isnan().all()) and int(r.out.isnan().sum()) == 3


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_pitch_and_in_place(gq, dtype):
    gen = torch.Generator(device=DEV).manual_seed(6)
    wide_g = normal(gen, 130, 560).to(dtype)
    g = wide_g[:, 32:32 + 272]
    pre = normal(gen, 130, 2, 272).to(dtype)
    want = gq.gated_backward(g.contiguous(), pre, fp8=True)
    got = gq.gated_backward(g, pre, fp8=True)
    for a, b in zip(want[:3], got[:3]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    r = gq.gated_backward(g, pre, out=pre, fp8=True)
    assert r.out is pre and torch.equal(pre, want.out)
    assert torch.equal(r.q.view(torch.uint8), want.q.view(torch.uint8))


# ------------------------------------------------------------------- use --

@pytest.mark.parametrize("M,N,K,offs", [(9, 144, 272, [4, 9]), (700, 272, 400, [300, 650])])
def test_streams_and_graphs(gq, M, N, K, offs):
    c = Case(M, N, K, offs, seed=7)
    n = c.end

    def step(stream=None):
        r = gq.grouped_gated_mm(*c.args(), fp8=True, keep=True, stream=stream)
        b = gq.gated_backward(r.out, r.pre, fp8=True, stream=stream)
        d = gq.grouped_gated_grad(b.q, b.scales, c.qb, c.sb, c.offs, stream=stream)
        return [t[:n].clone() if stream is None else t for t in (*r, *b[:3], d)]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = gq.grouped_gated_mm(*c.args(), fp8=True, keep=True)
        b = gq.gated_backward(r.out, r.pre, fp8=True)
        d = gq.grouped_gated_grad(b.q, b.scales, c.qb, c.sb, c.offs)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for w, g1, g2 in zip(want, got, (*r, *b[:3], d)):
        assert torch.equal(w.view(torch.uint8), g1[:n].view(torch.uint8))
        assert torch.equal(w.view(torch.uint8), g2[:n].view(torch.uint8))


@pytest.mark.parametrize("M,N,K,offs", [(12, 5008, 656, [4, 12]), (600, 48, 400, [300, 600]),
                                         (6200, 2576, 144, [3000, 6200]), (5, 4112, 4112, [5]),
                                         (129, 4112, 4112, [129])])
def test_timeouts_are_reported_not_hung(gq, M, N, K, offs):
    """A withheld accumulator release: every role leaves its loop after the
    (shortened) limit, the call reports GQ_ERR_TIMEOUT, the next call is fine.
    (Few rows, many, pairs of blocks, and blocks that share a tile's contraction.)"""
    c, t = Case(M, N, K, offs, seed=8), Case(M, K, N, offs, seed=9)
    calls = [lambda: gq.grouped_gated_mm(*c.args(), fp8=True).q,
             lambda: gq.grouped_gated_grad(t.qd, t.sd, t.qb, t.sb, t.offs)]
    for call in calls:
        want = call()
        try:
            gq.debug_set(skip_arrival=True, wait_timeout_ns=5_000_000)
            # contractions of three 128-blocks and more: the third waits for the first accumulator
            call()
            with pytest.raises(gq.GQError) as e:
                gq.check_device_error()
            assert e.value.status == 4
        finally:
            gq.debug_set(False, 0)
        got = call()
        gq.check_device_error()
        assert torch.equal(want.view(torch.uint8), got.view(torch.uint8))


def test_empty(gq):
    z = lambda *s, dtype=E4M3: torch.zeros(*s, device=DEV, dtype=torch.float32).to(dtype)
    f = torch.float32
    offs = torch.tensor([0, 0], dtype=torch.int32, device=DEV)
    r = gq.grouped_gated_mm(z(0, 32), z(0, 1, dtype=f), z(2, 2, 48, 32), z(2, 2, 1, 1, dtype=f), offs, fp8=True, keep=True)
    assert r.out.shape == (0, 48) and r.q.shape == (0, 48) and r.scales.shape == (0, 1) and r.pre.shape == (0, 2, 48)
    r = gq.grouped_gated_mm(z(4, 32), z(4, 1, dtype=f), z(2, 2, 0, 32), z(2, 2, 0, 1, dtype=f), offs)
    assert r.out.shape == (4, 0)
    assert gq.grouped_gated_grad(z(0, 2, 48), z(0, 2, 1, dtype=f), z(2, 2, 48, 32), z(2, 2, 1, 1, dtype=f), offs).shape == (0, 32)
    assert gq.gated_backward(z(0, 16, dtype=f), z(0, 2, 16, dtype=f)).out.shape == (0, 2, 16)
    # every group empty, rows behind them: nothing is written
    out = sentinel((4, 48), torch.bfloat16)
    gq.grouped_gated_mm(z(4, 32), z(4, 1, dtype=f), z(2, 2, 48, 32), z(2, 2, 1, 1, dtype=f), offs, out=out)
    assert untouched(out)


def test_many_experts(gq):
    """As many experts as a call takes, most of them without rows."""
    E, M = 1024, 3000
    g = torch.Generator(device=DEV).manual_seed(13)
    offs = torch.randint(0, M + 1, (E,), device=DEV, generator=g).sort().values.tolist()
    for rows, ends in ((M, offs), (40, [min(o // 75, 40) for o in offs])):  # many rows and few
        c = Case(rows, 48, 144, ends, seed=14)
        n = c.end
        pre, epre, h, eh = c.forward("gelu")
        r = gq.grouped_gated_mm(*c.args(), activation="gelu", fp8=True, keep=True)
        check_bf16(r.out[:n], h[:n], eh[:n])
        check_bf16(r.pre[:n], pre[:n], epre[:n])
        check_quantized(r.q[:n], r.scales[:n], h[:n], eh[:n])
        want, S = c.grad()
        check_bf16(gq.grouped_gated_grad(c.qd, c.sd, c.qb, c.sb, c.offs)[:n], want[:n], 2.0 ** -12 * S[:n])


@pytest.mark.parametrize("K", [16, 48])
def test_past_2_31_elements(gq, K):
    """Outputs of more than 2^31 elements; K of 48: no multiple of 64, block pairs."""
    M, N = 140_000, 16384
    g = torch.Generator(device=DEV).manual_seed(15)
    qa, sa = codes(g, M, K), scales(g, M, 1)
    qb, sb = codes(g, 2, 2, N, K), scales(g, 2, 2, N // 128, 1)
    offs = torch.tensor([70_001, M], dtype=torch.int32, device=DEV)
    r = gq.grouped_gated_mm(qa, sa, qb, sb, offs, fp8=True, keep=True)
    rows = torch.tensor([0, 3, 65535, 65536, 70_000, 70_001, 131_071, 131_072, M - 2, M - 1], device=DEV)
    a = wide(qa[rows], sa[rows], 1)
    e = (rows >= 70_001).long()
    pre, S = (torch.stack([torch.stack([f(wide(qb[i, j], sb[i, j], 128)) @ f(x) for j in range(2)])
                           for x, i in zip(a, e.tolist())]) for f in (lambda v: v, torch.abs))
    epre = 2.0 ** -12 * S
    check_bf16(r.pre[rows], pre, epre)
    x, u = pre[:, 0], pre[:, 1]
    sig = torch.sigmoid(x)
    eh = (1.13 * epre[:, 0] * (u.abs() + epre[:, 1]) + (x * sig).abs() * epre[:, 1]
          + ((x.abs() + 8) * 2.0 ** -22 + 3 * 2.0 ** -24) * (x * sig * u).abs() + 2.0 ** -126 * (x * u).abs())
    check_bf16(r.out[rows], x * sig * u, eh)
    check_quantized(r.q[rows], r.scales[rows], x * sig * u, eh)
    del r
    # the same sizes the other way round
    qd, sd = codes(g, M, 2, K), scales(g, M, 2, 1)
    wb, swb = codes(g, 2, 2, K, N), scales(g, 2, 2, 1, N // 128)
    out = gq.grouped_gated_grad(qd, sd, wb, swb, offs)
    gq.check_device_error()
    for i, row in zip(e.tolist(), rows.tolist()):
        d = wide(qd[row], sd[row], 1)
        w = [wide(wb[i, j], swb[i, j], 128) for j in range(2)]
        want, size = sum(d[j] @ w[j] for j in range(2)), sum(d[j].abs() @ w[j].abs() for j in range(2))
        check_bf16(out[row], want, 2.0 ** -12 * size)


def test_backward_past_2_31_elements(gq):
    M, N = 70_000, 16384
    g = torch.empty(M, N, dtype=torch.bfloat16, device=DEV).normal_()
    pre = torch.empty(M, 2, N, dtype=torch.bfloat16, device=DEV).normal_()
    r = gq.gated_backward(g, pre, fp8=True)
    for row in (0, 32767, 32768, 65535, 65536, M - 1):
        one = gq.gated_backward(g[row:row + 1].clone(), pre[row:row + 1].clone(), fp8=True)
        for a, b in zip(r[:3], one[:3]):
            assert torch.equal(a[row:row + 1].view(torch.uint8), b.view(torch.uint8))


def test_refusals(gq):
    c = Case(4, 48, 32, [4])
    with pytest.raises(ValueError, match="activation"):
        gq.grouped_gated_mm(*c.args(), activation="relu")
    with pytest.raises(ValueError, match="neither"):
        gq.grouped_gated_mm(*c.args(), plain=False)
    with pytest.raises(ValueError, match="two matrices"):
        gq.grouped_gated_mm(c.qa, c.sa, c.qb[:, :1].contiguous(), c.sb, c.offs)
    with pytest.raises(ValueError, match="columns"):
        gq.grouped_gated_mm(c.qa[:, :16].contiguous(), c.sa, c.qb, c.sb, c.offs)
    with pytest.raises(ValueError, match="pre must have shape"):
        gq.grouped_gated_mm(*c.args(), pre=torch.empty(4, 1, 48, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError, match="scales must have shape"):
        gq.grouped_gated_mm(*c.args(), scales=torch.empty(4, 2, device=DEV))
    with pytest.raises(ValueError, match="qd must have shape"):
        gq.grouped_gated_grad(c.qd[:, :1].contiguous(), c.sd, c.qb, c.sb, c.offs)
    g = torch.zeros(4, 48, device=DEV)
    with pytest.raises(ValueError, match="pre must be a 3-D"):
        gq.gated_backward(g, torch.zeros(4, 2, 48, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dense rows"):
        gq.gated_backward(g.t(), torch.zeros(48, 2, 4, device=DEV))
    with pytest.raises(gq.GQError, match="multiple of 16"):
        gq.gated_backward(g[:, :20].contiguous(), torch.zeros(4, 2, 20, device=DEV))
