"""The MoE-layer operators against plain implementations in 64 bits.

Bounds, all from the formulas:
* positions, copies, quantized bytes and scales are unique: equal bit for bit
  (the scale is one IEEE fp32 division, the product one fp32 multiply, the
  cast one rounding to e4m3);
* combine: top_k fp32 fused multiply-adds, each rounding at most 2^-24 of a
  partial sum no larger than S = sum |w y|, then one rounding to the output
  type (bf16: 2^-9 of the result, doubled for the error that comes before it);
* dweights: H fp32 fused multiply-adds and additions of partial sums no
  larger than S = sum |g y|: H * 2^-24 * S covers any order;
* grouped_mm: |err| <= 2^-8 |exact| + 2^-12 S, S = the sum of |a b|: bf16
  rounding and an fp32 accumulation of up to 2^11 partial sums in any order,
  each rounding at most 2^-24 of a partial sum no larger than S, with the
  three fp32 roundings of each block's scale factor (3 * 2^-24 S) inside it.
"""
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


def rng(seed):
    return np.random.default_rng(seed)


# ------------------------------------------------------------ plain forms --

def sort_plain(ids, E):
    flat = ids.reshape(-1)
    rows = np.concatenate([np.flatnonzero(flat == e) for e in range(E)])
    offs = np.cumsum([int((flat == e).sum()) for e in range(E)]).astype(np.int32)
    pos = np.full(flat.size, -1, np.int32)
    pos[rows] = np.arange(rows.size)
    token = np.full(flat.size, -1, np.int32)
    token[:rows.size] = rows // ids.shape[1]
    return offs, pos.reshape(ids.shape), token


def e4m3(v):
    """Nearest e4m3 value of float64 v, ties to even, saturating."""
    a = np.maximum(np.abs(v), 2.0 ** -30)
    step = np.exp2(np.clip(np.floor(np.log2(a)), -6, 8) - 3)
    return np.clip(np.rint(v / step) * step, -448, 448)


def scale_plain(amax, pow2):
    s = np.float32(448) / np.maximum(amax.astype(np.float32), np.float32(1e-12))
    if pow2:
        s = np.exp2(np.floor(np.log2(s.astype(np.float64)))).astype(np.float32)
    return s


def block_plain(x, tall, pow2=False):
    """x (R, C) float32 -> (values float64, scales), blocks of tall x 128."""
    R, C = x.shape
    nr, nc = -(-R // tall), -(-C // 128)
    s = np.zeros((nr, nc), np.float32)
    q = np.zeros((R, C))
    for i in range(nr):
        for j in range(nc):
            at = np.s_[i * tall:(i + 1) * tall, j * 128:(j + 1) * 128]
            s[i, j] = scale_plain(np.abs(x[at]).max(), pow2)
            q[at] = e4m3((x[at] * s[i, j]).astype(np.float64))
    return q, s


def activations(seed, R, C, dtype):
    r = rng(seed)
    x = r.standard_normal((R, C)) * np.exp(r.standard_normal((R, 1)) + 0.7 * r.standard_normal(C))
    x[r.random((R, C)) < 0.05] = 0.0
    return torch.from_numpy(x).to(dtype).to(DEV)


def f32(t):
    return t.float().cpu().numpy()


# ------------------------------------------------------------------- sort --

@pytest.mark.parametrize("T,k,E,drop", [
    (0, 2, 5, 0.0), (1, 1, 1, 0.0), (1, 8, 64, 0.0), (3, 5, 2, 0.5), (31, 1, 7, 0.0), (32, 4, 256, 0.2),
    (33, 3, 1024, 0.1), (257, 6, 160, 0.7), (1000, 8, 8, 0.0), (4096, 8, 1024, 0.05), (5000, 2, 1, 0.3),
    (64, 2, 16, 1.0), (40001, 7, 130, 0.1), (200003, 5, 999, 0.01),
])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(gq, T, k, E, drop, dtype):
    r = rng(T + 7 * k + E)
    ids = r.integers(0, E, (T, k))
    ids[:, :1] = np.minimum(ids[:, :1], r.integers(0, E, (T, 1)))  # uneven load
    gone = r.random((T, k)) < drop
    ids[gone] = r.choice([-1, -7, E, E + 3, 2 ** 31 - 1, -2 ** 31], gone.sum())
    got = gq.sort_tokens(torch.from_numpy(ids).to(dtype).to(DEV), E)
    for g, w, what in zip(got, sort_plain(ids, E), ("offs", "pos", "token")):
        assert g.dtype == torch.int32
        assert np.array_equal(g.cpu().numpy(), w), what


def test_sort_wide_ids_are_not_truncated(gq):
    ids = torch.tensor([[2 ** 32, 1], [-2 ** 32, 2 ** 40 + 1]], device=DEV)
    offs, pos, token = gq.sort_tokens(ids, 4)
    assert pos.tolist() == [[-1, 0], [-1, -1]]
    assert offs.tolist() == [0, 1, 1, 1] and token.tolist() == [0, -1, -1, -1]


# --------------------------------------------------------------- dispatch --

def routing(gq, seed, T, k, E, local):
    ids = torch.from_numpy(rng(seed).integers(0, E, (T, k))).to(DEV)
    ids = torch.where(ids < local, ids, -1)
    return gq.sort_tokens(ids, local)


@pytest.mark.parametrize("T,k,H,dtype", [
    (1, 1, 8, torch.bfloat16), (1, 8, 4096, torch.bfloat16), (37, 3, 1040, torch.float32),
    (300, 6, 2064, torch.bfloat16), (65, 2, 16, torch.uint8), (9, 10, 8200, torch.bfloat16),
    (2000, 4, 272, torch.bfloat16),
])
def test_dispatch(gq, T, k, H, dtype):
    order = routing(gq, T + H, T, k, 16, 11)
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randint(0, 256, (T, H * torch.empty((), dtype=dtype).element_size()), dtype=torch.uint8,
                      device=DEV, generator=g).view(dtype)
    out = torch.full((T * k, x.view(torch.uint8).shape[1]), 0x5A, dtype=torch.uint8, device=DEV)
    gq.dispatch(x, order.pos, out=out.view(dtype))
    token = order.token.cpu().numpy()
    want = np.full(out.shape, 0x5A, np.uint8)
    want[token >= 0] = x.view(torch.uint8).cpu().numpy()[token[token >= 0]]
    assert np.array_equal(out.cpu().numpy(), want)


def test_dispatch_pitch_and_short_output(gq):
    """Rows of a wider array, and an output that holds fewer rows than there
    are slots: positions behind it are dropped."""
    T, k, H = 50, 2, 96
    wide = torch.randn(T, 3 * H, device=DEV).to(torch.bfloat16)
    x = wide[:, H:2 * H]
    order = routing(gq, 5, T, k, 4, 4)
    full = gq.dispatch(x, order.pos)
    short = torch.zeros(61, H, dtype=torch.bfloat16, device=DEV)
    gq.dispatch(x, order.pos, out=short)
    assert torch.equal(short, full[:61])
    assert torch.equal(full, x[order.token.long()])
    q, s = gq.dispatch_block(x, order.pos)
    q2, s2 = gq.block_rows(x.contiguous())
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)[order.token.long()])
    assert torch.equal(s, s2[order.token.long()])
    assert torch.equal(gq.dispatch(x[:, :0], order.pos), x.new_empty(T * k, 0))


# ------------------------------------------------------ block quantization --

@pytest.mark.parametrize("R,K", [(1, 16), (1, 4096), (3, 128), (129, 144), (77, 2064), (1000, 512), (5, 8208)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pow2", [False, True])
def test_block_rows(gq, R, K, dtype, pow2):
    x = activations(R + K, R, K, dtype)
    x[0, :16] = 0.0
    x[R // 2] = 0.0  # an all-zero row
    x[R - 1, -1] = 2.0 ** -133  # the smallest bf16 subnormal
    q, s = gq.block_rows(x, pow2_scales=pow2)
    wq, ws = block_plain(f32(x), 1, pow2)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(f32(q).astype(np.float64), wq)


@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (2, 128, 128), (3, 130, 144), (1, 700, 2000), (4, 257, 640), (2, 127, 112)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pow2", [False, True])
def test_block_tiles(gq, E, N, K, dtype, pow2):
    w = activations(N + K, E * N, K, dtype).view(E, N, K)
    w[E - 1, :128, :128] = 0.0
    q, s = gq.block_tiles(w, pow2_scales=pow2)
    for e in range(E):
        wq, ws = block_plain(f32(w[e]), 128, pow2)
        assert np.array_equal(s[e].cpu().numpy(), ws)
        assert np.array_equal(f32(q[e]).astype(np.float64), wq)


@pytest.mark.parametrize("T,k,K,dtype", [(1, 8, 4096, torch.bfloat16), (130, 6, 1040, torch.float32), (700, 40, 528, torch.bfloat16)])
def test_dispatch_block(gq, T, k, K, dtype):
    order = routing(gq, T + K, T, k, 16, 11)
    x = activations(T, T, K, dtype)
    nb = -(-K // 128)
    out = torch.full((T * k, K), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((T * k, nb), -3.0, device=DEV)
    gq.dispatch_block(x, order.pos, out=out, scales=scales)
    wq, ws = block_plain(f32(x), 1)
    token = order.token.cpu().numpy()
    live = token >= 0
    assert np.array_equal(f32(out.view(torch.float8_e4m3fn))[live].astype(np.float64), wq[token[live]])
    assert np.array_equal(scales.cpu().numpy()[live], ws[token[live]])
    assert (out.cpu().numpy()[~live] == 0x5A).all() and (scales.cpu().numpy()[~live] == -3.0).all()


# ---------------------------------------------------------------- combine --

def combine_plain(y, pos, w):
    """float64 out and S for numpy y (rows, H), pos, w."""
    T, k = pos.shape
    out, S = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for j in range(k):
        t = np.flatnonzero((pos[:, j] >= 0) & (pos[:, j] < y.shape[0]))
        r = y[pos[t, j]].astype(np.float64)
        out[t] += w[t, j, None] * r
        S[t] += np.abs(w[t, j, None] * r)
    return out, S


COMBINE = [
    (1, 1, 8, torch.bfloat16), (1, 8, 4096, torch.bfloat16), (64, 8, 1040, torch.float32), (37, 3, 12, torch.float32),
    (300, 6, 2064, torch.bfloat16), (5, 19, 520, torch.bfloat16), (500, 2, 8200, torch.bfloat16), (9, 33, 264, torch.float32),
]


@pytest.mark.parametrize("T,k,H,dtype", COMBINE)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(gq, T, k, H, dtype, weighted):
    order = routing(gq, T + H, T, k, 16, 9)
    y = activations(H, T * k, H, dtype)
    w = torch.from_numpy(rng(T).random((T, k)).astype(np.float32)).to(DEV)
    dead = order.pos < 0
    w = torch.where(dead, torch.full_like(w, float("nan")), w)  # a dropped slot's weight counts for nothing
    y[int(order.offs[-1]):] = float("nan")  # nor does a row behind the last group
    out = gq.combine(y, order.pos, w if weighted else None)
    wn = np.where(dead.cpu().numpy(), 0.0, w.cpu().numpy().astype(np.float64)) if weighted else np.ones((T, k))
    want, S = combine_plain(f32(y), order.pos.cpu().numpy(), wn)
    bound = (k + 1) * 2.0 ** -24 * S + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    assert (np.abs(f32(out) - want) <= bound).all()
    empty = dead.all(1).cpu().numpy()
    assert (f32(out)[empty] == 0).all()


@pytest.mark.parametrize("T,k,H,dtype", COMBINE)
def test_combine_backward(gq, T, k, H, dtype):
    order = routing(gq, T + H, T, k, 16, 9)
    y = activations(H, T * k, H, dtype)
    g = activations(H + 1, T, H, dtype)
    w = torch.from_numpy(rng(T).random((T, k)).astype(np.float32)).to(DEV)
    pos, live = order.pos.cpu().numpy(), int(order.offs[-1])
    y[live:] = float("nan")
    dy = torch.full_like(y, 7.0)
    dy, dw = gq.combine_backward(g, y, order.pos, w, dy=dy)
    t, j = np.nonzero(pos >= 0)
    want = (w.cpu()[t, j][:, None] * g.float().cpu()[t]).to(dtype)  # one fp32 product, one rounding
    assert torch.equal(dy.cpu()[pos[t, j]], want)
    assert (dy[live:] == 7.0).all()
    prod = f32(g).astype(np.float64)[t] * f32(y).astype(np.float64)[pos[t, j]]
    got = dw.cpu().numpy()
    assert (np.abs(got[t, j] - prod.sum(1)) <= H * 2.0 ** -24 * np.abs(prod).sum(1)).all()
    assert (got[pos < 0] == 0).all()


def test_combine_gradients_against_differences(gq):
    """combine is linear in y and in the weights: the difference of the loss
    sum(g * out) along a direction is the gradient's product with it.  The
    direction is a small multiple of 2^-10 and all values are multiples of
    2^-4 or 2^-10 with few bits, so that fp32 holds every term exactly."""
    T, k, H = 40, 3, 64
    order = routing(gq, 3, T, k, 8, 6)
    r = rng(4)

    def few_bits(shape, step):
        return torch.from_numpy((r.integers(-8, 9, shape) * step).astype(np.float32)).to(DEV)

    y, g, w = few_bits((T * k, H), 2.0 ** -4), few_bits((T, H), 2.0 ** -4), few_bits((T, k), 2.0 ** -4)
    ey, ew = few_bits((T * k, H), 2.0 ** -4), few_bits((T, k), 2.0 ** -4)
    dy, dw = gq.combine_backward(g, y, order.pos, w, dy=torch.zeros_like(y))

    def loss(y, w):
        return (g.double() * gq.combine(y, order.pos, w).double()).sum()

    h = 2.0 ** -3
    assert (loss(y + h * ey, w) - loss(y - h * ey, w)) / (2 * h) == (dy.double() * ey.double()).sum()
    assert (loss(y, w + h * ew) - loss(y, w - h * ew)) / (2 * h) == (dw.double() * ew.double()).sum()


def test_dispatch_and_unweighted_combine_are_adjoint(gq):
    T, k, H = 33, 4, 128
    order = routing(gq, 6, T, k, 8, 5)
    r = rng(8)
    x = torch.from_numpy(r.integers(-8, 9, (T, H)).astype(np.float32)).to(DEV)
    d = torch.from_numpy(r.integers(-8, 9, (T * k, H)).astype(np.float32)).to(DEV)
    out = gq.dispatch(x, order.pos, out=torch.zeros_like(d))
    back = gq.combine(d, order.pos)
    assert (out.double() * d.double()).sum() == (back.double() * x.double()).sum()


# ------------------------------------------------------------- grouped_mm --

def product_inputs(seed, M, N, K, E, transposed):
    r = rng(seed)
    inner = N if transposed else K
    a = r.standard_normal((M, inner)) * np.exp(0.5 * r.standard_normal(inner))
    w = r.standard_normal((E * N, K)) * np.exp(0.5 * r.standard_normal((E * N, 1)))
    return a.astype(np.float32), w.astype(np.float32).reshape(E, N, K)


def product_plain(qa, sa, qb, sb, offs, transposed, M, outer):
    """float64 out and S (NaN-free), rows outside the groups None."""
    qa, sa = f32(qa).astype(np.float64), sa.cpu().numpy().astype(np.float64)
    a = qa / np.repeat(sa, 128, 1)[:, :qa.shape[1]]
    out, S = np.zeros((M, outer)), np.zeros((M, outer))
    start, covered = 0, np.zeros(M, bool)
    for e, end in enumerate(offs):
        end = min(max(int(end), start), M)
        if end > start:
            q = f32(qb[e]).astype(np.float64)
            s = sb[e].cpu().numpy().astype(np.float64)
            w = q / np.repeat(np.repeat(s, 128, 0), 128, 1)[:q.shape[0], :q.shape[1]]
            w = w if transposed else w.T
            out[start:end] = a[start:end] @ w
            S[start:end] = np.abs(a[start:end]) @ np.abs(w)
            covered[start:end] = True
        start = end
    return out, S, covered


def check_product(gq, M, N, K, offs, transposed, seed=0):
    E = len(offs)
    a, w = product_inputs(seed + M + N + K, M, N, K, E, transposed)
    qa, sa = gq.block_rows(torch.from_numpy(a).to(DEV))
    qb, sb = gq.block_tiles(torch.from_numpy(w).to(DEV))
    outer = K if transposed else N
    out = torch.full((M, outer), 77.0, dtype=torch.bfloat16, device=DEV)
    o = torch.tensor(offs, dtype=torch.int32, device=DEV)
    gq.grouped_mm(qa, sa, qb, sb, o, transpose_b=transposed, out=out)
    gq.check_device_error()
    want, S, covered = product_plain(qa, sa, qb, sb, offs, transposed, M, outer)
    got = f32(out).astype(np.float64)
    assert (got[~covered] == 77.0).all(), "rows behind the last group"
    err = np.abs(got - want)[covered]
    bad = err > (2.0 ** -8 * np.abs(want) + 2.0 ** -12 * S)[covered]
    assert not bad.any(), f"{bad.sum()} of {bad.size} out of bound; first {np.argwhere(bad)[0]}"


PRODUCTS = [
    # M, N, K, offs
    (1, 16, 16, [1]),
    (1, 128, 128, [0, 1]),
    (8, 256, 384, [1, 2, 3, 4, 5, 6, 7, 8]),
    (5, 144, 272, [0, 0, 5, 5]),
    (40, 400, 1040, [3, 3, 20, 33]),               # rows behind the last group
    (300, 272, 400, [1, 128, 129, 300]),
    (700, 512, 256, [127, 255, 256, 384, 700]),
    (1000, 640, 1168, [500, 400, 900, 2000]),      # out of contract: read as 500, 500, 900, 1000
    (513, 1296, 144, [0, 513]),
    (64, 2064, 4112, [10, 20, 40, 64]),
    (2600, 768, 640, [2600]),
    (260, 48, 2048, [130, 260]),
    (520, 400, 528, [0, 3, 3, 303, 310, 311, 311, 312, 360, 400, 401, 402, 403, 404, 405, 520]),  # uneven
    (1500, 528, 1296, [5, 10, 700, 700, 1500]),
    (97, 1040, 656, [97]),
    (96, 272, 144, [33, 96]),
]


@pytest.mark.parametrize("M,N,K,offs", PRODUCTS)
@pytest.mark.parametrize("transposed", [False, True])
def test_grouped_mm(gq, M, N, K, offs, transposed):
    check_product(gq, M, N, K, offs, transposed)


@pytest.mark.parametrize("rows", [20, 200])  # either kernel
@pytest.mark.parametrize("transposed", [False, True])
def test_grouped_mm_keeps_nan_in_its_group(gq, rows, transposed):
    """NaN in one expert's weights, in one group's rows and behind the last
    group reaches no other group's results (ragged N and K: tiles and
    128-blocks reach past each expert's own)."""
    N, K, E = 272, 400, 4
    M = rows * E + 5
    a, w = product_inputs(rows, M, N, K, E, transposed)
    qa, sa = gq.block_rows(torch.from_numpy(a).to(DEV))
    qb, sb = gq.block_tiles(torch.from_numpy(w).to(DEV))
    o = torch.arange(rows, rows * E + 1, rows, dtype=torch.int32, device=DEV)
    want = gq.grouped_mm(qa, sa, qb, sb, o, transpose_b=transposed)
    qb.view(torch.uint8)[1] = 0x7F
    sb[1] = float("nan")
    qa.view(torch.uint8)[2 * rows:3 * rows] = 0xFF
    sa[2 * rows:3 * rows] = float("nan")
    qa.view(torch.uint8)[E * rows:] = 0x7F
    sa[E * rows:] = float("nan")
    got = gq.grouped_mm(qa, sa, qb, sb, o, transpose_b=transposed)
    gq.check_device_error()
    for g in range(E):
        at = slice(g * rows, (g + 1) * rows)
        if g in (1, 2):
            assert got[at].isnan().all()
        else:
            assert torch.equal(got[at], want[at]), g


def test_grouped_mm_is_deterministic(gq):
    M, N, K, E = 3000, 1040, 1296, 7
    a, w = product_inputs(9, M, N, K, E, False)
    qa, sa = gq.block_rows(torch.from_numpy(a).to(DEV))
    qb, sb = gq.block_tiles(torch.from_numpy(w).to(DEV))
    o = torch.tensor([100, 100, 900, 1500, 1501, 2800, 3000], dtype=torch.int32, device=DEV)
    first = gq.grouped_mm(qa, sa, qb, sb, o)
    for _ in range(10):
        assert torch.equal(gq.grouped_mm(qa, sa, qb, sb, o), first)


@pytest.mark.parametrize("transposed", [False, True])
def test_grouped_mm_many_groups(gq, transposed):
    r = rng(12)
    sizes = r.integers(0, 5, 1000) * (r.random(1000) < 0.6)
    offs = np.cumsum(sizes)
    check_product(gq, int(offs[-1]), 144, 160, offs.tolist(), transposed)


@pytest.mark.parametrize("M", [3000, 20000])  # either kernel
def test_grouped_mm_unordered_ends_of_many_groups(gq, M):
    """Ends that fall back (also below zero) leave empty groups, ends past M
    stop there; more groups than the tile table takes at a time."""
    r = rng(13)
    ends = np.sort(r.integers(0, M, 300))
    back = r.choice(290, 60, replace=False)
    ends[back] = r.integers(-M, np.maximum(ends[back], 1))
    ends[297:] = M + 7, 5, M + 1
    check_product(gq, M, 144, 160, ends.tolist(), False)


def test_grouped_mm_input_and_output_gradient_are_adjoint(gq):
    """The product is linear in A: along any direction D the difference of
    sum(G * out) is sum(G * product(D)), which grad_input has to give as
    sum(product_t(G) * D).  Small integers with unit scales: every sum is
    exact in fp32, and the outputs are held to few enough bits for bf16."""
    M, N, K, offs = 150, 256, 384, [40, 40, 150]
    r = rng(20)
    E = len(offs)

    def fp8(shape, p):
        v = r.integers(-2, 3, shape) * (r.random(shape) < p)
        return torch.from_numpy(v.astype(np.float32)).to(DEV).to(torch.float8_e4m3fn)

    D, G, W = fp8((M, K), 0.2), fp8((M, N), 0.2), fp8((E, N, K), 0.2)
    one = lambda *shape: torch.ones(shape, device=DEV)  # noqa: E731
    o = torch.tensor(offs, dtype=torch.int32, device=DEV)
    sb = one(E, N // 128, K // 128)
    fwd = gq.grouped_mm(D, one(M, K // 128), W, sb, o)
    bwd = gq.grouped_mm(G, one(M, N // 128), W, sb, o, transpose_b=True)
    gq.check_device_error()
    assert fwd.float().abs().max() < 256 and bwd.float().abs().max() < 256  # integers below 2^8: exact in bf16
    assert (fwd.double() * G.double()).sum() == (bwd.double() * D.double()).sum()


def test_past_2_31_elements(gq):
    """Offsets past 31 bits: 65 x 8192 x 4096 weights (2.2e9), 300,000 rows of
    8192 (2.5e9) into and out of expert order, checked on sampled rows."""
    E, N, K = 65, 8192, 4096
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV).normal_()
    qb, sb = gq.block_tiles(w)
    for e in (0, E - 1):
        blocks = w[e].float().view(N // 128, 128, K // 128, 128)
        assert torch.equal(sb[e], 448.0 / blocks.abs().amax((1, 3)).clamp_min(1e-12)) or \
            torch.allclose(sb[e], 448.0 / blocks.abs().amax((1, 3)), rtol=2 ** -22, atol=0)
        err = (qb[e].float().view_as(blocks) / sb[e][:, None, :, None] - blocks).abs()
        assert (err <= blocks.abs() * 2 ** -4 + 2.0 ** -10 / sb[e][:, None, :, None]).all()
    del w
    a = activations(3, 4, K, torch.bfloat16)
    qa, sa = gq.block_rows(a)
    offs = torch.zeros(E, dtype=torch.int32, device=DEV)
    offs[E - 1] = 4
    got = gq.grouped_mm(qa, sa, qb, sb, offs)
    gq.check_device_error()
    want, S, _ = product_plain(qa, sa, qb[E - 1:], sb[E - 1:], [4], False, 4, N)
    assert (np.abs(f32(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * S).all()
    del qb

    T, k, H = 150000, 2, 8192
    ids = torch.from_numpy(rng(5).integers(0, 8, (T, k))).to(DEV)
    order = gq.sort_tokens(ids, 8)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).normal_()
    rows = gq.dispatch(x, order.pos)
    q, s = gq.dispatch_block(x, order.pos)
    plain_q, plain_s = gq.block_rows(x)
    some = torch.from_numpy(rng(6).integers(0, T * k, 2000)).to(DEV)
    some[:2] = torch.tensor([0, T * k - 1])
    token = order.token[some].long()
    assert torch.equal(rows[some], x[token])
    assert torch.equal(q.view(torch.uint8)[some], plain_q.view(torch.uint8)[token])
    assert torch.equal(s[some], plain_s[token])
    w = torch.rand(T, k, device=DEV)
    some = some // k
    pos = order.pos[some].long()
    out = gq.combine(rows, order.pos, w)[some].double()
    want = (rows[pos].double() * w[some, :, None].double()).sum(1)
    assert ((out - want).abs() <= 2 ** -7 * want.abs()).all()  # both rows are the token's own
    dy, dw = gq.combine_backward(x, rows, order.pos, w)
    assert torch.equal(dy[pos], (w[some, :, None] * x[some][:, None].float()).to(torch.bfloat16))
    want = (x[some][:, None].double() * rows[pos].double()).sum(2)
    assert ((dw[some] - want).abs() <= H * 2.0 ** -24 * want).all()  # sums of squares


def test_other_stream_and_graph(gq):
    """The chain on a stream of its own, and replayed from a CUDA graph on
    changed inputs, equals the plain calls."""
    T, k, E, H, N = 50, 4, 8, 256, 384
    ids = torch.from_numpy(rng(30).integers(0, E, (T, k))).to(DEV)
    x = activations(31, T, H, torch.bfloat16)
    w = activations(32, E * N, H, torch.bfloat16).view(E, N, H)
    qb, sb = gq.block_tiles(w)
    wt = torch.rand(T, k, device=DEV)

    def chain():
        order = gq.sort_tokens(ids, E)
        q, s = gq.dispatch_block(x, order.pos)
        return gq.combine(gq.grouped_mm(q, s, qb, sb, order.offs), order.pos, wt)

    want = chain()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = chain()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    x.mul_(-2.0)
    ids.copy_((ids + 3) % E)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, chain())
    gq.check_device_error()


def test_kernels_wait_for_what_the_stream_waits_for(gq):
    """A kernel may be brought up while the one before it runs; between two of
    them, a wait for another stream's event, a copy from the host and a plain
    kernel still come first, and a late reader sees complete results."""
    T, k, E, H = 512, 4, 8, 1024
    r = rng(41)
    ids = torch.from_numpy(r.integers(0, E, (T, k))).to(DEV)
    host = [torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).pin_memory()
            for _ in range(3)]
    busy = torch.randn(4096, 4096, device=DEV)
    x = torch.zeros(3, T, H, dtype=torch.bfloat16, device=DEV)
    late = host[0].to(DEV)
    torch.cuda.synchronize()
    other, mine = torch.cuda.Stream(), torch.cuda.Stream()
    event = torch.cuda.Event()
    with torch.cuda.stream(other):
        for _ in range(20):
            busy = busy @ busy * 1e-3
        x[0].copy_(late)
        event.record()
    with torch.cuda.stream(mine):
        order = gq.sort_tokens(ids, E)
        mine.wait_event(event)
        first = gq.dispatch(x[0], order.pos)
        x[1].copy_(host[1], non_blocking=True)
        second, _ = gq.dispatch_block(x[1], order.pos)
        x[2].copy_(host[2].to(DEV, non_blocking=True))
        third = gq.combine(gq.dispatch(x[2], order.pos), order.pos)
        x.zero_()
    torch.cuda.synchronize()
    pos = order.pos.long()
    assert torch.equal(first[pos], late[:, None].expand(T, k, H))
    q, _ = gq.block_rows(host[1].to(DEV))
    assert torch.equal(second.view(torch.uint8)[pos], q.view(torch.uint8)[:, None].expand(T, k, H))
    assert torch.equal(third, host[2].to(DEV) * k)  # k copies of a row: exact


@pytest.mark.parametrize("T,k,E,H,N", [(1, 8, 16, 512, 256), (96, 4, 8, 1040, 528), (1500, 2, 4, 256, 640)])
def test_steps_that_share_buffers(gq, T, k, E, H, N):
    """Steps on other inputs run one after the other through the same buffers
    and without a stop give what they give alone: no kernel reads or writes a
    buffer that one before it still uses."""
    r = rng(42)
    steps = 40
    x = torch.from_numpy(r.standard_normal((steps, T, H)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    ids = torch.from_numpy(r.integers(0, E, (steps, T, k))).to(DEV)
    wt = torch.from_numpy(r.random((steps, T, k)).astype(np.float32)).to(DEV)
    qw, sw = gq.block_tiles(torch.from_numpy(r.standard_normal((E, N, H)).astype(np.float32)).to(DEV))
    q = torch.empty(T * k, H, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(T * k, -(-H // 128), device=DEV)
    y, dy = (torch.empty(T * k, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dx_rows = torch.empty(T * k, H, dtype=torch.bfloat16, device=DEV)

    def step(i, out, dw, dx, stop):
        order = gq.sort_tokens(ids[i], E)
        stop()
        gq.dispatch_block(x[i], order.pos, out=q, scales=s)
        stop()
        gq.grouped_mm(q, s, qw, sw, order.offs, out=y)
        stop()
        gq.combine(y, order.pos, wt[i], out=out)
        stop()
        gq.combine_backward(out, y, order.pos, wt[i], dy=dy, dweights=dw)
        stop()
        qd, sd = gq.block_rows(dy)
        stop()
        gq.grouped_mm(qd, sd, qw, sw, order.offs, transpose_b=True, out=dx_rows)
        stop()
        gq.combine(dx_rows, order.pos, out=dx)
        stop()

    def run(stop):
        out = torch.empty(steps, T, N, dtype=torch.bfloat16, device=DEV)
        dw = torch.empty(steps, T, k, device=DEV)
        dx = torch.empty(steps, T, H, dtype=torch.bfloat16, device=DEV)
        for i in range(steps):
            step(i, out[i], dw[i], dx[i], stop)
        gq.check_device_error()
        return out, dw, dx

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        for g, w in zip(run(lambda: None), want):
            assert torch.equal(g, w)
    # and the same from one CUDA graph, where nothing but the GPU sets the pace
    out, dw, dx = (torch.zeros_like(w) for w in want)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for i in range(steps):
                step(i, out[i], dw[i], dx[i], lambda: None)
    torch.cuda.synchronize()
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    for g, w in zip((out, dw, dx), want):
        assert torch.equal(g, w)


def test_binding_refuses_bad_arguments(gq):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    w = torch.zeros(4, 2, device=DEV)
    for call in (
        lambda: gq.sort_tokens(pos.float(), 4),
        lambda: gq.sort_tokens(pos[:, :1].expand(4, 2), 4),
        lambda: gq.dispatch(x, pos[:3]),
        lambda: gq.dispatch(x.t(), pos),
        lambda: gq.dispatch(x, pos, out=x.float()),
        lambda: gq.block_rows(x.half()),
        lambda: gq.block_rows(x[:1].expand(4, 64)),
        lambda: gq.block_rows(x, scales=w),
        lambda: gq.dispatch_block(x, None),
        lambda: gq.block_tiles(x),
        lambda: gq.combine(x, pos, w[:3]),
        lambda: gq.combine(x, pos.long(), w),
        lambda: gq.combine_backward(x.float(), x, pos, w),
        lambda: gq.combine_backward(x, x, pos, None),
        lambda: gq.grouped_mm(x.view(torch.uint8), w, x.view(torch.uint8)[None], w[None], pos[:, 0]),
    ):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(gq.GQError):
        gq.sort_tokens(pos, 0)
    with pytest.raises(gq.GQError):
        gq.block_rows(torch.zeros(4, 40, dtype=torch.bfloat16, device=DEV))


def test_grouped_mm_timeout_is_reported_not_hung(gq):
    """A withheld accumulator release makes the first pair's MMAs wait in
    vain: every role leaves its loop after the (shortened) limit, the call
    reports GQ_ERR_TIMEOUT, and the next call is fine."""
    M, N, K = 64, 256, 1024
    qa, sa = gq.block_rows(activations(1, M, K, torch.bfloat16))
    qb, sb = gq.block_tiles(activations(2, N, K, torch.bfloat16)[None])
    o = torch.tensor([M], dtype=torch.int32, device=DEV)
    try:
        gq.debug_set(skip_arrival=True, wait_timeout_ns=5_000_000)
        gq.grouped_mm(qa, sa, qb, sb, o)
        with pytest.raises(gq.GQError) as e:
            gq.check_device_error()
        assert e.value.status == 4
    finally:
        gq.debug_set(False, 0)
    check_product(gq, M, N, K, [M], False)
