"""The MoE-layer operators at their edges: what the plain sizes do not reach."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def gq():
    import __graft_entry__

    __graft_entry__.build()
    import fp8_quantization_moe_gb300 as m

    return m


def randn(seed, *shape, dtype=torch.bfloat16):
    r = np.random.default_rng(seed)
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(DEV).to(dtype)


def draw_ids(seed, T, k, E, local):
    ids = torch.from_numpy(np.random.default_rng(seed).integers(0, E, (T, k))).to(DEV)
    return torch.where(ids < local, ids, -1)


# ------------------------------------------------------------------ slots --

def test_dispatch_block_refuses_tokens_without_slots(gq):
    """An empty position array has no address; it must not be taken for the
    call without positions, which writes a row per token."""
    x = randn(1, 4, 64)
    pos = torch.empty(4, 0, dtype=torch.int32, device=DEV)
    out = torch.full((4, 64), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((4, 1), -3.0, device=DEV)
    with pytest.raises(ValueError):
        gq.dispatch_block(x, pos, out=out, scales=scales)
    assert (out == 0x5A).all() and (scales == -3.0).all()
    with pytest.raises(ValueError):
        gq.dispatch_block(x, pos)
    q, s = gq.dispatch_block(x[:0], pos[:0])  # no tokens either: nothing to do
    assert q.shape == (0, 64) and s.shape == (0, 1)


def test_counts_past_32_bits_are_refused(gq):
    """The library takes slots per token and experts as 32-bit numbers; larger
    ones are not cut to their lower half."""
    many = torch.empty(1, 2 ** 32 + 2, dtype=torch.int32, device=DEV)
    many[:, :2] = 0
    x = randn(2, 1, 64)
    out, scales = torch.zeros(1, 64, dtype=torch.float8_e4m3fn, device=DEV), torch.zeros(1, 1, device=DEV)
    for call in (
        lambda: gq.sort_tokens(many, 4),
        lambda: gq.dispatch(x, many, out=x.clone()),
        lambda: gq.dispatch_block(x, many, out=out, scales=scales),
        lambda: gq.combine(x, many),
        lambda: gq.sort_tokens(torch.zeros(1, 1, dtype=torch.int32, device=DEV), 2 ** 32 + 4),
    ):
        with pytest.raises(gq.GQError) as e:
            call()
        assert e.value.status == 2
        torch.cuda.empty_cache()


def outside(rows, T, k, seed):
    """Positions of which about half lie outside a buffer of `rows` rows."""
    r = np.random.default_rng(seed)
    pos = np.full(T * k, -1, np.int64)
    inside = r.permutation(T * k)[:rows]
    pos[inside] = r.permutation(rows)[:inside.size]
    bad = pos < 0
    pos[bad] = r.choice([-1, -5, -2 ** 31, rows, rows + 1, rows + 1000, 2 ** 31 - 1], bad.sum())
    return torch.from_numpy(pos.reshape(T, k).astype(np.int32)).to(DEV)


@pytest.mark.parametrize("T,k,rows,H,dtype", [
    (60, 4, 100, 264, torch.bfloat16), (33, 3, 40, 136, torch.float32), (20, 12, 130, 2064, torch.bfloat16),
    (5, 2, 0, 64, torch.bfloat16),  # an empty row buffer: every position is outside
])
def test_positions_outside_the_rows_are_dropped_slots(gq, T, k, rows, H, dtype):
    pos = outside(rows, T, k, T)
    live = (pos >= 0) & (pos < rows)
    plain = torch.where(live, pos, -1)
    y, g, w = randn(3, rows, H, dtype=dtype), randn(4, T, H, dtype=dtype), torch.rand(T, k, device=DEV)
    out = gq.combine(y, pos, w)
    assert torch.equal(out, gq.combine(y, plain, w))
    assert (out[~live.any(1)] == 0).all()
    dy, dw = gq.combine_backward(g, y, pos, w, dy=torch.full_like(y, 7.0))
    dy2, dw2 = gq.combine_backward(g, y, plain, w, dy=torch.full_like(y, 7.0))
    assert torch.equal(dy, dy2) and torch.equal(dw, dw2)
    assert (dw[~live] == 0).all()
    t, j = live.nonzero(as_tuple=True)
    if H % 16 == 0:
        q = torch.full((rows, H), 0x5A, dtype=torch.uint8, device=DEV)
        s = torch.full((rows, -(-H // 128)), -3.0, device=DEV)
        gq.dispatch_block(g, pos, out=q, scales=s)
        want_q, want_s = gq.block_rows(g)
        at = pos[t, j].long()
        assert torch.equal(q[at], want_q.view(torch.uint8)[t]) and torch.equal(s[at], want_s[t])
        named = torch.zeros(rows, dtype=torch.bool, device=DEV)
        named[at] = True
        assert (q[~named] == 0x5A).all() and (s[~named] == -3.0).all()


# ----------------------------------------------------- non-finite values --

def holes(seed, R, K):
    """A mask of single elements, whole and half 16-column units, and whole
    128-blocks."""
    r = np.random.default_rng(seed)
    m = r.random((R, K)) < 0.01
    for _ in range(R // 2):
        row, unit = r.integers(R), 16 * r.integers(K // 16)
        m[row, unit + r.integers(2):unit + 16:r.integers(1, 3)] = True
        m[r.integers(R), unit:unit + 16] = True
    m[R // 3, :128] = True
    return torch.from_numpy(m).to(DEV)


@pytest.mark.parametrize("form", ["rows", "dispatch", "tiles"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_block_scales_do_not_count_nan(gq, form, dtype):
    """A NaN becomes e4m3's NaN and counts for nothing in its block's scale,
    wherever it stands and in either type: the block's other values are
    quantized as if it were zero."""
    R, K = 130, 400
    x, nan = randn(5, R, K, dtype=dtype), holes(6, R, K)

    def quantized(v):
        if form == "rows":
            return gq.block_rows(v)
        if form == "tiles":
            return gq.block_tiles(v.view(2, R // 2, K))
        return gq.dispatch_block(v, torch.arange(R, dtype=torch.int32, device=DEV).flip(0)[:, None])

    want_q, want_s = quantized(x.masked_fill(nan, 0.0))
    for sign in (1.0, -1.0):
        q, s = quantized(x.masked_fill(nan, 0.0) + torch.where(nan, sign * NAN, 0.0).to(dtype))
        at = nan.flip(0) if form == "dispatch" else nan
        assert torch.equal(s, want_s)
        q, wq = q.view(torch.uint8).reshape(R, K), want_q.view(torch.uint8).reshape(R, K)
        assert ((q[at] & 0x7F) == 0x7F).all()
        assert torch.equal(q[~at], wq[~at])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinities_stay_in_their_block(gq, dtype):
    """An infinite row leaves the other rows of a 1x128 quantization as they
    are, an infinite element the other tiles of a matrix."""
    R, K = 200, 400
    x = randn(7, R, K, dtype=dtype)
    want_q, want_s = gq.block_rows(x)
    bad = x.clone()
    bad[3], bad[150, 200] = INF, -INF
    q, s = gq.block_rows(bad)
    keep = torch.ones(R, 4, dtype=torch.bool, device=DEV)
    keep[3], keep[150, 1] = False, False
    assert torch.equal(s[keep], want_s[keep])
    cols = keep.repeat_interleave(128, 1)[:, :K]
    assert torch.equal(q.view(torch.uint8)[cols], want_q.view(torch.uint8)[cols])
    tq, ts = gq.block_tiles(x[None])
    bq, bs = gq.block_tiles(torch.where(torch.arange(R * K, device=DEV).view(R, K) == 150 * K + 200, INF, x)[None].to(dtype))
    tile = torch.zeros(2, 4, dtype=torch.bool, device=DEV)
    tile[1, 1] = True
    assert torch.equal(bs[0][~tile], ts[0][~tile])
    cols = tile.repeat_interleave(128, 0)[:R].repeat_interleave(128, 1)[:, :K]
    assert torch.equal(bq[0].view(torch.uint8)[~cols], tq[0].view(torch.uint8)[~cols])


@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_combine_keeps_non_finite_values_in_their_token(gq, value):
    """Behind the last group, in the weight of a dropped slot and in another
    token's rows they count for nothing."""
    T, k, H = 70, 4, 264
    order = gq.sort_tokens(draw_ids(8, T, k, 8, 5), 5)
    y, g, w = randn(9, T * k, H), randn(10, T, H), torch.rand(T, k, device=DEV)
    dead = order.pos < 0
    want = gq.combine(y, order.pos, w)
    want_dy, want_dw = gq.combine_backward(g, y, order.pos, w, dy=torch.zeros_like(y))
    t = int((~dead).sum(1).argmax())
    r = order.pos[t][~dead[t]][0].long()
    y[int(order.offs[-1]):] = value
    y[r] = value
    w = torch.where(dead, value, w)
    out = gq.combine(y, order.pos, w)
    dy, dw = gq.combine_backward(g, y, order.pos, w, dy=torch.zeros_like(y))
    others = torch.arange(T, device=DEV) != t
    assert torch.equal(out[others], want[others]) and torch.equal(dw[others], want_dw[others])
    assert not out[t].isfinite().any()
    assert torch.equal(dy, want_dy)  # dy does not read y


@pytest.mark.parametrize("rows", [20, 200])  # either kernel
@pytest.mark.parametrize("transposed", [False, True])
def test_grouped_mm_keeps_infinities_in_their_group(gq, rows, transposed):
    """Infinities in one expert's weights, in one group's rows and behind the
    last group, quantized as they come, reach no other group's results."""
    N, K, E = 272, 400, 4
    M = rows * E + 5
    inner = N if transposed else K
    x, w = randn(11, M, inner), randn(12, E, N, K)
    o = torch.arange(rows, rows * E + 1, rows, dtype=torch.int32, device=DEV)
    want = gq.grouped_mm(*gq.block_rows(x), *gq.block_tiles(w), o, transpose_b=transposed)
    w[1, ::7] = INF
    x[2 * rows:3 * rows, 5] = -INF
    x[E * rows:] = INF
    got = gq.grouped_mm(*gq.block_rows(x), *gq.block_tiles(w), o, transpose_b=transposed)
    gq.check_device_error()
    for g in range(E):
        at = slice(g * rows, (g + 1) * rows)
        if g in (1, 2):
            assert not got[at].isfinite().any()
        else:
            assert torch.equal(got[at], want[at]), g


# ------------------------------------------------------------ large sizes --

@pytest.mark.parametrize("M,E,outer,inner", [(530_000, 3, 4096, 128), (40_000, 1024, 65_536, 16)])  # either kernel
@pytest.mark.parametrize("transposed", [False, True])
def test_grouped_mm_outputs_past_2_31_elements(gq, M, E, outer, inner, transposed):
    """Entries -2 .. 2 of which one in five is not zero, with unit scales: the
    results are integers below 256, which bf16 holds, and the test is exact."""
    gen = torch.Generator(device=DEV).manual_seed(M)

    def fp8(*shape):
        v = torch.randint(-2, 3, shape, device=DEV, generator=gen, dtype=torch.int8)
        keep = torch.randint(0, 4, shape, device=DEV, generator=gen, dtype=torch.int8) == 0
        return (v * keep).to(torch.float8_e4m3fn)

    qa, w = fp8(M, inner), fp8(E, *((inner, outer) if transposed else (outer, inner)))
    sb = torch.ones(E, -(-w.shape[1] // 128), -(-w.shape[2] // 128), device=DEV)
    offs = torch.randint(0, M + 1, (E,), device=DEV, generator=gen).sort().values.to(torch.int32)
    offs[-1] = M
    out = gq.grouped_mm(qa, torch.ones(M, 1, device=DEV), w, sb, offs, transpose_b=transposed)
    gq.check_device_error()
    assert out.numel() > 2 ** 31
    start = 0
    for e, end in enumerate(offs.tolist()):
        for at in range(start, end, 50_000):
            rows = slice(at, min(end, at + 50_000))
            m = w[e].float()
            want = qa[rows].float() @ (m if transposed else m.t())
            assert want.abs().max() < 256
            assert torch.equal(out[rows].float(), want), e
        start = end


# ---------------------------------------------------------------- streams --

def stream_of(t):
    """The stream whose pool the allocator took t's memory from."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def test_outputs_belong_to_the_stream_of_the_call(gq):
    """A call on another stream takes its outputs from that stream's memory:
    what the current stream has freed may still be in use there."""
    T, k, E, H, N = 64, 4, 8, 256, 128
    x, w, g, ids = randn(13, T, H), randn(14, E, N, H), randn(15, T, N), draw_ids(16, T, k, E, E)
    wt = torch.rand(T, k, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, torch.cuda.ExternalStream(side.cuda_stream)):
        order = gq.sort_tokens(ids, E, stream=stream)
        rows = gq.dispatch(x, order.pos, stream=stream)
        q, s = gq.dispatch_block(x, order.pos, stream=stream)
        q2, s2 = gq.block_rows(x, stream=stream)
        qw, sw = gq.block_tiles(w, stream=stream)
        y = gq.grouped_mm(q, s, qw, sw, order.offs, stream=stream)
        out = gq.combine(y, order.pos, wt, stream=stream)
        dy, dw = gq.combine_backward(g, y, order.pos, wt, stream=stream)
        for t in (*order, rows, q, s, q2, s2, qw, sw, y, out, dy, dw):
            assert stream_of(t) == side.cuda_stream
        torch.cuda.synchronize()
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    assert stream_of(gq.block_rows(x)[0]) == torch.cuda.default_stream().cuda_stream
    assert stream_of(gq.block_rows(x, stream=torch.cuda.default_stream())[0]) == torch.cuda.default_stream().cuda_stream


def test_outputs_of_the_per_group_calls_belong_to_the_stream_of_the_call(gq):
    """The same of the calls that scale per token group."""
    M, K, G = 256, 128, 4
    x, w = randn(22, M, K), randn(23, G, K, K)
    xt = x.t().contiguous()
    offs = torch.arange(M // G, M + 1, M // G, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q, s = gq.colwise(x, offs, stream=side)
    qt, st = gq.rowwise_t(xt, offs, stream=side)
    outs = [q, s, qt, st, gq.grouped_wgrad(qt, st, q, s, offs, stream=side)]
    for call in (gq.expert_dim1, gq.expert_rowwise):
        outs += call(w, stream=side)
    outs += gq.mxfp8_dim0(x, stream=side)
    outs += gq.colwise_noalloc(x, offs, stream=side)
    torch.cuda.synchronize()
    gq.check_device_error()
    assert len(outs) == 13
    assert all(stream_of(t) == side.cuda_stream for t in outs)


def test_chain_on_a_passed_stream_beside_the_current_one(gq):
    """The chain with stream=, while the current stream frees and allocates
    buffers of the same sizes, gives what it gives alone."""
    T, k, E, H, N = 256, 4, 8, 512, 384
    x, w, wt = randn(17, T, H), randn(18, E, N, H), torch.rand(T, k, device=DEV)
    ids = draw_ids(19, T, k, E, 6)
    qw, sw = gq.block_tiles(w)

    def chain(stream=None):
        order = gq.sort_tokens(ids, E, stream=stream)
        q, s = gq.dispatch_block(x, order.pos, stream=stream)
        y = gq.grouped_mm(q, s, qw, sw, order.offs, stream=stream)
        return gq.combine(y, order.pos, wt, stream=stream)

    want = chain()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    sums, kept = [], torch.ones(T * k, N, dtype=torch.bfloat16, device=DEV)
    for _ in range(30):
        # twins of the chain's buffers, read on the current stream after they were freed
        for shape, dtype in (((T * k, H), torch.uint8), ((T * k, N), torch.bfloat16), ((T, N), torch.bfloat16)):
            b = torch.ones(shape, dtype=dtype, device=DEV)
            sums.append((b.double().sum(), b.numel()))
            del b
        kept = kept @ torch.eye(N, dtype=torch.bfloat16, device=DEV)
        got.append(chain(side))
    torch.cuda.synchronize()
    gq.check_device_error()
    assert all(torch.equal(g, want) for g in got)
    assert all(float(s) == n for s, n in sums) and (kept == 1).all()


# ------------------------------------------------------------------ waits --

@pytest.mark.parametrize("M", [40, 64])  # either kernel
@pytest.mark.parametrize("transposed", [False, True])
def test_grouped_mm_waits_run_out(gq, M, transposed):
    """A withheld accumulator release makes the first block's MMAs wait in vain
    (eight 128-blocks, more than either kernel has accumulators): every role
    leaves its loop after the shortened limit, the status is GQ_ERR_TIMEOUT,
    and the next call is right."""
    N, K = (1024, 256) if transposed else (256, 1024)
    qa, sa = gq.block_rows(randn(20, M, 1024))
    qb, sb = gq.block_tiles(randn(21, 1, N, K))
    o = torch.tensor([M], dtype=torch.int32, device=DEV)
    want = gq.grouped_mm(qa, sa, qb, sb, o, transpose_b=transposed)
    gq.check_device_error()
    try:
        gq.debug_set(skip_arrival=True, wait_timeout_ns=5_000_000)
        gq.grouped_mm(qa, sa, qb, sb, o, transpose_b=transposed)
        with pytest.raises(gq.GQError) as e:
            gq.check_device_error()
        assert e.value.status == 4
    finally:
        gq.debug_set(False, 0)
    assert torch.equal(gq.grouped_mm(qa, sa, qb, sb, o, transpose_b=transposed), want)
    gq.check_device_error()
