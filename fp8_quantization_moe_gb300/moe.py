"""The operators of an fp8 MoE layer around the grouped products.

* ``sort_tokens(ids, n_experts)``    -- stable sort of the tokens' expert choices;
* ``dispatch(x, pos)``               -- token rows copied into expert order;
* ``dispatch_block(x, pos)``         -- the same, quantized per 1x128 block;
* ``block_rows(x)``                  -- rows quantized per 1x128 block;
* ``block_tiles(w)``                 -- stacked weights quantized per 128x128 block;
* ``grouped_mm(qa, sa, qb, sb, offs)`` -- the grouped product of the two;
* ``grouped_gated_mm(qa, sa, qb, sb, offs)`` -- both projections of a gated
  feed-forward block, its activation and product;
* ``gated_backward(g, pre)``         -- the gradients of the two projections;
* ``grouped_gated_grad(qd, sd, qb, sb, offs)`` -- their grad_input;
* ``combine(y, pos, weights)``       -- the weighted way back to the tokens;
* ``combine_backward(g, y, pos, weights)`` -- its gradients.

Argument marshalling over include/gq_fp8.h, as in the rest of the binding:
torch supplies device memory and streams, every call is asynchronous on
``stream`` (default: the current stream), and can be captured into a CUDA
graph.  Outputs that are not passed in are allocated uninitialised, on
``stream``; rows that a call does not write keep what they held.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from ._binding import (GQ_ACT_GELU, GQ_ACT_SILU, GQ_DTYPE_BF16, GQ_DTYPE_F32, GQ_SCALE_POW2,
                       _check, _empty_on, lib)

BLOCK = 128
_DTYPES = {torch.bfloat16: GQ_DTYPE_BF16, torch.float32: GQ_DTYPE_F32}


class TokenOrder(NamedTuple):
    """The order that ``sort_tokens`` found: ``offs`` int32 (n_experts,) end
    offsets, ``pos`` int32 (tokens, top_k) sorted row of each slot (-1:
    dropped), ``token`` int32 (tokens * top_k,) token of each sorted row (-1
    behind the last)."""
    offs: torch.Tensor
    pos: torch.Tensor
    token: torch.Tensor


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


# The largest count of the library's 32-bit arguments, which it refuses: passed
# for every larger one, which ctypes would cut to its lower half.
_MOST = (1 << 31) - 1

# A call on small sizes is as long as its host side: the current stream and
# device are asked for directly (0.1 us each; torch.cuda.current_stream takes
# 2 us), and an argument's checks are one expression.
_raw_stream = torch._C._cuda_getCurrentRawStream
_get_device = torch._C._cuda_getDevice


def _call(name: str, index: int, stream, fn, *args):
    """Calls the library on device ``index``; the stream is its last argument."""
    sh = _raw_stream(index) if stream is None else stream.cuda_stream
    if _get_device() == index:
        st = fn(*args, sh)
    else:
        with torch.cuda.device(index):
            st = fn(*args, sh)
    if st:
        _check(st, name)


def _need(t, what: str, ndim: int, dtypes, index: int = -1, shape=None, contiguous: bool = True):
    """Raises ValueError unless t is a CUDA tensor of that rank, type and, where
    given, device and shape."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == ndim
            and (t.get_device() == index if index >= 0 else t.is_cuda)
            and (shape is None or t.shape == shape) and (not contiguous or t.is_contiguous())):
        return
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype not in dtypes or t.dim() != ndim:
        raise ValueError(f"{what} must be a {ndim}-D tensor of "
                         + " or ".join(str(d).removeprefix("torch.") for d in dtypes))
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if index >= 0 and t.get_device() != index:
        raise ValueError(f"{what} must be on cuda:{index}")
    raise ValueError(f"{what} must be contiguous")


_INT = (torch.int32, torch.int64)
_I32 = (torch.int32,)
_F32 = (torch.float32,)
_FP8 = (torch.float8_e4m3fn, torch.uint8)
_FLOAT = (torch.bfloat16, torch.float32)


def _pitch(x: torch.Tensor, what: str) -> int:
    """Elements from one row of x to the next; the rows themselves are dense."""
    rows, cols = x.shape
    pitch, step = x.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{what} must have dense rows")
    if rows <= 1:
        return cols
    if pitch < cols:
        raise ValueError(f"{what} must have rows that do not overlap")
    return pitch


def sort_tokens(ids: torch.Tensor, n_experts: int, *, stream=None) -> TokenOrder:
    """Stable sort of the tokens' expert choices by expert.

    ids: int32 or int64 (tokens, top_k) CUDA tensor; a slot whose id lies
    outside [0, n_experts) is dropped.  Live slots of one expert keep their
    order (token, then choice).  Returns a TokenOrder.
    """
    _need(ids, "sort_tokens: ids", 2, _INT)
    T, k = ids.shape
    dev = ids.device
    empty = torch.empty if stream is None else _empty_on(stream, dev.index)
    offs = empty(n_experts if n_experts > 0 else 0, dtype=torch.int32, device=dev)
    pos = empty((T, k), dtype=torch.int32, device=dev)
    token = empty(T * k, dtype=torch.int32, device=dev)
    _call("gq_moe_sort", dev.index, stream, lib().gq_moe_sort, ids.data_ptr(), ids.element_size(),
          T, k if k < _MOST else _MOST, n_experts if n_experts < _MOST else _MOST,
          offs.data_ptr(), pos.data_ptr(), token.data_ptr())
    return TokenOrder(offs, pos, token)


def dispatch(x: torch.Tensor, pos: torch.Tensor, *, out=None, stream=None) -> torch.Tensor:
    """Token rows copied into sorted order: out[pos[t, j]] = x[t].

    x: (tokens, H) CUDA tensor of any type, rows of a multiple of 16 bytes,
    possibly with a pitch; pos: int32 (tokens, top_k) of ``sort_tokens``.
    Returns out (rows, H), by default with tokens * top_k rows.  Slots whose
    position lies outside ``out`` are dropped, rows that no slot names keep
    ``out``.  ``dispatch(g, pos)`` is also the gradient of ``combine``
    without weights.
    """
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 2):
        raise ValueError("dispatch: x must be a 2-D CUDA tensor")
    T, H = x.shape
    dev = x.device
    empty = torch.empty if stream is None else _empty_on(stream, dev.index)
    pitch = _pitch(x, "dispatch: x")
    _need(pos, "dispatch: pos", 2, _I32, dev.index)
    if pos.shape[0] != T:
        raise ValueError("dispatch: pos must have a row for each row of x")
    k = pos.shape[1]
    if out is None:
        out = empty((T * k, H), dtype=x.dtype, device=dev)
    else:
        _need(out, "dispatch: out", 2, (x.dtype,), dev.index)
        if out.shape[1] != H:
            raise ValueError(f"dispatch: out must have rows of {H} columns")
    size = x.element_size()
    _call("gq_moe_dispatch", dev.index, stream, lib().gq_moe_dispatch, x.data_ptr(), T, H * size,
          pitch * size, pos.data_ptr(), k if k < _MOST else _MOST, out.shape[0], out.data_ptr())
    return out


def _block_rows(name, x, pos, out, scales, pow2_scales, stream):
    _need(x, name + ": x", 2, _FLOAT, contiguous=False)
    T, K = x.shape
    dev = x.device
    empty = torch.empty if stream is None else _empty_on(stream, dev.index)
    index = dev.index
    pitch = _pitch(x, name + ": x")
    k, rows, to = 1, T, None
    if pos is not None:
        _need(pos, name + ": pos", 2, _I32, index)
        tokens, k = pos.shape
        if tokens != T:
            raise ValueError(f"{name}: pos must have a row for each row of x")
        if T > 0 and k == 0:  # an empty tensor's address is NULL: no positions, a row per token
            raise ValueError(f"{name}: pos must have at least one column")
        rows = T * k
        to = pos.data_ptr()
        if out is not None:
            _need(out, name + ": out", 2, _FP8, index)
            rows = out.shape[0]
    if out is None:
        out = empty((rows, K), dtype=torch.float8_e4m3fn, device=dev)
    else:
        _need(out, name + ": out", 2, _FP8, index, (rows, K))
    if scales is None:
        scales = empty((rows, _blocks(K)), dtype=torch.float32, device=dev)
    else:
        _need(scales, name + ": scales", 2, _F32, index, (rows, _blocks(K)))
    _call("gq_fp8_block_rows", index, stream, lib().gq_fp8_block_rows, x.data_ptr(),
          _DTYPES[x.dtype], T, K, pitch, to, k if k < _MOST else _MOST, rows,
          out.data_ptr(), scales.data_ptr(), GQ_SCALE_POW2 if pow2_scales else 0)
    return out, scales


def block_rows(x: torch.Tensor, *, out=None, scales=None, pow2_scales: bool = False, stream=None):
    """Rows quantized with one scale per 1x128 block: x bf16 or float32 (M, K)
    CUDA tensor, K % 16 == 0, possibly with a pitch.  Returns (q
    float8_e4m3fn (M, K), scales float32 (M, ceil(K / 128)))."""
    return _block_rows("block_rows", x, None, out, scales, pow2_scales, stream)


def dispatch_block(x: torch.Tensor, pos: torch.Tensor, *, out=None, scales=None,
                   pow2_scales: bool = False, stream=None):
    """``dispatch`` of the rows that ``block_rows`` gives: each token is
    quantized once and its row and scales go to the token's sorted rows.
    Returns (q float8_e4m3fn (rows, K), scales float32 (rows,
    ceil(K / 128))), by default with tokens * top_k rows."""
    if pos is None:
        raise ValueError("dispatch_block: pos must be a CUDA tensor")
    return _block_rows("dispatch_block", x, pos, out, scales, pow2_scales, stream)


def block_tiles(w: torch.Tensor, *, out=None, scales=None, pow2_scales: bool = False, stream=None):
    """Stacked expert weights quantized with one scale per 128x128 block: w
    bf16 or float32 (E, N, K) CUDA tensor, K % 16 == 0.  Returns (q
    float8_e4m3fn (E, N, K), scales float32 (E, ceil(N / 128),
    ceil(K / 128)))."""
    _need(w, "block_tiles: w", 3, _FLOAT)
    E, N, K = w.shape
    dev = w.device
    empty = torch.empty if stream is None else _empty_on(stream, dev.index)
    if out is None:
        out = empty((E, N, K), dtype=torch.float8_e4m3fn, device=dev)
    else:
        _need(out, "block_tiles: out", 3, _FP8, dev.index, (E, N, K))
    if scales is None:
        scales = empty((E, _blocks(N), _blocks(K)), dtype=torch.float32, device=dev)
    else:
        _need(scales, "block_tiles: scales", 3, _F32, dev.index, (E, _blocks(N), _blocks(K)))
    _call("gq_fp8_block_tiles", dev.index, stream, lib().gq_fp8_block_tiles, w.data_ptr(),
          _DTYPES[w.dtype], E, N, K, out.data_ptr(), scales.data_ptr(),
          GQ_SCALE_POW2 if pow2_scales else 0)
    return out, scales


def grouped_mm(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor,
               offs: torch.Tensor, *, transpose_b: bool = False, out=None, stream=None):
    """The grouped product of block-quantized rows with block-quantized
    stacked weights, one expert per token group.

    qa e4m3 (M, K) with scales sa float32 (M, ceil(K / 128)) as
    ``block_rows`` or ``dispatch_block`` gives them; qb e4m3 (E, N, K) with
    scales sb float32 (E, ceil(N / 128), ceil(K / 128)) as ``block_tiles``
    gives them; offs int32 (E,) end offsets along M.  Returns out bf16 (M, N)
    = A @ W[g].T for the rows of each group g.  With ``transpose_b`` qa is
    (M, N) and out (M, K) = A @ W[g]: grad_input with the same weights.  Rows
    behind the last end keep ``out``.
    """
    _need(qb, "grouped_mm: qb", 3, _FP8)
    E, N, K = qb.shape
    dev = qb.device
    empty = torch.empty if stream is None else _empty_on(stream, dev.index)
    index = dev.index
    inner, outer = (N, K) if transpose_b else (K, N)
    _need(qa, "grouped_mm: qa", 2, _FP8, index)
    M = qa.shape[0]
    if qa.shape[1] != inner:
        raise ValueError(f"grouped_mm: qa must have {inner} columns, not {qa.shape[1]}")
    _need(sa, "grouped_mm: sa", 2, _F32, index, (M, _blocks(inner)))
    _need(sb, "grouped_mm: sb", 3, _F32, index, (E, _blocks(N), _blocks(K)))
    _need(offs, "grouped_mm: offs", 1, _I32, index, (E,))
    if out is None:
        out = empty((M, outer), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, "grouped_mm: out", 2, (torch.bfloat16,), index, (M, outer))
    _call("gq_grouped_mm", index, stream, lib().gq_grouped_mm, qa.data_ptr(), sa.data_ptr(), M,
          qb.data_ptr(), sb.data_ptr(), N, K, 1 if transpose_b else 0, offs.data_ptr(), E,
          out.data_ptr())
    return out


class GatedRows(NamedTuple):
    """What the gated block's calls write: ``out`` rows unquantized, ``q``
    e4m3 rows with float32 ``scales`` per 1x128 block, ``pre`` bf16 (M, 2, N),
    the two projections; None for what was not asked for."""
    out: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    pre: Optional[torch.Tensor]


_ACTIVATIONS = {"silu": GQ_ACT_SILU, "gelu": GQ_ACT_GELU}
_BF16 = (torch.bfloat16,)


def _activation(name: str, activation: str) -> int:
    code = _ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"{name}: activation must be 'silu' or 'gelu', not {activation!r}")
    return code


def _gated_outputs(name, shape, dtype, dev, plain, fp8, out, q, scales, empty):
    """The buffers of a call's rows, allocated where they are asked for and not given."""
    index = dev.index
    if out is not None:
        _need(out, name + ": out", len(shape), (dtype,), index, shape)
    elif plain:
        out = empty(shape, dtype=dtype, device=dev)
    blocks = (*shape[:-1], _blocks(shape[-1]))
    if q is not None:
        _need(q, name + ": q", len(shape), _FP8, index, shape)
    elif fp8 or scales is not None:
        q = empty(shape, dtype=torch.float8_e4m3fn, device=dev)
    if scales is not None:
        _need(scales, name + ": scales", len(shape), _F32, index, blocks)
    elif q is not None:
        scales = empty(blocks, dtype=torch.float32, device=dev)
    if out is None and q is None:
        raise ValueError(f"{name}: neither plain nor fp8 rows are asked for")
    return out, q, scales


def _gated_weights(name, qb, sb, offs):
    _need(qb, name + ": qb", 4, _FP8)
    E, two, N, K = qb.shape
    if two != 2:
        raise ValueError(f"{name}: qb must have two matrices per expert, not {two}")
    index = qb.get_device()
    _need(sb, name + ": sb", 4, _F32, index, (E, 2, _blocks(N), _blocks(K)))
    _need(offs, name + ": offs", 1, _I32, index, (E,))
    return E, N, K


def grouped_gated_mm(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor,
                     offs: torch.Tensor, *, activation: str = "silu", plain: bool = True,
                     fp8: bool = False, keep: bool = False, out=None, q=None, scales=None,
                     pre=None, pow2_scales: bool = False, stream=None) -> GatedRows:
    """The gated feed-forward block of each expert: act(x) * u for the two
    projections x = A @ W[g, 0].T and u = A @ W[g, 1].T of each group's rows.

    qa e4m3 (M, K) with scales sa float32 (M, ceil(K / 128)) and offs int32
    (E,) as in ``grouped_mm``; qb e4m3 (E, 2, N, K), gate before up, with
    scales sb float32 (E, 2, ceil(N / 128), ceil(K / 128)): ``block_tiles`` of
    the weights viewed as (2 * E, N, K).  activation: "silu", or "gelu" (its
    tanh form).

    Writes the bf16 rows (M, N) with ``plain`` or ``out``; the rows quantized
    as ``block_rows`` does it, from fp32, with ``fp8``, ``q`` or ``scales``;
    and both projections as bf16 (M, 2, N), for ``gated_backward``, with
    ``keep`` or ``pre``.  ``plain=False, fp8=True`` is the form that the next
    ``grouped_mm`` takes.  Rows behind the last end keep what the outputs
    held.
    """
    name = "grouped_gated_mm"
    E, N, K = _gated_weights(name, qb, sb, offs)
    dev = qb.device
    empty = torch.empty if stream is None else _empty_on(stream, dev.index)
    index = dev.index
    act = _activation(name, activation)
    _need(qa, name + ": qa", 2, _FP8, index)
    M = qa.shape[0]
    if qa.shape[1] != K:
        raise ValueError(f"{name}: qa must have {K} columns, not {qa.shape[1]}")
    _need(sa, name + ": sa", 2, _F32, index, (M, _blocks(K)))
    out, q, scales = _gated_outputs(name, (M, N), torch.bfloat16, dev, plain, fp8, out, q, scales, empty)
    if pre is not None:
        _need(pre, name + ": pre", 3, _BF16, index, (M, 2, N))
    elif keep:
        pre = empty((M, 2, N), dtype=torch.bfloat16, device=dev)
    _call("gq_grouped_gated_mm", index, stream, lib().gq_grouped_gated_mm, qa.data_ptr(),
          sa.data_ptr(), M, qb.data_ptr(), sb.data_ptr(), N, K, act, offs.data_ptr(), E,
          None if out is None else out.data_ptr(), None if q is None else q.data_ptr(),
          None if q is None else scales.data_ptr(), None if pre is None else pre.data_ptr(),
          GQ_SCALE_POW2 if pow2_scales else 0)
    return GatedRows(out, q, scales, pre)


def gated_backward(g: torch.Tensor, pre: torch.Tensor, *, activation: str = "silu",
                   plain: bool = True, fp8: bool = False, out=None, q=None, scales=None,
                   pow2_scales: bool = False, stream=None) -> GatedRows:
    """The gradients of the two projections of ``grouped_gated_mm``: g (M, N),
    possibly with a pitch, is the gradient of its rows, pre (M, 2, N) the
    projections, both bf16 or both float32.  Returns GatedRows: out (M, 2, N)
    of g's type (``plain`` or ``out``, which may be ``pre`` itself, but no
    output may overlap an input otherwise), q e4m3 (M, 2, N) and scales float32
    (M, 2, ceil(N / 128)) for ``grouped_gated_grad`` (``fp8``, ``q`` or
    ``scales``)."""
    name = "gated_backward"
    _need(g, name + ": g", 2, _FLOAT, contiguous=False)
    M, N = g.shape
    dev = g.device
    empty = torch.empty if stream is None else _empty_on(stream, dev.index)
    pitch = _pitch(g, name + ": g")
    act = _activation(name, activation)
    _need(pre, name + ": pre", 3, (g.dtype,), dev.index, (M, 2, N))
    out, q, scales = _gated_outputs(name, (M, 2, N), g.dtype, dev, plain, fp8, out, q, scales, empty)
    _call("gq_gated_backward", dev.index, stream, lib().gq_gated_backward, g.data_ptr(),
          pre.data_ptr(), _DTYPES[g.dtype], M, N, pitch, act,
          None if out is None else out.data_ptr(), None if q is None else q.data_ptr(),
          None if q is None else scales.data_ptr(), GQ_SCALE_POW2 if pow2_scales else 0)
    return GatedRows(out, q, scales, None)


def grouped_gated_grad(qd: torch.Tensor, sd: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor,
                       offs: torch.Tensor, *, out=None, stream=None) -> torch.Tensor:
    """grad_input of ``grouped_gated_mm``: the sum of both projections'
    products, D[:, 0] @ W[g, 0] + D[:, 1] @ W[g, 1] for the rows of each group.

    qd e4m3 (M, 2, N) with scales sd float32 (M, 2, ceil(N / 128)) as
    ``gated_backward`` gives them; qb, sb and offs as in ``grouped_gated_mm``.
    Returns out bf16 (M, K).  Rows behind the last end keep ``out``.
    """
    name = "grouped_gated_grad"
    E, N, K = _gated_weights(name, qb, sb, offs)
    dev = qb.device
    empty = torch.empty if stream is None else _empty_on(stream, dev.index)
    index = dev.index
    _need(qd, name + ": qd", 3, _FP8, index)
    M = qd.shape[0]
    if qd.shape[1:] != (2, N):
        raise ValueError(f"{name}: qd must have shape {(M, 2, N)}, not {tuple(qd.shape)}")
    _need(sd, name + ": sd", 3, _F32, index, (M, 2, _blocks(N)))
    if out is None:
        out = empty((M, K), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, name + ": out", 2, _BF16, index, (M, K))
    _call("gq_grouped_gated_grad", index, stream, lib().gq_grouped_gated_grad, qd.data_ptr(),
          sd.data_ptr(), M, qb.data_ptr(), sb.data_ptr(), N, K, offs.data_ptr(), E, out.data_ptr())
    return out


def combine(y: torch.Tensor, pos: torch.Tensor, weights: Optional[torch.Tensor] = None, *,
            out=None, stream=None) -> torch.Tensor:
    """The way back to the tokens: out[t] = sum over j of weights[t, j] *
    y[pos[t, j]], in fp32, rounded once.

    y: bf16 or float32 (rows, H) CUDA tensor, rows of a multiple of 16 bytes;
    pos: int32 (tokens, top_k); weights: float32 (tokens, top_k), or None for
    ones (the gradient of ``dispatch``).  Dropped slots (positions outside
    [0, rows)) add nothing; a token without live slots gets zeros.  Returns
    out (tokens, H) of y's type.
    """
    _need(y, "combine: y", 2, _FLOAT)
    rows, H = y.shape
    dev = y.device
    empty = torch.empty if stream is None else _empty_on(stream, dev.index)
    index = dev.index
    _need(pos, "combine: pos", 2, _I32, index)
    T, k = pos.shape
    if weights is not None:
        _need(weights, "combine: weights", 2, _F32, index, (T, k))
    if out is None:
        out = empty((T, H), dtype=y.dtype, device=dev)
    else:
        _need(out, "combine: out", 2, (y.dtype,), index, (T, H))
    _call("gq_moe_combine", index, stream, lib().gq_moe_combine, y.data_ptr(), _DTYPES[y.dtype],
          rows, H, pos.data_ptr(), None if weights is None else weights.data_ptr(), T,
          k if k < _MOST else _MOST, out.data_ptr())
    return out


def combine_backward(g: torch.Tensor, y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor,
                     *, dy=None, dweights=None, stream=None):
    """The gradients of ``combine`` with weights: g (tokens, H) is the
    gradient of its output, of y's type.  Returns (dy (rows, H) =
    weights[t, j] * g[t] at row pos[t, j], dweights float32 (tokens, top_k) =
    <g[t], y[pos[t, j]]>, 0 for a dropped slot).  Rows of dy that no slot
    names keep ``dy``."""
    _need(y, "combine_backward: y", 2, _FLOAT)
    rows, H = y.shape
    dev = y.device
    empty = torch.empty if stream is None else _empty_on(stream, dev.index)
    index = dev.index
    _need(pos, "combine_backward: pos", 2, _I32, index)
    T, k = pos.shape
    _need(g, "combine_backward: g", 2, (y.dtype,), index, (T, H))
    _need(weights, "combine_backward: weights", 2, _F32, index, (T, k))
    if dy is None:
        dy = empty((rows, H), dtype=y.dtype, device=dev)
    else:
        _need(dy, "combine_backward: dy", 2, (y.dtype,), index, (rows, H))
    if dweights is None:
        dweights = empty((T, k), dtype=torch.float32, device=dev)
    else:
        _need(dweights, "combine_backward: dweights", 2, _F32, index, (T, k))
    _call("gq_moe_combine_backward", index, stream, lib().gq_moe_combine_backward, g.data_ptr(),
          y.data_ptr(), _DTYPES[y.dtype], rows, H, pos.data_ptr(), weights.data_ptr(), T,
          k if k < _MOST else _MOST, dy.data_ptr(), dweights.data_ptr())
    return dy, dweights
