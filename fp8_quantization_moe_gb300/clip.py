"""The norm of a list of gradients, and the gradients scaled to a largest norm.

* ``grad_norm(grads)``            -- the norm over all elements of all tensors;
* ``clip_grads(grads, max_norm)`` -- the tensors scaled by min(1, max_norm / norm).

Argument marshalling over include/gq_fp8.h, as in the rest of the binding: the
calls are asynchronous on ``stream`` (default: the current stream), never look
at a value on the host, and can be captured into a CUDA graph, which then holds
the tensors' addresses.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from ._binding import _empty_on, lib
from .moe import _DTYPES, _call, _need, _F32


def _lists(name: str, what: str, tensors, index: int = -1):
    """(addresses, sizes, type codes, device) of a list of tensors, as C arrays."""
    if isinstance(tensors, torch.Tensor):
        raise ValueError(f"{name}: {what} must be a list of tensors")
    tensors = list(tensors)
    if index < 0 and tensors and isinstance(tensors[0], torch.Tensor):
        index = tensors[0].get_device()
    codes = []
    for i, t in enumerate(tensors):
        code = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
        if code is None or index < 0 or t.get_device() != index or not t.is_contiguous():
            _refuse(name, f"{what}[{i}]", t, index)
        codes.append(code)
    n = len(tensors)
    return ((ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors]),
            (ctypes.c_int64 * n)(*[t.numel() for t in tensors]), (ctypes.c_int32 * n)(*codes),
            index, tensors)


def _refuse(name: str, what: str, t, index: int):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError(f"{name}: {what} must be a CUDA tensor")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name}: {what} must be bfloat16 or float32, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: {what} must be contiguous")
    raise ValueError(f"{name}: {what} must be on cuda:{index}")


def _norm_buffers(index: int, count: int, stream):
    """The norm and the call's scratch.  The scratch is not kept: what is freed
    here is handed out again on the same stream only, in that stream's order."""
    empty = torch.empty if stream is None else _empty_on(stream, index)
    dev = torch.device("cuda", index)
    size = lib().gq_grad_norm_workspace_bytes(count)
    return (empty((), dtype=torch.float32, device=dev),
            empty(size, dtype=torch.uint8, device=dev), size)


def grad_norm(grads: Sequence[torch.Tensor], *, stream=None) -> torch.Tensor:
    """sqrt of the sum of the squares of all elements of all tensors.

    grads: contiguous bfloat16 or float32 CUDA tensors of one device, of any
    shapes, both types in one list too; a tensor may come more than once and
    counts each time.  Squares are summed in fp32 over 32 elements and in fp64
    beyond, in a fixed order; no finite value overflows on the way.  Returns
    the norm, a float32 scalar on the device.
    """
    ptrs, sizes, codes, index, grads = _lists("grad_norm", "grads", grads)
    if index < 0:
        raise ValueError("grad_norm: no tensors")
    norm, scratch, size = _norm_buffers(index, len(grads), stream)
    _call("gq_grad_norm", index, stream, lib().gq_grad_norm, ptrs, sizes, codes, len(grads),
          norm.data_ptr(), scratch.data_ptr(), size)
    return norm


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, *,
               norm: Optional[torch.Tensor] = None, out: Optional[Sequence[torch.Tensor]] = None,
               stream=None) -> torch.Tensor:
    """Scales the tensors by max_norm / norm where their norm is above
    max_norm, in fp32, rounded once to each tensor's type.

    grads: as in ``grad_norm``, each tensor once.  norm: a float32 scalar on
    the device to use instead of the tensors' own norm (that of more tensors
    than these, say).  out: tensors to write, of the same types and sizes
    (each its own gradient, or memory of no other); by default the gradients
    themselves, which are then left alone where nothing is to be scaled.
    Returns the norm.  A NaN norm makes every element a NaN, an infinite one
    every finite element zero.
    """
    name = "clip_grads"
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"{name}: max_norm must be at least 0, not {max_norm}")
    ptrs, sizes, codes, index, grads = _lists(name, "grads", grads)
    if index < 0:
        raise ValueError(f"{name}: no tensors")
    outs = None
    if out is not None:
        outs, out_sizes, out_codes, _, out = _lists(name, "out", out, index)
        if len(out) != len(grads) or out_sizes[:] != sizes[:] or out_codes[:] != codes[:]:
            raise ValueError(f"{name}: out must have the types and sizes of grads")
    if norm is not None:
        _need(norm, name + ": norm", 0, _F32, index)
        _call("gq_clip_grads", index, stream, lib().gq_clip_grads, ptrs, outs, sizes, codes,
              len(grads), max_norm, norm.data_ptr(), None, None, 0)
        return norm
    norm, scratch, size = _norm_buffers(index, len(grads), stream)
    _call("gq_clip_grads", index, stream, lib().gq_clip_grads, ptrs, outs, sizes, codes,
          len(grads), max_norm, None, norm.data_ptr(), scratch.data_ptr(), size)
    return norm
