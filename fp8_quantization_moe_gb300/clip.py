"""The norm of a list of gradients, and the gradients scaled to a largest norm.

* ``grad_norm(grads)``            -- the norm over all elements of all tensors;
* ``clip_grads(grads, max_norm)`` -- the tensors scaled by min(1, max_norm / norm).

Argument marshalling over include/gq_fp8.h, as in the rest of the binding: the
calls are asynchronous on ``stream`` (default: the current stream), never look
at a value on the host, and can be captured into a CUDA graph, which then holds
the tensors' addresses.
"""
from __future__ import annotations

from array import array
from operator import attrgetter
from typing import Optional, Sequence

import torch

from ._binding import _empty_on, lib
from .moe import _DTYPES, _call, _need, _F32


_data_ptr, _numel = torch.Tensor.data_ptr, torch.Tensor.numel
_device, _contiguous = torch.Tensor.get_device, torch.Tensor.is_contiguous
_dtype = attrgetter("dtype")


def _lists(name: str, what: str, tensors, index: int = -1):
    """(addresses, sizes, type codes, device) of a list of tensors, the first
    three as arrays.  A pass over the list for each attribute, without
    bytecode in between: 0.3 us a tensor, a loop with its checks takes 0.8."""
    if isinstance(tensors, torch.Tensor):
        raise ValueError(f"{name}: {what} must be a list of tensors")
    tensors = list(tensors)
    try:
        devices = set(map(_device, tensors))
        if index >= 0:
            devices.add(index)
        codes = list(map(_DTYPES.get, map(_dtype, tensors)))
        fine = (len(devices) < 2 and -1 not in devices and None not in codes
                and all(map(_contiguous, tensors)))
    except TypeError:  # no tensor
        fine = False
    if not fine:
        _refuse(name, what, tensors, index)
    if devices:
        index = devices.pop()
    return (array("Q", map(_data_ptr, tensors)), array("q", map(_numel, tensors)),
            array("i", codes), index)


def _refuse(name: str, what: str, tensors, index: int):
    """Raises for the first tensor that cannot be taken."""
    for i, t in enumerate(tensors):
        which = f"{name}: {what}[{i}]"
        if not (isinstance(t, torch.Tensor) and t.is_cuda):
            raise ValueError(f"{which} must be a CUDA tensor")
        if t.dtype not in _DTYPES:
            raise ValueError(f"{which} must be bfloat16 or float32, not {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{which} must be contiguous")
        index = t.get_device() if index < 0 else index
        if t.get_device() != index:
            raise ValueError(f"{which} must be on cuda:{index}")


def _address(a: array) -> int:
    return a.buffer_info()[0]


def _norm_buffers(index: int, sizes: array, codes: array, stream):
    """The norm, and the call's scratch where it needs some.  The scratch is not
    kept: what is freed here is handed out again on the same stream only, in that
    stream's order."""
    empty = torch.empty if stream is None else _empty_on(stream, index)
    dev = torch.device("cuda", index)
    size = lib().gq_grad_norm_workspace_bytes(_address(sizes), _address(codes), len(sizes))
    return (empty((), dtype=torch.float32, device=dev),
            empty(size, dtype=torch.uint8, device=dev) if size else None, size)


def grad_norm(grads: Sequence[torch.Tensor], *, stream=None) -> torch.Tensor:
    """sqrt of the sum of the squares of all elements of all tensors.

    grads: contiguous bfloat16 or float32 CUDA tensors of one device, of any
    shapes, both types in one list too; a tensor may come more than once and
    counts each time.  Squares are summed in fp32 over some 32 elements and in
    fp64 beyond, in an order that goes by the sizes and the alignment; no finite
    value overflows on the way.  Returns the norm, a float32 scalar on the device.
    """
    ptrs, sizes, codes, index = _lists("grad_norm", "grads", grads)
    if index < 0:
        raise ValueError("grad_norm: no tensors")
    count = len(ptrs)
    norm, scratch, size = _norm_buffers(index, sizes, codes, stream)
    _call("gq_grad_norm", index, stream, lib().gq_grad_norm, _address(ptrs), _address(sizes),
          _address(codes), count, norm.data_ptr(),
          None if scratch is None else scratch.data_ptr(), size)
    return norm


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, *,
               norm: Optional[torch.Tensor] = None, out: Optional[Sequence[torch.Tensor]] = None,
               stream=None) -> torch.Tensor:
    """Scales the tensors by max_norm / norm where their norm is above
    max_norm, in fp32, rounded once to each tensor's type.

    grads: as in ``grad_norm``, each tensor once.  norm: a float32 scalar on
    the device to use instead of the tensors' own norm (that of more tensors
    than these, say), no element of a tensor that is written.  out: tensors to
    write, of the same types and sizes (each its own gradient, or memory of no
    other); by default the gradients themselves, which are then left alone
    where nothing is to be scaled.
    Returns the norm.  A NaN norm makes every element a NaN, an infinite one
    (also of finite elements, past 3.4e38) every finite element zero.
    ``norm=grad_norm(grads)`` gives the same bits as none.
    """
    name = "clip_grads"
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"{name}: max_norm must be at least 0, not {max_norm}")
    ptrs, sizes, codes, index = _lists(name, "grads", grads)
    if index < 0:
        raise ValueError(f"{name}: no tensors")
    count = len(ptrs)
    outs = None
    if out is not None:
        out_ptrs, out_sizes, out_codes, _ = _lists(name, "out", out, index)
        if out_sizes != sizes or out_codes != codes:
            raise ValueError(f"{name}: out must have the types and sizes of grads")
        outs = _address(out_ptrs)
    scratch, size, given = None, 0, None
    if norm is not None:
        _need(norm, name + ": norm", 0, _F32, index)
        given = norm.data_ptr()
    else:
        norm, scratch, size = _norm_buffers(index, sizes, codes, stream)
    _call("gq_clip_grads", index, stream, lib().gq_clip_grads, _address(ptrs), outs,
          _address(sizes), _address(codes), count, max_norm, given, norm.data_ptr(),
          None if scratch is None else scratch.data_ptr(), size)
    return norm
