"""Global norm and clipping of gradients (argument marshalling only).

What lies between the gradients of a model and its optimizer: the norm of
all of them together, and all of them scaled so that it is at most a bound;
``include/gemm_f32.h`` (gemm_f32_grad_*) gives the formulas.  Asynchronous on
``stream`` (None: the current one); the norm stays on the device.

    norm = clip_([dx, dw], 1.0)       # in place; norm: float32, one element

Gradients are CUDA tensors of bfloat16, float16 or float32, mixed as they
come, all on one device: contiguous of any shape, or matrices with rows
further apart (a view's, or a padded one's); a tensor that is to be clipped is
listed once.  A norm that is not finite clips nothing.  Autograd records none
of this.
"""

from __future__ import annotations

import array
import itertools

import torch

from . import gemm as _g
from .loss import _bytes, _new, _on, _stream

__all__ = ["global_norm", "clip_", "workspace_size"]

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def workspace_size(tensors) -> int:
    """Workspace bytes for a number of gradients."""
    n = int(_g.lib().gemm_f32_grad_workspace_size(int(tensors)))
    if n < 0:
        _g._check(-n, "gemm_f32_grad_workspace_size")
    return n


def _row_step(t, shape, name):
    """The leading dimension of a matrix whose rows are apart."""
    if len(shape) == 2:
        step, one = t.stride()
        if (one == 1 or shape[1] == 1) and step >= shape[1]:
            return step
    raise ValueError(f"{name} must be contiguous, or a matrix whose rows "
                     "are, one behind the other")


_ptr, _device = torch.Tensor.data_ptr, torch.Tensor.get_device
_numel, _whole = torch.Tensor.numel, torch.Tensor.is_contiguous
_ONES = itertools.repeat(1)


def _checked(tensors, name):
    """(device index, data types) of a list of CUDA tensors."""
    if not all(issubclass(k, torch.Tensor) for k in set(map(type, tensors))):
        raise TypeError(f"{name} must be torch tensors")
    kinds = [t.dtype for t in tensors]
    if not _TYPES.keys() >= set(kinds):
        raise TypeError(f"{name} must be bfloat16, float16 or float32 torch "
                        "tensors")
    where = set(map(_device, tensors))
    if min(where) < 0 or not tensors[0].is_cuda:  # (-1: the host's)
        raise ValueError(f"{name} must live on a CUDA device")
    if len(where) > 1:
        raise ValueError(f"{name} must live on one device")
    return where.pop(), kinds


def _table(tensors, out):
    """gemm_f32_grad of each tensor, and their device.  (A column of the table
    at a time: a model has hundreds of gradients, and what is done for each is
    the time of a call.)"""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("no gradients: the device of their norm is unknown")
    index, kinds = _checked(tensors, "gradients")
    n = len(tensors)
    whole, whole_out = list(map(_whole, tensors)), _ONES
    at, sizes = list(map(_ptr, tensors)), list(map(_numel, tensors))
    targets, to = tensors, at
    if out is not None:
        targets = list(out)
        if len(targets) != n:
            raise ValueError("out must have a tensor for each gradient")
        where, kinds_out = _checked(targets, "out")
        if where != index:
            raise ValueError("out must live on the gradients' device")
        if kinds_out != kinds:
            raise TypeError("out must have the gradients' types")
        if list(map(_numel, targets)) != sizes:
            raise ValueError("out must have the gradients' shapes")
        to = list(map(_ptr, targets))
        whole_out = list(map(_whole, targets))
    table = array.array("q", itertools.chain.from_iterable(
        zip(at, to, _ONES, sizes, sizes, sizes, map(_TYPES.get, kinds))))
    if not (all(whole) and (whole_out is _ONES or all(whole_out))):
        if whole_out is _ONES:
            whole_out = whole
        for i, (t, o) in enumerate(zip(tensors, targets)):
            if whole[i] and whole_out[i]:
                continue
            shape = t.shape
            if o is not t and o.shape != shape:
                raise ValueError("out must have the gradients' shapes")
            ld = 0 if whole[i] else _row_step(t, shape, "gradients")
            ld_out = ld if o is t else \
                0 if whole_out[i] else _row_step(o, shape, "out")
            rows, cols = shape
            k = 7 * i
            table[k + 2], table[k + 3] = rows, cols
            table[k + 4], table[k + 5] = ld or cols, ld_out or cols
    return table, n, tensors[0].device


def _scratch(workspace, n, device, stream):
    """(workspace, pointer, bytes), allocated when not given."""
    if workspace is None:
        workspace = _new(workspace_size(n), torch.uint8, device, stream)
    return _bytes(workspace, "workspace", device, "the gradients'")


def global_norm(tensors, workspace=None, stream=None):
    """The norm of all elements of all tensors (float32, one element)."""
    table, n, device = _table(tensors, None)
    with _on(device):
        norm = _new(1, torch.float32, device, stream)
        workspace, wp, size = _scratch(workspace, n, device, stream)
        st = _g.lib().gemm_f32_grad_norm(n, table.buffer_info()[0],
                                         norm.data_ptr(), wp, size,
                                         _stream(stream, device))
    if st:
        _g._check(st, "gemm_f32_grad_norm")
    return norm


def clip_(tensors, max_norm, out=None, workspace=None, stream=None):
    """Scales the tensors by min(1, max_norm / norm), in place or into
    ``out``; returns their norm before it (float32, one element).  out: a
    tensor for each, of its type and shape and in memory of its own (of a
    contiguous gradient also another shape of as many elements, as a piece of
    a flat buffer)."""
    table, n, device = _table(tensors, out)
    with _on(device):
        norm = _new(1, torch.float32, device, stream)
        workspace, wp, size = _scratch(workspace, n, device, stream)
        st = _g.lib().gemm_f32_grad_clip(n, table.buffer_info()[0],
                                         float(max_norm), norm.data_ptr(), wp,
                                         size, _stream(stream, device))
    if st:
        _g._check(st, "gemm_f32_grad_clip")
    return norm
