"""Global norm and clipping of gradients (argument marshalling only).

What lies between the gradients of a model and its optimizer: the norm of
all of them together, and all of them scaled so that it is at most a bound;
``include/gemm_f32.h`` (gemm_f32_grad_*) gives the formulas.  Asynchronous on
``stream`` (None: the current one); the norm stays on the device.

    norm = clip_([dx, dw], 1.0)       # in place; norm: float32, one element

Gradients are CUDA tensors of bfloat16, float16 or float32, mixed as they
come, all on one device: contiguous of any shape, or matrices with rows
further apart (a view's, or a padded one's).  A norm that is not finite clips
nothing.  Autograd records none of this.
"""

from __future__ import annotations

import array

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


def _rows(t, name):
    """(rows, columns, leading dimension): one row of a contiguous tensor."""
    if t.is_contiguous():
        n = t.numel()
        return 1, n, n
    if t.dim() == 2:
        rows, cols = t.shape
        step, one = t.stride()
        if (one == 1 or cols == 1) and (step >= cols or rows == 1):
            return rows, cols, step if rows > 1 else cols
    raise ValueError(f"{name} must be contiguous, or a matrix whose rows "
                     "are, one behind the other")


def _table(tensors, out):
    """gemm_f32_grad of each tensor, and their device."""
    tensors = list(tensors)
    for t in tensors:
        if not isinstance(t, torch.Tensor) or t.dtype not in _TYPES:
            raise TypeError("gradients must be bfloat16, float16 or float32 "
                            "torch tensors")
        if not t.is_cuda:
            raise ValueError("gradients must live on a CUDA device")
    if not tensors:
        raise ValueError("no gradients: the device of their norm is unknown")
    device = tensors[0].device
    index = device.index
    targets = tensors
    if out is not None:
        targets = list(out)
        if len(targets) != len(tensors):
            raise ValueError("out must have a tensor for each gradient")
    table = array.array("q")
    for t, o in zip(tensors, targets):
        if t.get_device() != index:
            raise ValueError("gradients must live on one device")
        if o is t:
            if t.is_contiguous():
                p, n = t.data_ptr(), t.numel()
                table.extend((p, p, 1, n, n, n, _TYPES[t.dtype]))
                continue
            rows, cols, ld = _rows(t, "a gradient")
            p, q, ld_out = t.data_ptr(), t.data_ptr(), ld
        else:
            if not isinstance(o, torch.Tensor) or o.dtype != t.dtype:
                raise TypeError("out must have the gradients' types")
            if o.shape != t.shape:
                raise ValueError("out must have the gradients' shapes")
            if o.get_device() != index:
                raise ValueError("out must live on the gradients' device")
            p, q = t.data_ptr(), o.data_ptr()
            if t.is_contiguous() and o.is_contiguous():
                n = t.numel()
                table.extend((p, q, 1, n, n, n, _TYPES[t.dtype]))
                continue
            rows, cols, ld = _rows(t, "a gradient")
            rows2, cols2, ld_out = _rows(o, "out")
            if rows2 != rows:  # one of them is one row: cut it up
                rows, cols = t.shape
                ld = cols if rows2 != 1 else ld
                ld_out = cols if rows2 == 1 else ld_out
        table.extend((p, q, rows, cols, ld, ld_out, _TYPES[t.dtype]))
    return table, len(tensors), device


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
    ``out`` (a tensor for each, in memory of its own); returns their norm
    before it (float32, one element)."""
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
