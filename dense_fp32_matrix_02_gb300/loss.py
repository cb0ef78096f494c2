"""Vocabulary losses of torch CUDA tensors (argument marshalling only).

The last product of a language model, logits = x·wᵀ with x (tokens × width)
the hidden states and w (vocab × width) the output matrix, together with its
loss: softmax cross entropy, or distillation from a teacher's top logits.
The logits are never stored; ``include/gemm_f32.h`` (gemm_f32_vocab_*) gives
the formulas.  Like every call of the binding these are asynchronous on
``stream`` (None: the current one), raise ``GemmError`` for a status other
than 0, and take an optional ``workspace`` (a CUDA tensor of at least
``workspace_size`` bytes; allocated here when None).

    loss, lse = cross_entropy(x, w, targets)             # per token, fp32
    dx, dw = cross_entropy_grad(x, w, targets, lse, grad_loss)

Autograd records none of this: results of inputs that require gradients have
no graph, and the gradients come from the _grad calls, which overwrite dx and
dw (in memory of their own).
"""

from __future__ import annotations

import contextlib
import functools

import torch

from . import gemm as _g

__all__ = ["cross_entropy", "cross_entropy_grad", "distill", "distill_grad",
           "workspace_size"]

_TYPES = {torch.bfloat16: _g.MIXED_BF16, torch.float16: _g.MIXED_F16}
_FLOAT, _INT = (torch.float32,), (torch.int64,)
_STAY = contextlib.nullcontext()


@functools.lru_cache(maxsize=256)
def _size(tokens, vocab, width, top, grad, aligned):
    n = int(_g.lib().gemm_f32_vocab_workspace_size(tokens, vocab, width, top,
                                                   grad, aligned))
    if n < 0:
        _g._check(-n, "gemm_f32_vocab_workspace_size")
    return n


def workspace_size(tokens, vocab, width, top=1, grad=False,
                   aligned=True) -> int:
    """Workspace bytes of the forward calls, or of the gradients with
    ``grad``.  ``aligned``: x and w start on 16-byte boundaries and their
    rows are multiples of 8 elements apart."""
    return _size(int(tokens), int(vocab), int(width), int(top),
                 int(bool(grad)), int(bool(aligned)))


def _matrix(t, name, dtypes, like=None):
    """(rows, columns, pointer or None, leading dimension) of a row-major
    CUDA matrix (on like's device)."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        names = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise TypeError(f"{name} must be a {names} torch tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if like is not None and t.device != like:
        raise ValueError(f"{name} must live on x's device")
    rows, cols = t.shape
    step, one = t.stride()
    if cols > 1 and one != 1 and rows:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    # a single row has no meaningful row stride unless it spans the width
    return (rows, cols, t.data_ptr() or None,
            step if rows > 1 or step > cols else max(cols, 1))


def _vector(t, name, n, dtype, device, expand=False):
    """(pointer or None, stride) of a vector of n elements."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {str(dtype).replace('torch.', '')} "
                        "torch tensor")
    if t.device != device:
        raise ValueError(f"{name} must live on x's device")
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape {(n,)}")
    stride = t.stride(0) if n > 1 else 1
    if stride != 1 and not (expand and stride >= 0):
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None, stride


def _teacher(top_logits, top_ids, T, device):
    """(entries a token, logits pointer, ldt, ids pointer, ldi)."""
    rows, top, up, ldt = _matrix(top_logits, "top_logits", _FLOAT, device)
    rows2, top2, ip, ldi = _matrix(top_ids, "top_ids", _INT, device)
    if rows != T or rows2 != T:
        raise ValueError("top_logits and top_ids must have one row per token")
    if top != top2:
        raise ValueError("top_logits and top_ids have different widths")
    return top, up, ldt, ip, ldi


def _operands(x, w):
    """(type, T, V, D, x pointer, ldx, w pointer, ldw) and whether both have
    the alignment that needs no copies."""
    T, D, xp, ldx = _matrix(x, "x", _TYPES)
    V, D2, wp, ldw = _matrix(w, "w", _TYPES, x.device)
    if x.dtype != w.dtype:
        raise TypeError("x and w must have the same 16-bit dtype")
    if D != D2:
        raise ValueError(f"widths differ: x {tuple(x.shape)}, w "
                         f"{tuple(w.shape)}")
    aligned = ((xp or 0) | (wp or 0)) % 16 == 0 and (ldx | ldw) % 8 == 0
    return (_TYPES[x.dtype], T, V, D, xp, ldx, wp, ldw), int(aligned)


def _on(device):
    """The device made current, where it is not already."""
    return _STAY if torch.cuda.current_device() == device.index else \
        torch.cuda.device(device)


def _new(shape, dtype, device, stream):
    """A tensor allocated here, known to the allocator to be in use on
    `stream` when that is not the current one."""
    out = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        _g._in_use_on(out, stream)
    return out


def _out(t, shape, dtype, device, name, stream):
    """(tensor, pointer, leading dimension) of an output matrix."""
    if t is None:
        t = _new(shape, dtype, device, stream)
    rows, cols, p, ld = _matrix(t, name, (dtype,), device)
    if (rows, cols) != shape:
        raise ValueError(f"{name} must have shape {shape}")
    return t, p, ld


def _scratch(workspace, head, top, grad, aligned, device, stream):
    """(workspace, pointer, bytes), allocated when not given."""
    if workspace is None:
        n = _size(head[1], head[2], head[3], top, grad, aligned)
        workspace = _new(n, torch.uint8, device, stream)
    else:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError("workspace must be a torch tensor")
        if workspace.device != device:
            raise ValueError("workspace must live on x's device")
        if not workspace.is_contiguous():  # (an expanded one has fewer bytes)
            raise ValueError("workspace must be contiguous")
        n = workspace.numel() * workspace.element_size()
    return workspace, workspace.data_ptr() or None, n


def _stream(stream, device):
    """The stream's handle, or NULL (the current stream's without the object
    that torch.cuda.current_stream makes: 2 us of a call)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index) or None
    return (stream.cuda_stream if hasattr(stream, "cuda_stream") else
            int(stream)) or None


def _forward(name, x, w, head, aligned, top, target_args, workspace, stream):
    device, T = x.device, head[1]
    with _on(device):
        loss = _new(T, torch.float32, device, stream)
        lse = _new(T, torch.float32, device, stream)
        workspace, wp, n = _scratch(workspace, head, top, 0, aligned, device,
                                    stream)
        st = getattr(_g.lib(), name)(
            *head, *target_args, loss.data_ptr() or None,
            lse.data_ptr() or None, wp, n, _stream(stream, device))
    if st:
        _g._check(st, name)
    return loss, lse


def _backward(name, x, w, head, aligned, top, target_args, lse, grad_loss, dx,
              dw, workspace, stream):
    device, (_, T, V, D) = x.device, head[:4]
    lp, _ = _vector(lse, "lse", T, torch.float32, device)
    gp, gs = _vector(grad_loss, "grad_loss", T, torch.float32, device,
                     expand=True)
    with _on(device):
        dx, dxp, lddx = _out(dx, (T, D), x.dtype, device, "dx", stream)
        dw, dwp, lddw = _out(dw, (V, D), x.dtype, device, "dw", stream)
        workspace, wp, n = _scratch(workspace, head, top, 1, aligned, device,
                                    stream)
        st = getattr(_g.lib(), name)(
            *head, *target_args, lp, gp, gs, dxp, lddx, dwp, lddw, wp, n,
            _stream(stream, device))
    if st:
        _g._check(st, name)
    return dx, dw


def cross_entropy(x, w, targets, workspace=None, stream=None):
    """(loss, lse), float32, one value per token: lse = log Σ exp(logits),
    loss = lse − logits[targets].  targets: int64; a target outside
    [0, vocab) marks a token that is not learnt from (loss and lse 0)."""
    head, aligned = _operands(x, w)
    y, _ = _vector(targets, "targets", head[1], torch.int64, x.device)
    return _forward("gemm_f32_vocab_ce", x, w, head, aligned, 1, (y,),
                    workspace, stream)


def cross_entropy_grad(x, w, targets, lse, grad_loss, dx=None, dw=None,
                       workspace=None, stream=None):
    """(dx, dw) in x's dtype from the gradient of each token's loss
    (float32; an expanded scalar is taken as it is); lse as cross_entropy
    returned it."""
    head, aligned = _operands(x, w)
    y, _ = _vector(targets, "targets", head[1], torch.int64, x.device)
    return _backward("gemm_f32_vocab_ce_grad", x, w, head, aligned, 1, (y,),
                     lse, grad_loss, dx, dw, workspace, stream)


def distill(x, w, top_logits, top_ids, temperature=1.0, workspace=None,
            stream=None):
    """(loss, lse), float32, one value per token: τ² times the divergence
    of softmax(logits/τ) from softmax(top_logits/τ) over the teacher's
    entries (float32 logits and int64 ids, tokens × top; an id outside
    [0, vocab) or a logit of −inf: no entry)."""
    head, aligned = _operands(x, w)
    teacher = _teacher(top_logits, top_ids, head[1], x.device)
    return _forward("gemm_f32_vocab_distill", x, w, head, aligned,
                    teacher[0], (*teacher, float(temperature)), workspace,
                    stream)


def distill_grad(x, w, top_logits, top_ids, lse, grad_loss, temperature=1.0,
                 dx=None, dw=None, workspace=None, stream=None):
    """(dx, dw) in x's dtype from the gradient of each token's loss; lse as
    distill returned it."""
    head, aligned = _operands(x, w)
    teacher = _teacher(top_logits, top_ids, head[1], x.device)
    return _backward("gemm_f32_vocab_distill_grad", x, w, head, aligned,
                     teacher[0], (*teacher, float(temperature)), lse,
                     grad_loss, dx, dw, workspace, stream)
