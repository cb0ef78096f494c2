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
"""

from __future__ import annotations

from . import gemm as _g

__all__ = ["cross_entropy", "cross_entropy_grad", "distill", "distill_grad",
           "workspace_size"]


def workspace_size(tokens, vocab, width, top=1, grad=False,
                   aligned=True) -> int:
    """Workspace bytes of the forward calls, or of the gradients with
    ``grad``.  ``aligned``: x and w start on 16-byte boundaries and their
    rows are multiples of 8 elements apart."""
    n = int(_g.lib().gemm_f32_vocab_workspace_size(
        int(tokens), int(vocab), int(width), int(top), int(bool(grad)),
        int(bool(aligned))))
    if n < 0:
        _g._check(-n, "gemm_f32_vocab_workspace_size")
    return n


def _operands(x, w):
    """(type, T, V, D, x pointer, ldx, w pointer, ldw, aligned)."""
    import torch
    dt = (torch.bfloat16, torch.float16)
    T, D, xp, ldx = _g._matrix_args(x, "x", dt)
    V, D2, wp, ldw = _g._matrix_args(w, "w", dt)
    if x.dtype != w.dtype:
        raise TypeError("x and w must have the same 16-bit dtype")
    if D != D2:
        raise ValueError(f"widths differ: x {tuple(x.shape)}, w "
                         f"{tuple(w.shape)}")
    if w.device != x.device:
        raise ValueError("w must live on x's device")
    aligned = xp % 16 == 0 and wp % 16 == 0 and ldx % 8 == 0 and ldw % 8 == 0
    return _g._mixed_type(x.dtype), T, V, D, xp, ldx, wp, ldw, aligned


def _vector(t, name, n, dtype, like, expand=False):
    """(pointer, stride) of a vector of n elements on like's device."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {str(dtype).replace('torch.', '')} "
                        "torch tensor")
    if t.device != like.device:
        raise ValueError(f"{name} must live on x's device")
    if tuple(t.shape) != (n,):
        raise ValueError(f"{name} must have shape {(n,)}")
    stride = t.stride(0) if n > 1 else 1
    if stride != 1 and not (expand and stride >= 0):
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() if n else 0, stride


def _teacher(top_logits, top_ids, T, like):
    """(top, logits pointer, ldt, ids pointer, ldi)."""
    import torch
    out = []
    for t, name, dtype in ((top_logits, "top_logits", torch.float32),
                           (top_ids, "top_ids", torch.int64)):
        rows, cols, p, ld = _g._matrix_args(t, name, (dtype,))
        if t.device != like.device:
            raise ValueError(f"{name} must live on x's device")
        if rows != T:
            raise ValueError(f"{name} must have one row per token")
        out.append((cols, p, ld))
    if out[0][0] != out[1][0]:
        raise ValueError("top_logits and top_ids have different widths")
    return (out[0][0], out[0][1] or None, out[0][2], out[1][1] or None,
            out[1][2])


def _new(shape, dtype, like, stream):
    """An output allocated here, known to the allocator to be in use on
    `stream` when that is not the current one."""
    import torch
    out = torch.empty(shape, dtype=dtype, device=like.device)
    if stream is not None:
        _g._in_use_on(out, stream)
    return out


def _given(t, shape, dtype, like, name, stream):
    """(tensor, pointer, leading dimension) of an output."""
    if t is None:
        t = _new(shape, dtype, like, stream)
    rows, cols, p, ld = _g._matrix_args(t, name, (dtype,))
    if (rows, cols) != tuple(shape) or t.device != like.device:
        raise ValueError(f"{name} must have shape {tuple(shape)} on x's "
                         "device")
    return t, p or None, ld


def _workspace(workspace, need, like, stream):
    if workspace is None:
        workspace = _g._scratch(need, like.device, stream)
    elif workspace.device != like.device:
        raise ValueError("workspace must live on x's device")
    n = workspace.numel() * workspace.element_size()
    return workspace, workspace.data_ptr() if n else None, n


def _forward(name, x, w, target_args, make_targets, top, workspace, stream):
    import torch
    ty, T, V, D, xp, ldx, wp, ldw, aligned = _operands(x, w)
    args = make_targets(T)
    with torch.cuda.device(x.device):
        if top is None:
            top = args[0]
        ws, wsp, wsn = _workspace(
            workspace, 0 if workspace is not None else
            workspace_size(T, V, D, top, False, aligned), x, stream)
        loss = _new((T,), torch.float32, x, stream)
        lse = _new((T,), torch.float32, x, stream)
        st = getattr(_g.lib(), name)(
            ty, T, V, D, xp or None, ldx, wp or None, ldw, *args,
            *target_args, loss.data_ptr() or None, lse.data_ptr() or None,
            wsp, wsn, _g._handle(stream, x.device) or None)
    _g._check(st, name)
    return loss, lse


def _backward(name, x, w, target_args, make_targets, top, lse, grad_loss, dx,
              dw, workspace, stream):
    import torch
    ty, T, V, D, xp, ldx, wp, ldw, aligned = _operands(x, w)
    args = make_targets(T)
    lp, _ = _vector(lse, "lse", T, torch.float32, x)
    gp, gs = _vector(grad_loss, "grad_loss", T, torch.float32, x, expand=True)
    with torch.cuda.device(x.device):
        if top is None:
            top = args[0]
        ws, wsp, wsn = _workspace(
            workspace, 0 if workspace is not None else
            workspace_size(T, V, D, top, True, aligned), x, stream)
        dx, dxp, lddx = _given(dx, (T, D), x.dtype, x, "dx", stream)
        dw, dwp, lddw = _given(dw, (V, D), x.dtype, x, "dw", stream)
        st = getattr(_g.lib(), name)(
            ty, T, V, D, xp or None, ldx, wp or None, ldw, *args,
            *target_args, lp or None, gp or None, gs, dxp, lddx, dwp, lddw,
            wsp, wsn, _g._handle(stream, x.device) or None)
    _g._check(st, name)
    return dx, dw


def cross_entropy(x, w, targets, workspace=None, stream=None):
    """(loss, lse), float32, one value per token: lse = log Σ exp(logits),
    loss = lse − logits[targets].  targets: int64; a target outside
    [0, vocab) marks a token that is not learnt from (loss and lse 0)."""
    import torch

    def targets_of(T):
        return (_vector(targets, "targets", T, torch.int64, x)[0] or None,)

    return _forward("gemm_f32_vocab_ce", x, w, (), targets_of, 1, workspace,
                    stream)


def cross_entropy_grad(x, w, targets, lse, grad_loss, dx=None, dw=None,
                       workspace=None, stream=None):
    """(dx, dw) in x's dtype from the gradient of each token's loss
    (float32; an expanded scalar is taken as it is); lse as cross_entropy
    returned it."""
    import torch

    def targets_of(T):
        return (_vector(targets, "targets", T, torch.int64, x)[0] or None,)

    return _backward("gemm_f32_vocab_ce_grad", x, w, (), targets_of, 1, lse,
                     grad_loss, dx, dw, workspace, stream)


def distill(x, w, top_logits, top_ids, temperature=1.0, workspace=None,
            stream=None):
    """(loss, lse), float32, one value per token: τ² times the divergence
    of softmax(logits/τ) from softmax(top_logits/τ) over the teacher's
    entries (float32 logits and int64 ids, tokens × top; an id outside
    [0, vocab) or a logit of −inf: no entry)."""
    return _forward("gemm_f32_vocab_distill", x, w, (float(temperature),),
                    lambda T: _teacher(top_logits, top_ids, T, x), None,
                    workspace, stream)


def distill_grad(x, w, top_logits, top_ids, lse, grad_loss, temperature=1.0,
                 dx=None, dw=None, workspace=None, stream=None):
    """(dx, dw) in x's dtype from the gradient of each token's loss; lse as
    distill returned it."""
    return _backward("gemm_f32_vocab_distill_grad", x, w,
                     (float(temperature),),
                     lambda T: _teacher(top_logits, top_ids, T, x), None, lse,
                     grad_loss, dx, dw, workspace, stream)
