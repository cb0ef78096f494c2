"""Vocabulary losses and log probabilities of torch CUDA tensors (argument
marshalling only).

The last product of a language model, logits = x·wᵀ with x (tokens × width)
the hidden states and w (vocab × width) the output matrix, together with its
loss: softmax cross entropy, or distillation from a teacher's top logits; or
with the log probabilities of given words, their distribution's entropy and
the likeliest words.  The losses never store the logits;
``include/gemm_f32.h`` (gemm_f32_vocab_*) gives the formulas.  Like every call
of the binding these are asynchronous on ``stream`` (None: the current one), raise
``GemmError`` for a status other than 0, and take an optional ``workspace`` (a
CUDA tensor of at least ``workspace_size`` bytes; allocated here when None).

    loss, lse = cross_entropy(x, w, targets)             # per token, fp32
    dx, dw = cross_entropy_grad(x, w, targets, lse, grad_loss)

    s = log_probs(x, w, ids, top=5)        # s.logp, s.entropy, s.top_ids, …
    s = log_probs(x, w, ids, keep=True)    # with the logits, for the gradients
    dx, dw = log_probs_grad(x, w, ids, s, grad_logp, grad_entropy)

Autograd records none of this: results of inputs that require gradients have
no graph, and the gradients come from the _grad calls, which overwrite dx and
dw (in memory of their own).
"""

from __future__ import annotations

import contextlib
import functools
import typing

import torch

from . import gemm as _g

__all__ = ["cross_entropy", "cross_entropy_grad", "distill", "distill_grad",
           "LogProbs", "log_probs", "log_probs_grad", "score_workspace_size",
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


@functools.lru_cache(maxsize=256)
def _score_size(tokens, vocab, width, top, keep, grad, aligned):
    n = int(_g.lib().gemm_f32_vocab_score_workspace_size(
        tokens, vocab, width, top, keep, grad, aligned))
    if n < 0:
        _g._check(-n, "gemm_f32_vocab_score_workspace_size")
    return n


def score_workspace_size(tokens, vocab, width, top=0, keep=False, grad=False,
                         aligned=True) -> int:
    """Workspace bytes of log_probs, or of log_probs_grad with ``grad``;
    ``aligned`` as for workspace_size."""
    return _score_size(int(tokens), int(vocab), int(width), int(top),
                       int(bool(keep)), int(bool(grad)), int(bool(aligned)))


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


def _bytes(t, name, device, whose="x's"):
    """(tensor, pointer, bytes) of a buffer."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} must live on {whose} device")
    if not t.is_contiguous():  # (an expanded one has fewer bytes)
        raise ValueError(f"{name} must be contiguous")
    return t, t.data_ptr() or None, t.numel() * t.element_size()


def _scratch(workspace, head, top, grad, aligned, device, stream):
    """(workspace, pointer, bytes), allocated when not given."""
    if workspace is None:
        n = _size(head[1], head[2], head[3], top, grad, aligned)
        workspace = _new(n, torch.uint8, device, stream)
    return _bytes(workspace, "workspace", device)


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


class LogProbs(typing.NamedTuple):
    """What log_probs returns: float32 values per token, top_logp and
    top_ids (int64) tokens × top or None, and the kept logits or None."""
    logp: torch.Tensor
    lse: torch.Tensor
    entropy: torch.Tensor
    top_logp: torch.Tensor | None
    top_ids: torch.Tensor | None
    kept: torch.Tensor | None


def log_probs(x, w, ids, top=0, temperature=1.0, keep=False, workspace=None,
              stream=None):
    """LogProbs of one given word per token (ids: int64) under
    softmax(logits/temperature): its log probability, lse = log Σ
    exp(logits/temperature), the distribution's entropy and, with ``top``, the
    likeliest words, largest first, equal logits by the lower id.  A token
    whose id is outside [0, vocab) is not scored (zeros; ids of -1).  ``keep``:
    the logits stay in memory (4 bytes each, 4 GB of 8192 tokens and 128000
    words) for log_probs_grad, and a copy of w if its rows do not start on
    16-byte boundaries."""
    head, aligned = _operands(x, w)
    device, T, V = x.device, head[1], head[2]
    y, _ = _vector(ids, "ids", T, torch.int64, device)
    top, keep = int(top), int(bool(keep))
    if top < 0:
        raise ValueError("top must not be negative")
    with _on(device):
        # (one allocation for the three: they are views of it)
        out = _new((3, T), torch.float32, device, stream)
        logp, lse, entropy = out.unbind()
        top_logp = top_ids = kept = None
        tp = ip = kp = None
        kn = 0
        if top:
            top_logp = _new((T, top), torch.float32, device, stream)
            top_ids = _new((T, top), torch.int64, device, stream)
            tp, ip = top_logp.data_ptr() or None, top_ids.data_ptr() or None
        if keep:
            kn = int(_g.lib().gemm_f32_vocab_score_kept_size(
                T, V, head[3], int((head[6] or 0) % 16 == 0
                                   and head[7] % 8 == 0)))
            if kn < 0:
                _g._check(-kn, "gemm_f32_vocab_score_kept_size")
            kept = _new(kn, torch.uint8, device, stream)
            kp = kept.data_ptr() or None
        if workspace is None:
            workspace = _new(_score_size(T, V, head[3], top, keep, 0, aligned),
                             torch.uint8, device, stream)
        workspace, wp, n = _bytes(workspace, "workspace", device)
        op = out.data_ptr()
        st = _g.lib().gemm_f32_vocab_score(
            *head, y, float(temperature), top, op or None,
            op + 4 * T or None, op + 8 * T or None, tp, ip, kp, kn, wp, n,
            _stream(stream, device))
    if st:
        _g._check(st, "gemm_f32_vocab_score")
    return LogProbs(logp, lse, entropy, top_logp, top_ids, kept)


def log_probs_grad(x, w, ids, scores, grad_logp, grad_entropy=None,
                   temperature=1.0, dx=None, dw=None, workspace=None,
                   stream=None):
    """(dx, dw) in x's dtype from the gradients of each token's logp and
    entropy (float32; an expanded scalar is taken as it is; None: 0).
    ``scores``: what log_probs returned for the same operands, ids and
    temperature with ``keep``; there is no form that makes the logits again, as
    the losses' gradients do.  A batch whose logits are too many is given in
    parts, whose dw (overwritten by each call) the caller adds up."""
    head, aligned = _operands(x, w)
    device, (_, T, V, D) = x.device, head[:4]
    y, _ = _vector(ids, "ids", T, torch.int64, device)
    if scores.kept is None:
        raise ValueError("the gradients need the logits: log_probs(keep=True)")
    lp, _ = _vector(scores.lse, "lse", T, torch.float32, device)
    hp, _ = _vector(scores.entropy, "entropy", T, torch.float32, device)
    _, kp, kn = _bytes(scores.kept, "kept", device)
    ap, a_step = _vector(grad_logp, "grad_logp", T, torch.float32, device,
                         expand=True)
    bp, b_step = None, 0
    if grad_entropy is not None:
        bp, b_step = _vector(grad_entropy, "grad_entropy", T, torch.float32,
                             device, expand=True)
    with _on(device):
        dx, dxp, lddx = _out(dx, (T, D), x.dtype, device, "dx", stream)
        dw, dwp, lddw = _out(dw, (V, D), x.dtype, device, "dw", stream)
        if workspace is None:
            workspace = _new(_score_size(T, V, D, 0, 1, 1, aligned),
                             torch.uint8, device, stream)
        workspace, wp, n = _bytes(workspace, "workspace", device)
        st = _g.lib().gemm_f32_vocab_score_grad(
            *head, y, float(temperature), lp, hp, kp, kn, ap, a_step, bp,
            b_step, dxp, lddx, dwp, lddw, wp, n, _stream(stream, device))
    if st:
        _g._check(st, "gemm_f32_vocab_score_grad")
    return dx, dw
