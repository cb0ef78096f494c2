"""The vocabulary losses in float64, from their definitions, with a bound on
what a kernel may differ by, element by element.

The bound follows the kernels' arithmetic, not their results.  With
u = 2^-8 (bfloat16) or 2^-11 (binary16), the rounding to the operands' type:
  * logits: the library's own bound for a product,
    d_t = max_v 1e-5·√D·Σ_k |x||w| / τ;
  * lse: d_t, plus 2e-5 for the exponentials (an argument of up to about 100
    rounds to 2^-17, each sum has at most a few hundred terms in a row), plus
    1e-6·|lse| for the logarithm and its argument;
  * loss: τ²·(d_t + lse's + 1e-6·(|log q| + |z/τ|) + 2e-5);
  * G: one rounding, u·|G|, and p's own error, |g|·τ·p·(d_t + lse's + 2e-5),
    plus binary16's smallest step under the scale that brings the largest
    |g·τ| to at least 2^13;
  * dX, dW: G's error times |W| or |X|, a product's sum,
    1e-5·√terms·Σ |G||W|, and one rounding of the result.
"""

from __future__ import annotations

import math

import torch


def cross_entropy_targets(targets, V):
    """(ids, log q) of a target vector; log q = -inf: no entry."""
    ids = targets[:, None]
    lq = torch.zeros(ids.shape, dtype=torch.float64, device=ids.device)
    return ids, lq.masked_fill((ids < 0) | (ids >= V), -math.inf)


def distill_targets(logits, ids, tau, V):
    u = logits.double() / tau
    u = u.masked_fill((ids < 0) | (ids >= V), -math.inf)
    return ids, u - torch.logsumexp(u, 1, keepdim=True).clamp_min(-1e300)


def loss_and_grads(x, w, ids, log_q, tau, g=None):
    """{"loss", "lse", "dx", "dw"} in float64 and {"..._tol"}; g (a vector)
    asks for the gradients."""
    T, D = x.shape
    V = w.shape[0]
    learnt = (log_q > -math.inf).any(1)
    u = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -11
    step = 0.0 if x.dtype == torch.bfloat16 else 2.0 ** -25
    X = torch.where(learnt[:, None], x.double(), 0.0)
    W = w.double()
    z = X @ W.t() / tau
    d = (1e-5 * math.sqrt(D) * (X.abs() @ W.abs().t()) / tau).amax(1)
    lse = torch.logsumexp(z, 1)
    q = log_q.exp()
    safe = ids.clamp(0, V - 1)
    at = z.gather(1, safe)
    counts = q > 0
    terms = torch.where(counts, q * (log_q - (at - lse[:, None])), 0.0)
    lse_tol = d + 2e-5 + 1e-6 * lse.abs()
    size = torch.where(counts, log_q.abs() + at.abs(), 0.0).amax(1)
    zero = torch.zeros(T, dtype=torch.float64, device=x.device)

    def rows(v):
        return torch.where(learnt, v, zero)

    out = {"loss": rows(tau * tau * terms.sum(1)), "lse": rows(lse),
           "lse_tol": rows(lse_tol),
           "loss_tol": rows(tau * tau * (d + lse_tol + 1e-6 * size + 2e-5))}
    if g is None:
        return out
    p = (z - lse[:, None]).exp()
    Q = torch.zeros_like(p).scatter_add_(
        1, safe, torch.where(counts, q, 0.0))
    gt = rows(g.double() * tau)[:, None]
    G = gt * (p - Q)
    dG = u * G.abs() + gt.abs() * p * (d + lse_tol + 2e-5)[:, None]
    if step:
        dG = dG + learnt[:, None] * float(gt.abs().max()) * step / 2.0 ** 13
    out["dx"], out["dw"] = G @ W, G.t() @ X
    for name, other, left, dleft, terms_n in (
            ("dx", W, G, dG, V), ("dw", X, G.t(), dG.t(), max(T, 1))):
        out[name + "_tol"] = (
            dleft @ other.abs()
            + 1e-5 * math.sqrt(terms_n) * (left.abs() @ other.abs())
            + u * out[name].abs() + step)
    return out
