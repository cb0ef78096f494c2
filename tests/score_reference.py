"""Log probabilities, entropy, the likeliest words and their gradients in
float64, from the definitions, with a bound on what a kernel may differ by,
element by element.

The bound follows the kernels' arithmetic.  u, d_t (a logit's error) and lse's
are those of tests/vocab_reference.py; e = 2e-5 is what the exponentials and
the sums of a few hundred terms add to a logarithm.
  * logp: d + lse's + 1e-6·|z/τ| + e;
  * entropy: its derivative with respect to log p_v is −p_v·(log p_v + H), whose
    sizes add up to at most 2·H; so 2·H·(d + e), plus what the two terms whose
    difference it is (log S and E/S, each at most log V) round: 2e-6·log V + e;
  * top_logp: as logp, a logit and lse: d + lse's + 1e-6·|z/τ| + e;
  * G: one rounding, u·|G|; p's own error, a factor 1 ± (d + lse's + e); the
    error of log p + H in the second term; and binary16's smallest step under
    the scale that brings the largest (|a| + |b|·(0.4 + H))/τ to 2^14;
  * dX, dW: as for the losses.
"""

from __future__ import annotations

import math

import torch


def scores(x, w, ids, tau=1.0, top=0):
    """{"logp", "lse", "entropy", "top_logp", "top_ids"} and {"..._tol"}."""
    T, D = x.shape
    V = w.shape[0]
    scored = (ids >= 0) & (ids < V)
    X = torch.where(scored[:, None], x.double(), 0.0)
    W = w.double()
    z = X @ W.t() / tau
    d = (1e-5 * math.sqrt(D) * (X.abs() @ W.abs().t()) / tau).amax(1)
    lse = torch.logsumexp(z, 1)
    log_p = z - lse[:, None]
    p = log_p.exp()
    H = -torch.where(p > 0, p * log_p, 0.0).sum(1)
    at = z.gather(1, ids.clamp(0, V - 1)[:, None])[:, 0]
    e = 2e-5
    lse_tol = d + e + 1e-6 * lse.abs()
    zero = torch.zeros_like(lse)

    def rows(v):
        return torch.where(scored, v, zero)

    out = {"logp": rows(at - lse), "lse": rows(lse), "entropy": rows(H),
           "logp_tol": rows(d + lse_tol + 1e-6 * at.abs() + e),
           "lse_tol": rows(lse_tol),
           "entropy_tol": rows(2 * H * (d + e) + 2e-6 * math.log(V + 1) + e),
           "z": z, "log_p": log_p, "d": d, "scored": scored}
    if top:
        best, order = z.sort(dim=1, descending=True, stable=True)
        best, order = best[:, :top], order[:, :top]
        out["top_ids"] = torch.where(scored[:, None], order, -1)
        out["top_logp"] = torch.where(scored[:, None], best - lse[:, None], 0.0)
        out["top_logp_tol"] = torch.where(
            scored[:, None],
            (d + lse_tol + e)[:, None] + 1e-6 * best.abs(), 0.0)
    return out


def gradients(x, w, ids, a, b=None, tau=1.0):
    """{"dx", "dw"} and {"..._tol"} for the gradients a of logp and b of
    entropy."""
    s = scores(x, w, ids, tau)
    T, V = s["z"].shape
    scored, log_p, H = s["scored"], s["log_p"], s["entropy"]
    u = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -11
    step = 0.0 if x.dtype == torch.bfloat16 else 2.0 ** -25
    X = torch.where(scored[:, None], x.double(), 0.0)
    W = w.double()
    a = torch.where(scored, a.double(), 0.0)[:, None] / tau
    b = torch.zeros_like(a) if b is None else \
        torch.where(scored, b.double(), 0.0)[:, None] / tau
    p = log_p.exp()
    rest = torch.where(p > 0, log_p + H[:, None], 0.0)
    G = -p * (a + b * rest)
    rows = scored.nonzero()[:, 0]
    G[rows, ids[rows]] += a[rows, 0]
    wrong = (s["d"] + s["lse_tol"] + 2e-5)[:, None]
    dG = (u * G.abs() + p * (a.abs() + b.abs() * rest.abs()) * wrong
          + p * b.abs() * (wrong + s["entropy_tol"][:, None]))
    if step:
        most = (a.abs() + b.abs() * (0.4 + H[:, None])).max()
        dG = dG + scored[:, None] * float(most) * step / 2.0 ** 13
    out = {"dx": G @ W, "dw": G.t() @ X}
    for name, other, left, dleft, n in (
            ("dx", W, G, dG, V), ("dw", X, G.t(), dG.t(), max(T, 1))):
        out[name + "_tol"] = (
            dleft @ other.abs()
            + 1e-5 * math.sqrt(n) * (left.abs() @ other.abs())
            + u * out[name].abs() + step)
    return out
