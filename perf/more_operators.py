"""Workloads of scoring and training with log probabilities, and of clipping gradients.

x (tokens x width) holds the last hidden states of a language model, w (vocab x width) the
rows of its output matrix, both 16-bit; the logits are z = x w^T / tau.

  score  for each token, given the id y_t that came next:
           lse_t = log sum_v exp z[t, v],   logp_t = z[t, y_t] - lse_t,
           entropy_t = -sum_v p log p with p = exp(z[t, :] - lse_t),
         and, asked for, the ids of the `top` largest logits with their log probabilities,
         largest first, equal logits by the lower id.  Rank is by the logits of the operands as
         they are, not as a sum in 32 bits rounds them.  A token with an id outside [0, vocab)
         is not scored: zeros, and -1 for its top ids.
  step   score without top, then its backward pass: from the gradients a_t of logp_t and
         b_t of entropy_t
           G[t, v] = (a_t ([v = y_t] - p) - b_t p (log p + entropy_t)) / tau,
           dx = G w, dw = G^T x, in the operands' type.
  clip   the global norm of a model's gradients, n = sqrt(sum of the squares of all their
         elements), and the gradients times min(1, max_norm / n), in their own type, written to
         buffers of their own.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _score(name, step, dtype, tokens, vocab, width, pad=0, ignored=0.0, top=0, tau=1.0):
    case = {"op": "step" if step else "score", "dtype": dtype, "tokens": tokens, "vocab": vocab, "width": width,
            "pad": pad, "ignored": ignored, "top": top, "tau": tau}
    return dict(case, name=name) if name else case


def _clip(name, layout, dtype, layers, width, vocab, pad=0, norm=3.0, salt=0):
    case = {"op": "clip", "layout": layout, "dtype": dtype, "layers": layers, "width": width, "vocab": vocab,
            "pad": pad, "norm": norm, "salt": salt}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token generated, with its five likeliest alternatives: latency
        _score("score_one", False, "bf16", 1, 32000, 768, top=5),
        # a batch of requests decoded, one token each, 20 alternatives: bound by the weights' bytes
        _score("score_decode", False, "bf16", 64, 128000, 4096, top=20, tau=0.7),
        # a prompt's own log probabilities with alternatives; odd vocabulary, padded rows
        _score("score_prompt", False, "f16", 2045, 50021, 1000, pad=24, ignored=0.25, top=5),
        # log probabilities and entropies of sampled answers under the old policy
        _score("score_rollouts", False, "bf16", 8192, 65536, 1024),
        # a teacher's best logits, written down for a student
        _score("score_teacher", False, "bf16", 1024, 100000, 2048, top=64),
        # a few tokens learnt from (online tuning): bound by the weights' bytes
        _score("step_few", True, "bf16", 16, 100000, 2048),
        # a policy-gradient step of a small transformer
        _score("step_small", True, "bf16", 8192, 32000, 768),
        # the same of answers behind long prompts, at the sampling temperature; a scaled loss
        _score("step_prompts", True, "f16", 6000, 65537, 2048, ignored=0.7, tau=0.7),
        # a step of a wide model with a large vocabulary: the largest
        _score("step_wide", True, "bf16", 4096, 128000, 4096),
        # gradients of one layer's adapters: a few small tensors, latency
        _clip("clip_small", "few", "bf16", 1, 768, 1000),
        # odd sizes, padded rows, several types, most of them tiny; the norm is within bounds
        _clip("clip_odd", "odd", "mixed", 150, 521, 9973, pad=3, norm=0.7),
        # every gradient of a wide model of a few layers
        _clip("clip_model", "model", "bf16", 4, 4096, 128000),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["score", "score", "step", "clip"])
    if op == "clip":
        layout = rng.choice(["few", "odd", "model"])
        dtype = rng.choice(["bf16", "f16", "f32", "mixed"])
        norm = rng.choice([0.7, 3.0, 40.0])
        if layout == "model":
            return _clip(None, layout, dtype, rng.randint(1, 4), spread(64, 2048) // 8 * 8, spread(1000, 131072),
                         0, norm, rng.randrange(1 << 20))
        return _clip(None, layout, dtype, spread(1, 400), spread(8, 2048), spread(1000, 131072),
                     rng.choice([0, 0, 8, 3]), norm, rng.randrange(1 << 20))
    step = op == "step"
    tokens, vocab, width = spread(1, 8192), spread(1000, 131072), spread(64, 4096)
    if rng.random() < 0.7:
        width = max(64, width // 8 * 8)  # most models' widths
    pad = rng.choice([0, 0, 8, 3])
    most = 4096 * 128000 * 4096 * 0.99
    tokens = max(1, min(tokens, int(most / (vocab * width)), 4096 * 128000 // vocab))
    top = 0 if step else rng.choice([0, 1, 5, 20, spread(1, 128)])
    return _score(None, step, rng.choice(["bf16", "f16"]), tokens, vocab, width, pad,
                  rng.choice([0.0, 0.1, 0.5]), top, rng.choice([1.0, 1.0, 0.7, 1.5]))


def _shapes(case):
    """The tensors of a clip case: (rows, columns, elements behind each row, type)."""
    rng = random.Random(case["salt"])
    D, V = case["width"], case["vocab"]

    def kind():
        return case["dtype"] if case["dtype"] != "mixed" else rng.choice(["bf16", "f16", "f32", "f32"])

    out = []
    if case["layout"] == "model":  # norms in 32 bits beside products' weights
        out.append((V, D, 0, kind()))
        for _ in range(case["layers"]):
            out += [(D, D, 0, kind()) for _ in range(4)]
            out += [(4 * D, D, 0, kind()), (D, 4 * D, 0, kind())]
            out += [(1, D, 0, "f32"), (1, D, 0, "f32")]
    elif case["layout"] == "few":  # adapters: down and up projections of rank 16, and their scales
        for _ in range(case["layers"]):
            out += [(16, D, case["pad"], kind()), (D, 16, 0, kind()), (1, 1, 0, "f32")]
    else:  # sizes of every order, rows off any boundary
        for _ in range(case["layers"]):
            rows = 1 if rng.random() < 0.5 else int(math.exp(rng.uniform(0, math.log(D))))
            cols = int(math.exp(rng.uniform(0, math.log(D))))
            out.append((rows, cols, case["pad"] if rows > 1 else 0, kind()))
        out.append((V, min(D, 64), case["pad"], kind()))
    return out


def _ignored(case):
    return int(case["tokens"] * case["ignored"])


def _rows(values, width, pad, dtype):
    """values as a matrix of dtype whose rows are width + pad apart."""
    store = torch.zeros(values.shape[0], width + pad, dtype=dtype, device=values.device)
    store[:, :width] = values
    return store[:, :width]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = torch.device("cuda")
    if case["op"] == "clip":
        shapes = _shapes(case)
        total = sum(r * c for r, c, _, _ in shapes)
        # elements of one size over all tensors, but for a factor of each tensor's own; 16-bit
        # floats of 5 exponent bits come from a scaled loss, and so does their bound
        scale = 1024.0 if any(t == "f16" for *_, t in shapes) else 1.0
        size = case["norm"] * scale / math.sqrt(total)
        # clipped, they go one behind the other into a buffer for each type, as an optimizer keeps them
        flat = {t: torch.zeros(sum(r * c for r, c, _, k in shapes if k == t), dtype=DTYPES[t], device=dev)
                for t in sorted({k for *_, k in shapes})}
        grads, out, at = [], [], dict.fromkeys(flat, 0)
        for r, c, pad, t in shapes:
            own_size = torch.rand(1, 1, generator=gen, device=dev) + 0.5
            grads.append(_rows(torch.randn(r, c, generator=gen, device=dev) * (size * own_size), c, pad, DTYPES[t]))
            out.append(flat[t][at[t]:at[t] + r * c].view(r, c))
            at[t] += r * c
        return {"case": case, "grads": grads, "out": out, "flat": flat, "max_norm": scale}
    dtype = DTYPES[case["dtype"]]
    T, V, D = case["tokens"], case["vocab"], case["width"]
    # weights of which random hidden states (of unit variance, as after a norm) make logits
    # of deviation 2; each token's state leans towards its own next token
    w = _rows(torch.randn(V, D, generator=gen, device=dev) * (2.0 / math.sqrt(D)), D, case["pad"], dtype)
    # frequent tokens come first: ids spread over the vocabulary's logarithm
    ids = (torch.exp(torch.rand(T, generator=gen, device=dev, dtype=torch.float64) * math.log(V)) - 1).long().clamp_(0, V - 1)
    lean = torch.rand(T, 1, generator=gen, device=dev) * 4.0
    x = _rows(torch.randn(T, D, generator=gen, device=dev) + lean * w[ids].float(), D, case["pad"], dtype)
    # the tokens that are not scored: whole runs of them, as prompts before answers
    n = _ignored(case)
    if n:
        runs = max(1, min(T // 700, n))
        at = torch.arange(T, device=dev)
        run = at * runs // T
        start = torch.div(run * T + runs - 1, runs, rounding_mode="floor")
        share = torch.div((run + 1) * n, runs, rounding_mode="floor") - torch.div(run * n, runs, rounding_mode="floor")
        ids = torch.where(at - start < share, -100, ids)
    state = {"case": case, "x": x, "w": w, "ids": ids}
    if case["op"] == "step":
        # a mean over the scored tokens of -advantage logp - 0.01 entropy
        scale = (1024.0 if case["dtype"] == "f16" else 1.0) / max(1, T - n)
        state["grad_logp"] = torch.randn(T, generator=gen, device=dev) * -scale
        state["grad_entropy"] = torch.full((T,), -0.01 * scale, device=dev)
    return state


def _plain_clip(state):
    total = 0.0
    for g in state["grads"]:
        total = total + (g.double() ** 2).sum()
    norm = torch.sqrt(total)
    factor = torch.clamp(state["max_norm"] / norm, max=1.0).float()
    for g, to in zip(state["grads"], state["out"]):
        to.copy_(g.float() * factor)
    return {"norm": norm.float().reshape(1), **state["flat"]}


def _plain_top(state, z, scored, lse):
    """The `top` largest logits of each row: found among the 32-bit ones with some to spare,
    ranked by the same logits in 64 bits."""
    case = state["case"]
    T, V, D, k = case["tokens"], case["vocab"], case["width"], case["top"]
    ids = z.topk(min(V, k + 8), dim=1).indices.sort(1).values
    exactly = torch.empty(ids.shape, dtype=torch.float64, device=z.device)
    piece = max(1, (1 << 27) // (ids.shape[1] * D))
    for t in range(0, T, piece):
        rows = state["w"][ids[t:t + piece]].double()
        exactly[t:t + piece] = (rows @ state["x"][t:t + piece].double()[:, :, None])[:, :, 0]
    best, order = exactly.sort(dim=1, descending=True, stable=True)
    logp = (best[:, :k] / case["tau"] - lse.double()).float()
    return torch.where(scored, logp, 0.0), torch.where(scored, ids.gather(1, order[:, :k]), -1)


def _plain(state):
    case = state["case"]
    if case["op"] == "clip":
        return _plain_clip(state)
    V, tau, dtype = case["vocab"], case["tau"], state["x"].dtype
    ids = state["ids"][:, None]
    scored = (ids >= 0) & (ids < V)
    ids = ids.clamp(0, V - 1)
    x = torch.where(scored, state["x"].float(), 0.0)
    w = state["w"].float()
    z = x @ w.t()
    if tau != 1.0:
        z /= tau
    peak = z.amax(1, keepdim=True)
    at = z.gather(1, ids)
    lse = peak + torch.log(torch.exp(z - peak).sum(1, keepdim=True))
    out = {"logp": torch.where(scored, at - lse, 0.0)[:, 0], "lse": torch.where(scored, lse, 0.0)[:, 0]}
    if case["top"]:
        out["top_logp"], out["top_ids"] = _plain_top(state, z, scored, lse)
    z -= lse
    p = torch.exp(z)
    entropy = -(p * z).sum(1, keepdim=True)
    out["entropy"] = torch.where(scored, entropy, 0.0)[:, 0]
    if case["op"] == "score":
        return out
    a = torch.where(scored, state["grad_logp"][:, None] / tau, 0.0)
    b = torch.where(scored, state["grad_entropy"][:, None] / tau, 0.0)
    z += entropy
    z *= -b
    z -= a
    z *= p
    z.scatter_add_(1, ids, a)
    out["dx"], out["dw"] = (z @ w).to(dtype), (z.t() @ x).to(dtype)
    return out


def run(state):
    if not own:
        return _plain(state)
    case = state["case"]
    if case["op"] == "clip":
        from dense_fp32_matrix_02_gb300 import grads as C
        norm = C.clip_(state["grads"], state["max_norm"], out=state["out"])
        return {"norm": norm, **state["flat"]}
    from dense_fp32_matrix_02_gb300 import loss as L
    x, w, ids, tau = state["x"], state["w"], state["ids"], case["tau"]
    step = case["op"] == "step"
    s = L.log_probs(x, w, ids, top=case["top"], temperature=tau, keep=step)
    out = {"logp": s.logp, "lse": s.lse, "entropy": s.entropy}
    if case["top"]:
        out["top_logp"], out["top_ids"] = s.top_logp, s.top_ids
    if step:
        out["dx"], out["dw"] = L.log_probs_grad(x, w, ids, s, state["grad_logp"], state["grad_entropy"],
                                                temperature=tau)
    return out


def work(case):
    if case["op"] == "clip":
        shapes = _shapes(case)
        return {"bytes": 4 + 2 * sum(r * c * (4 if t == "f32" else 2) for r, c, _, t in shapes),
                "flops": 3 * sum(r * c for r, c, _, _ in shapes)}
    T, V, D = case["tokens"], case["vocab"], case["width"]
    scored = T - _ignored(case)
    # x of the tokens that count, w, ids, the three numbers of a token and its alternatives
    nbytes = 2 * scored * D + 2 * V * D + T * (8 + 12 + 12 * case["top"])
    flops = 2 * scored * V * D
    if case["op"] == "step":
        nbytes += 2 * T * D + 2 * V * D + 8 * T
        flops *= 3
    return {"bytes": nbytes, "flops": flops}


def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    state = prepare(case, seed)
    if case["op"] == "clip":
        parts = [torch.linalg.vector_norm(g.double()) for g in state["grads"]]
        norm = torch.linalg.vector_norm(torch.stack(parts))
        over = norm > state["max_norm"]
        out = {"norm": norm.reshape(1)}
        for t in state["flat"]:
            every = torch.cat([g.reshape(-1) for g in state["grads"] if g.dtype == DTYPES[t]]).double()
            out[t] = torch.where(over, every * state["max_norm"] / norm, every)
        return out
    T, V, D, k, tau = case["tokens"], case["vocab"], case["width"], case["top"], case["tau"]
    every = state["ids"]
    rows = ((every >= 0) & (every < V)).nonzero()[:, 0]
    n, ids = rows.numel(), every[rows]
    x = state["x"][rows].double()
    dev = x.device
    piece = max(1, min(V, (1 << 27) // max(1, n)))
    lse = torch.full((n,), -math.inf, dtype=torch.float64, device=dev)
    best = torch.empty(n, 0, dtype=torch.float64, device=dev)
    names = torch.empty(n, 0, dtype=torch.int64, device=dev)
    for v in range(0, V if n else 0, piece):
        z = x @ state["w"][v:v + piece].double().t() / tau
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        if k:  # a stable sort keeps equal logits in the order of their ids
            few, order = z.sort(dim=1, descending=True, stable=True) if z.shape[1] <= k else z.topk(min(z.shape[1], k + 8), 1)
            order, by = order.sort(1)
            best = torch.cat([best, few.gather(1, by)], 1)
            names = torch.cat([names, order + v], 1)
            best, by = best.sort(dim=1, descending=True, stable=True)
            best, names = best[:, :k], names.gather(1, by[:, :k])
    entropy = torch.zeros(n, dtype=torch.float64, device=dev)
    for v in range(0, V if n else 0, piece):
        log_p = x @ state["w"][v:v + piece].double().t() / tau - lse[:, None]
        entropy -= (log_p.exp() * log_p).sum(1)
    logp = (x * state["w"][ids].double()).sum(1) / tau - lse

    def whole(values, fill=0):
        return torch.full((T, *values.shape[1:]), fill, dtype=values.dtype, device=dev).index_copy(0, rows, values)

    out = {"logp": whole(logp), "lse": whole(lse), "entropy": whole(entropy)}
    if k:
        out["top_logp"], out["top_ids"] = whole(best - lse[:, None]), whole(names, -1)
    if case["op"] == "score":
        return out
    a, b = state["grad_logp"][rows].double() / tau, state["grad_entropy"][rows].double() / tau
    dx = torch.zeros(n, D, dtype=torch.float64, device=dev)
    dw = torch.zeros(V, D, dtype=torch.float64, device=dev)
    for v in range(0, V if n else 0, piece):
        wv = state["w"][v:v + piece].double()
        log_p = x @ wv.t() / tau - lse[:, None]
        G = -log_p.exp() * (a[:, None] + b[:, None] * (log_p + entropy[:, None]))
        here = ((ids >= v) & (ids < v + piece)).nonzero()[:, 0]
        G[here, ids[here] - v] += a[here]
        dx += G @ wv
        dw[v:v + piece] = G.t() @ x
    out["dx"], out["dw"] = whole(dx), dw
    return out
