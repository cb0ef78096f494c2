"""Workloads of the vocabulary losses: a language model's last product with its loss.

x (tokens x width) holds the last hidden states, w (vocab x width) the rows of
the output matrix, both 16-bit; the logits are z = x w^T.  Two losses of them,
each forward ("score") and forward plus backward ("step"):

  ce  softmax cross entropy: loss_t = lse_t - z[t, y_t], lse_t = log sum_v exp z[t, v].
      A target outside [0, vocab) marks a token that is not learnt from: its loss and
      lse are 0 and it adds nothing to any gradient, whatever its row of x holds.
  kd  distillation from a teacher's top logits u[t, j] at ids i[t, j], temperature tau:
      q[t, :] = softmax of u[t, :] / tau over the entries that count,
      loss_t = tau^2 sum_j q[t, j] (log q[t, j] - (z[t, i[t, j]] / tau - lse_t)),
      lse_t = log sum_v exp(z[t, v] / tau).  An entry with an id outside [0, vocab) or a
      logit of -inf does not count; a token without entries is as an ignored one.

Backward, from the gradients g_t of the tokens' losses:
  ce  G = g (softmax(z) - onehot(y)),  kd  G = g tau (softmax(z / tau) - q at the ids);
  dx = G w, dw = G^T x, in the operands' type.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _case(name, op, step, dtype, tokens, vocab, width, pad=0, ignored=0.0, top=1, tau=1.0):
    case = {"op": op, "step": step, "dtype": dtype, "tokens": tokens, "vocab": vocab, "width": width,
            "pad": pad, "ignored": ignored, "top": top, "tau": tau}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token scored while generating: latency
        _case("ce_score_one", "ce", False, "bf16", 1, 32000, 768),
        # one short document scored; an odd vocabulary, padded rows, the prompt masked
        _case("ce_score_document", "ce", False, "f16", 509, 50021, 1000, pad=24, ignored=0.25),
        # evaluation over a full batch of tokens
        _case("ce_score_batch", "ce", False, "bf16", 8192, 65536, 1024),
        # a handful of tokens learnt from (online tuning): bound by the weights' bytes
        _case("ce_step_few", "ce", True, "bf16", 16, 100000, 2048),
        # a training step of the small transformer whose layer this repository's benchmark multiplies
        _case("ce_step_small", "ce", True, "bf16", 8192, 32000, 768),
        # instruction tuning: most tokens are prompts and are ignored
        _case("ce_step_prompts", "ce", True, "f16", 6000, 65537, 2048, ignored=0.7),
        # a training step of a wide model with a large vocabulary: the largest
        _case("ce_step_wide", "ce", True, "bf16", 4096, 128000, 4096),
        # a few tokens compared with a teacher's
        _case("kd_score_few", "kd", False, "f16", 7, 32000, 768, top=8, tau=1.0),
        # held-out tokens compared with a teacher's
        _case("kd_score_batch", "kd", False, "bf16", 2048, 50021, 768, ignored=0.1, top=32, tau=1.5),
        # odd sizes throughout: rows that start on any address, missing entries
        _case("kd_step_odd", "kd", True, "f16", 777, 9973, 521, ignored=0.2, top=5, tau=2.0),
        # a distillation step with a large vocabulary
        _case("kd_step_wide", "kd", True, "bf16", 4096, 128000, 2048, top=64, tau=2.0),
        # a student with a small vocabulary (bytes and a few symbols): many tokens, few columns
        _case("kd_step_short_vocab", "kd", True, "bf16", 8192, 1000, 512, top=16, tau=1.0),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ce", "kd"])
    step = rng.random() < 0.6
    tokens, vocab, width = spread(1, 8192), spread(1000, 131072), spread(64, 4096)
    if rng.random() < 0.7:
        width = max(64, width // 8 * 8)  # most models' widths
    pad = rng.choice([0, 0, 8, 3])
    most = 4096 * 128000 * 4096 * 0.99
    tokens = max(1, min(tokens, int(most / (vocab * width)), 4096 * 128000 // vocab))
    top = spread(1, 128) if op == "kd" else 1
    tau = rng.choice([1.0, 1.5, 2.0, 4.0]) if op == "kd" else 1.0
    return _case(None, op, step, rng.choice(["bf16", "f16"]), tokens, vocab, width, pad,
                 rng.choice([0.0, 0.1, 0.5]), top, tau)


def _ignored(case):
    return int(case["tokens"] * case["ignored"])


def _rows(values, width, pad, dtype):
    """values as a 16-bit matrix whose rows are width + pad apart."""
    rows = values.shape[0]
    store = torch.zeros(rows, width + pad, dtype=dtype, device=values.device)
    store[:, :width] = values
    return store[:, :width]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev, dtype = torch.device("cuda"), DTYPES[case["dtype"]]
    T, V, D, k = case["tokens"], case["vocab"], case["width"], case["top"]

    # weights of which random hidden states (of unit variance, as after a norm) make logits
    # of deviation 2; each token's state leans towards its own next token
    w = _rows(torch.randn(V, D, generator=gen, device=dev) * (2.0 / math.sqrt(D)), D, case["pad"], dtype)
    # frequent tokens come first: ids spread over the vocabulary's logarithm
    ids = (torch.exp(torch.rand(T, generator=gen, device=dev, dtype=torch.float64) * math.log(V)) - 1).long().clamp_(0, V - 1)
    lean = torch.rand(T, 1, generator=gen, device=dev) * 4.0
    x = torch.randn(T, D, generator=gen, device=dev) + lean * w[ids].float()
    # the masked tokens: whole runs of them, as prompts before answers
    n = _ignored(case)
    masked = torch.zeros(T, dtype=torch.bool, device=dev)
    if n:
        runs = max(1, min(T // 700, n))
        at = torch.arange(T, device=dev)
        run = at * runs // T
        start = torch.div(run * T + runs - 1, runs, rounding_mode="floor")
        share = torch.div((run + 1) * n, runs, rounding_mode="floor") - torch.div(run * n, runs, rounding_mode="floor")
        masked = at - start < share
    x = _rows(x, D, case["pad"], dtype)
    # mean over the tokens learnt from; 16-bit floats of 5 exponent bits are trained with a scaled loss
    g = torch.full((T,), (1024.0 if case["dtype"] == "f16" else 1.0) / max(1, T - n), device=dev)
    state = {"case": case, "x": x, "w": w, "g": g}
    if case["op"] == "ce":
        state["targets"] = torch.where(masked, -100, ids)
        return state
    # a teacher's k best: the token's own id first, the others anywhere, their logits falling off
    step = 1 + torch.randint(0, max(1, (V - 1) // max(k, 1)), (T, 1), generator=gen, device=dev)
    order = torch.arange(k, device=dev)
    top_ids = (ids[:, None] + order * step) % V
    fall = torch.rand(T, 1, generator=gen, device=dev) * 2.0 + 0.5
    logits = 12.0 - fall * torch.sqrt(order.float()) - 0.1 * torch.rand(T, k, generator=gen, device=dev)
    if case["ignored"] and k > 1:  # some rows hold fewer entries, some end in logits of -inf
        few = 1 + torch.randint(0, k, (T, 1), generator=gen, device=dev)
        cut = torch.rand(T, 1, generator=gen, device=dev)
        top_ids = torch.where((cut < 0.1) & (order >= few), -1, top_ids)
        logits = torch.where((cut > 0.9) & (order >= few), -math.inf, logits)
    top_ids = torch.where(masked[:, None], -1, top_ids)
    state["top_ids"], state["top_logits"] = top_ids, logits
    return state


def _targets(state):
    """The target distribution as (ids, weights, logarithms of weights where they count, tokens that count)."""
    V = state["case"]["vocab"]
    if state["case"]["op"] == "ce":
        ids = state["targets"][:, None]
        q = ((ids >= 0) & (ids < V)).float()
        log_q = torch.zeros_like(q)
    else:
        ids, u = state["top_ids"], state["top_logits"] / state["case"]["tau"]
        counts = (ids >= 0) & (ids < V) & (u != -math.inf)
        u = torch.where(counts, u, -math.inf)
        u = u - torch.where(counts.any(1, keepdim=True), u.amax(1, keepdim=True), 0.0)
        e = torch.exp(u)
        total = e.sum(1, keepdim=True)
        q = torch.where(total > 0, e / total, 0.0)
        log_q = torch.where(counts, u - torch.log(total), 0.0)
    return ids.clamp(0, V - 1), q, log_q, (q > 0).any(1, keepdim=True)


def _plain(state):
    case = state["case"]
    tau, dtype = case["tau"], state["x"].dtype
    ids, q, log_q, learnt = _targets(state)
    x = torch.where(learnt, state["x"].float(), 0.0)
    w = state["w"].float()
    z = x @ w.t()
    if tau != 1.0:
        z /= tau
    peak = z.amax(1, keepdim=True)
    at = z.gather(1, ids)
    z.sub_(peak).exp_()
    total = z.sum(1, keepdim=True)
    lse = peak + torch.log(total)
    loss = torch.where(learnt, tau * tau * (q * (log_q - (at - lse))).sum(1, keepdim=True), 0.0)[:, 0]
    lse_out = torch.where(learnt, lse, 0.0)[:, 0]
    if not case["step"]:
        return {"loss": loss, "lse": lse_out}
    z.div_(total)
    z.scatter_add_(1, ids, -q)
    z.mul_(torch.where(learnt, state["g"][:, None] * tau, 0.0))
    return {"loss": loss, "lse": lse_out, "dx": (z @ w).to(dtype), "dw": (z.t() @ x).to(dtype)}


def run(state):
    if not own:
        return _plain(state)
    from dense_fp32_matrix_02_gb300 import loss as L
    case, x, w = state["case"], state["x"], state["w"]
    if case["op"] == "ce":
        loss, lse = L.cross_entropy(x, w, state["targets"])
        if not case["step"]:
            return {"loss": loss, "lse": lse}
        dx, dw = L.cross_entropy_grad(x, w, state["targets"], lse, state["g"])
    else:
        loss, lse = L.distill(x, w, state["top_logits"], state["top_ids"], case["tau"])
        if not case["step"]:
            return {"loss": loss, "lse": lse}
        dx, dw = L.distill_grad(x, w, state["top_logits"], state["top_ids"], lse, state["g"], case["tau"])
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


def work(case):
    T, V, D, k = case["tokens"], case["vocab"], case["width"], case["top"]
    learnt = T - _ignored(case)
    # x of the tokens that count, w, targets (ids, and logits for kd), loss and lse
    nbytes = 2 * learnt * D + 2 * V * D + T * k * (8 if case["op"] == "ce" else 12) + 8 * T
    flops = 2 * learnt * V * D
    if case["step"]:
        nbytes += 2 * T * D + 2 * V * D + 4 * T
        flops *= 3
    return {"bytes": nbytes, "flops": flops}


def exact(case, seed):
    T, V, D = case["tokens"], case["vocab"], case["width"]
    if work(case)["flops"] > 8e12:
        return None
    state = prepare(case, seed)
    tau = case["tau"]
    inf = math.inf
    # the target distribution, entry by entry, from the definition
    if case["op"] == "ce":
        ids = state["targets"].reshape(T, 1)
        u = torch.zeros(T, 1, dtype=torch.float64, device=ids.device)
    else:
        ids, u = state["top_ids"], state["top_logits"].double() / tau
    u = u.masked_fill((ids < 0) | (ids >= V), -inf)
    rows = (u > -inf).any(1).nonzero()[:, 0]
    ids, u = ids[rows].clamp(0, V - 1), u[rows]
    log_q = u - torch.logsumexp(u, 1, keepdim=True)
    q = log_q.exp()
    x = state["x"][rows].double()
    n = rows.numel()
    piece = max(1, min(V, (1 << 27) // max(1, n)))
    lse = torch.full((n,), -inf, dtype=torch.float64, device=x.device)
    for v in range(0, V, piece):
        z = x @ state["w"][v:v + piece].double().t() / tau
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1)) if n else lse
    terms = torch.zeros_like(q)
    for j in range(q.shape[1]):
        log_p = (x * state["w"][ids[:, j]].double()).sum(1) / tau - lse
        terms[:, j] = torch.where(q[:, j] > 0, q[:, j] * (log_q[:, j] - log_p), 0.0)
    zero = torch.zeros(T, dtype=torch.float64, device=x.device)
    out = {"loss": zero.index_copy(0, rows, tau * tau * terms.sum(1)), "lse": zero.index_copy(0, rows, lse)}
    if not case["step"]:
        return out
    g = (state["g"][rows].double() * tau)[:, None]
    dx = torch.zeros(n, D, dtype=torch.float64, device=x.device)
    dw = torch.empty(V, D, dtype=torch.float64, device=x.device)
    for v in range(0, V, piece):
        wv = state["w"][v:v + piece].double()
        G = (x @ wv.t() / tau - lse[:, None]).exp()
        here = (ids >= v) & (ids < v + piece)
        G.scatter_add_(1, (ids - v).clamp(0, wv.shape[0] - 1), torch.where(here, -q, 0.0))
        G *= g
        dx += G @ wv
        dw[v:v + piece] = G.t() @ x
    out["dx"] = torch.zeros(T, D, dtype=torch.float64, device=x.device).index_copy(0, rows, dx)
    out["dw"] = dw
    return out
