"""How near the vocabulary losses come to float64, at the widths of real
models: bounds on the error's norm beside those on its elements, since a
bound on every element is a worst case that hides a lost column or a sum kept
in fewer bits.

Where the bounds come from:
  * a logit is sums of at most 16 steps of 64 terms in the tensor cores, 64
    additions of 16 terms, each short of about half a last place (2^-23 of it
    at most) of a sum that grows from 0: 64·2^-24/2 = 2e-6 of it; a few
    additions, an exponential and a logarithm in fp32 bring the norm of loss
    and lse to 3e-6 of theirs;
  * element by element an addition may be short of four last places:
    64·4·2^-23/2 = 1.5e-5 of the largest partial sum, weighted by the
    probabilities in lse; 1e-5 for exponentials and the logarithm, and 2^-21
    of what is subtracted;
  * dX and dW: two roundings to 16 bits (G's and their own), each of a mean
    square of at most u/√3, u = 2^-8 or 2^-11.
"""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import vocab_reference as ref  # noqa: E402
from dense_fp32_matrix_02_gb300 import gemm as G  # noqa: E402
from dense_fp32_matrix_02_gb300 import loss as L  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16


def operands(T, V, D, dtype, seed):
    """Hidden states that lean towards their own word, in rows that start on
    16 bytes."""
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def padded(m):
        store = torch.zeros(m.shape[0], (D + 7) // 8 * 8, dtype=dtype,
                            device=DEV)
        store[:, :D] = m
        return store[:, :D]

    w = padded(normal(V, D) * 2 / math.sqrt(D))
    y = torch.randint(0, V, (T,), generator=gen, device=DEV)
    x = padded(normal(T, D) + 2.0 * torch.rand(
        T, 1, generator=gen, device=DEV) * w[y].float())
    g = torch.rand(T, generator=gen, device=DEV) + 0.5
    return x, w, y, g, gen


def largest_partial(x, w, tau):
    """The sum over a logit's parts (16 steps of 64) of the largest partial
    sum's magnitude in each."""
    D = x.shape[1]
    total = x.new_zeros(x.shape[0], w.shape[0], dtype=torch.float64)
    for k0 in range(0, D, 1024):
        acc, most = torch.zeros_like(total), torch.zeros_like(total)
        for k in range(k0, min(D, k0 + 1024), 64):
            part = slice(k, min(k + 64, k0 + 1024, D))
            acc += x[:, part].double() @ w[:, part].double().t()
            most = torch.maximum(most, acc.abs())
        total += most
    return total / tau


def compare(got, x, w, ids, log_q, tau, g):
    """got against the definitions, by the bounds above."""
    want = ref.loss_and_grads(x, w, ids, log_q, tau, g)
    u = 2.0**-8 if x.dtype == BF16 else 2.0**-11
    learnt = (log_q > -math.inf).any(1)
    for name, most in (("loss", 3e-6), ("lse", 3e-6),
                       ("dx", 2 * u / math.sqrt(3.0)),
                       ("dw", 2 * u / math.sqrt(3.0))):
        a, b = got[name].double(), want[name]
        err = float((a - b).norm() / b.norm())
        assert err <= most, (name, err)
    X = torch.where(learnt[:, None], x.double(), 0.0)
    z = X @ w.double().t() / tau
    d = 1.5e-5 * largest_partial(torch.where(learnt[:, None], x, 0), w, tau)
    lse = want["lse"]
    p = torch.where(learnt[:, None], (z - lse[:, None]).exp(), 0.0)
    lse_tol = (p * d).sum(1) + 1e-5 + 2.0**-21 * lse.abs()
    assert bool(((got["lse"].double() - lse).abs() <= lse_tol)[learnt].all())
    safe, q = ids.clamp(0, w.shape[0] - 1), log_q.exp()
    terms = q * (d.gather(1, safe) + 2.0**-21 * (
        z.gather(1, safe).abs() + log_q.abs().nan_to_num(posinf=0)))
    tol = tau * tau * (lse_tol + terms.sum(1) + 1e-5)
    assert bool(((got["loss"].double() - want["loss"]).abs()
                 <= tol)[learnt].all())
    for name in ("loss", "lse", "dx"):
        assert bool((got[name][~learnt] == 0).all())
    assert G.device_status() == 0


def ce(x, w, y, g):
    loss, lse = L.cross_entropy(x, w, y)
    dx, dw = L.cross_entropy_grad(x, w, y, lse, g)
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


SIZES = [(300, 40000, 1100), (600, 5000, 4096), (20, 9000, 2048),
         (5, 20011, 3000), (257, 3001, 2050), (1300, 2500, 1536)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_cross_entropy(T, V, D, dtype):
    x, w, y, g, gen = operands(T, V, D, dtype, T)
    if T > 10:
        y[torch.rand(T, generator=gen, device=DEV) < 0.1] = -1
    compare(ce(x, w, y, g), x, w, *ref.cross_entropy_targets(y, V), 1.0, g)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_distillation(T, V, D, dtype):
    x, w, y, g, gen = operands(T, V, D, dtype, T + 1)
    top, tau = 12, 1.5
    ids = torch.randint(0, V, (T, top), generator=gen, device=DEV)
    ids[:, 0] = y
    u = 2.0 * torch.randn(T, top, generator=gen, device=DEV)
    ids[torch.rand(T, top, generator=gen, device=DEV) < 0.1] = -1
    loss, lse = L.distill(x, w, u, ids, tau)
    dx, dw = L.distill_grad(x, w, u, ids, lse, g, tau)
    compare({"loss": loss, "lse": lse, "dx": dx, "dw": dw}, x, w,
            *ref.distill_targets(u, ids, tau, V), tau, g)


@pytest.mark.parametrize("T,V,D", [(3, 20011, 1000), (300, 4131, 1100),
                                   (700, 1050, 200), (40, 65, 264)])
def test_last_words_weigh_most(T, V, D):
    """The words past the last multiple of 64 hold most of the probability:
    a lost column shows in every output."""
    x, w, _, g, gen = operands(T, V, D, BF16, T + 2)
    n = V % 64
    assert n
    x[:, 0] = 4.0
    w[:, 0] = 0.0
    w[V - n:, 0] = 2.0
    y = V - 1 - torch.randint(0, min(n, 5), (T,), generator=gen, device=DEV)
    compare(ce(x, w, y, g), x, w, *ref.cross_entropy_targets(y, V), 1.0, g)


@pytest.mark.parametrize("T,D", [(150, 64), (300, 2048)])
def test_not_finite_inputs_spread_as_the_formulas_say(T, D):
    V = 300
    x, w, y, g, _ = operands(T, V, D, BF16, T + 3)
    x[70, 3] = math.nan  # a token: its row, and every element of dw
    got = ce(x, w, y, g)
    for name in ("loss", "lse"):
        assert got[name].isnan().nonzero().flatten().tolist() == [70], name
    assert got["dx"].isnan().any(1).nonzero().flatten().tolist() == [70]
    assert bool(got["dx"][70].isnan().all())
    assert bool(got["dw"].isnan().all())

    # a word's row: its logits are Inf or -Inf by the sign of x
    x[70, 3] = 1.0
    x[:, 5] = torch.where(torch.arange(T, device=DEV) % 2 == 0, 1.0, -1.0)
    word = 123
    y = torch.where(y == word, y + 1, y)
    y[9] = word
    w[word, 5] = math.inf
    loss, lse = L.cross_entropy(x, w, y)
    assert not bool(loss[0::2].isfinite().any())
    assert float(loss[9]) == math.inf
    odd = torch.arange(1, T, 2, device=DEV)
    live = torch.cat([w[:word], w[word + 1:]])
    want = torch.logsumexp(x[odd].double() @ live.double().t(), 1)
    assert bool(((lse[odd].double() - want).abs() <= 1e-4).all())
    odd = odd[odd != 9]
    assert bool(loss[odd].isfinite().all())
    assert G.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("op", ["ce", "kd"])
def test_one_gradient_that_rounds_badly(op, dtype):
    """A mean's gradient, the same for every token, just short of half-way
    between two 16-bit numbers: its rounding would be the same in all targets
    (2^-8 in bfloat16, all of dx and dw).  Scaled to a power of two, a target's
    G = p - 1 is within u/2 of it, u = 2^-8 or 2^-11; the result's own rounding
    adds a mean square of u/√3 at most."""
    u = 2.0**-8 if dtype == BF16 else 2.0**-11
    T, V, D, tau = 400, 5000, 128, 1.0 if op == "ce" else 2.0
    x, w, y, _, _ = operands(T, V, D, dtype, 11)
    w.mul_(0.25)  # probabilities of a model at its start
    for size in (1.0, 2.0**-9, 2.0**9):
        g = torch.full((T,), (1 + u - 2.0**-20) * size / tau, device=DEV)
        if op == "ce":
            got = ce(x, w, y, g)
            targets = ref.cross_entropy_targets(y, V)
        else:
            ids = y[:, None]
            logits = torch.ones(T, 1, device=DEV)
            loss, lse = L.distill(x, w, logits, ids, tau)
            dx, dw = L.distill_grad(x, w, logits, ids, lse, g, tau)
            got = {"dx": dx, "dw": dw}
            targets = ref.distill_targets(logits, ids, tau, V)
        want = ref.loss_and_grads(x, w, *targets, tau, g)
        for name in ("dx", "dw"):
            b = want[name]
            err = float((got[name].double() - b).norm() / b.norm())
            assert err <= u * math.sqrt(1 / 3 + 1 / 4), (name, size, err)


def test_checked_build_runs_clean():
    """Sums of several parts, and deep ones, under the checked build, in a
    process of its own: no index leaves its buffer."""
    import os
    import subprocess
    import sys

    from dense_fp32_matrix_02_gb300 import build
    path = build.build(checked=True)
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k",
         "cross_entropy or distillation or last_words or deep or heart or"
         " lowest",
         os.path.join(here, "test_gpu_loss_accuracy.py"),
         os.path.join(here, "test_gpu_loss_edges.py")],
        env=dict(os.environ, GEMM_F32_LIBRARY=path), cwd=here,
        capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 31, 32, 33, 64, 65, 100, 128])
def test_few_tokens_round_once(T, dtype):
    """A few tokens' gradients are as near as their own rounding lets them: a
    mean square of u/√3 at most (u = 2^-8 or 2^-11), whatever the mantissas of
    their G.  Beside it lse's rounding, 8e-6 of g·τ, against G of 0.1 of it and
    more in the mean.  Some cases of one token, whose G has no others to average with."""
    u = 2.0**-8 if dtype == BF16 else 2.0**-11
    V, D, top, tau = 1500, 136, 3, 1.5
    for seed in range(12 if T < 4 else 2):
        x, w, y, g, gen = operands(T, V, D, dtype, 100 * T + seed)
        ids = torch.randint(0, V, (T, top), generator=gen, device=DEV)
        logits = 2.0 * torch.randn(T, top, generator=gen, device=DEV)
        z = x.double() @ w.double().t()
        p = torch.softmax(z, 1).gather(1, y[:, None])
        assert float((1 - p).square().mean()) > 0.01
        if T > 2:
            y[T // 2] = -1
            ids[T // 2] = V
        loss, lse = L.distill(x, w, logits, ids, tau)
        dx, dw = L.distill_grad(x, w, logits, ids, lse, g, tau)
        for got, targets, t in (
                (ce(x, w, y, g), ref.cross_entropy_targets(y, V), 1.0),
                ({"dx": dx, "dw": dw},
                 ref.distill_targets(logits, ids, tau, V), tau)):
            want = ref.loss_and_grads(x, w, *targets, t, g)
            for name in ("dx", "dw"):
                b = want[name]
                err = float((got[name].double() - b).norm() / b.norm())
                assert err <= u / math.sqrt(3.0) + 8e-5, (name, seed, err)
    assert G.device_status() == 0
