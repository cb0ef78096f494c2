"""Log probabilities where they can go wrong: products that give up, logits
that rounding would exchange, words that are all but certain."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from dense_fp32_matrix_02_gb300 import gemm as G  # noqa: E402
from dense_fp32_matrix_02_gb300 import loss as L  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])


def operands(T, V, D, dtype, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, D, generator=gen, device=DEV).to(dtype)
    w = (torch.randn(V, D, generator=gen, device=DEV) * 2 / D ** 0.5).to(dtype)
    ids = torch.randint(0, V, (T,), generator=gen, device=DEV)
    return x, w, ids


@pytest.fixture
def stalled():
    """Products whose operands never come."""
    old = G.set_wait_timeout_ns(20_000_000)
    G.set_debug_flags(G.DEBUG_STALL_PRODUCER)
    yield
    torch.cuda.synchronize()
    G.set_debug_flags(0)
    G.set_wait_timeout_ns(old)
    G.device_status()


@pytest.mark.parametrize("T,V,top", [(300, 20000, 256), (5, 3000, 120),
                                     (1, 700, 20), (300, 700, 20)])
def test_maxima_of_other_logits(stalled, T, V, top):
    """Where the products gave up, the workspace's maxima need not be its
    logits': fewer half tiles than words, whose logits are searched in a range
    that ends at those maxima.  The search ends, with words of the
    vocabulary.  (Logits above the maxima, below them, and any bits.)"""
    x, w, ids = operands(T, V, 64, BF16, T + V)
    n = L.score_workspace_size(T, V, 64, top)
    gen = torch.Generator(device=DEV).manual_seed(V)
    logits = (4 * T * ((V + 7) // 8 * 8) + 255) // 256 * 256
    for low, high in ((-1.0, 3.0), (3.0, -1.0), (0.0, 1e-30), (None, None)):
        ws = torch.randint(0, 256, (n,), generator=gen, device=DEV,
                           dtype=torch.uint8)
        if low is not None:  # (the logits are the workspace's last part)
            ws[n - logits:].view(torch.float32).normal_(high, 2.0,
                                                        generator=gen)
            ws[:n - logits].view(torch.float32).fill_(low)
        s = L.log_probs(x, w, ids, top=top, workspace=ws)
        torch.cuda.synchronize()
        assert G.device_status() == 4
        assert bool(((s.top_ids >= -1) & (s.top_ids < V)).all())


def scores_into(x, w, ids, top, workspace, fill):
    """The C call on outputs that hold `fill` before it: (top_logp, top_ids)."""
    T = x.shape[0]
    head, _ = L._operands(x, w)
    out = torch.full((3, T), fill, device=DEV)
    logp = torch.full((T, top), fill, device=DEV)
    words = torch.full((T, top), int(fill), dtype=torch.int64, device=DEV)
    st = G.lib().gemm_f32_vocab_score(
        *head, ids.data_ptr(), 1.0, top, *(row.data_ptr() for row in out),
        logp.data_ptr(), words.data_ptr(), None, 0, workspace.data_ptr(),
        workspace.numel(), torch.cuda.current_stream().cuda_stream or None)
    assert st == 0
    torch.cuda.synchronize()
    return logp, words


@pytest.mark.parametrize("T,V,top", [(300, 40000, 20), (300, 40000, 256),
                                     (3, 20000, 20), (70, 3000, 120)])
def test_every_word_is_written_where_the_products_gave_up(stalled, T, V, top):
    """Maxima that no logit reaches: no word is found, and none of the outputs
    is left as it was."""
    x, w, ids = operands(T, V, 64, BF16, T + V)
    n = L.score_workspace_size(T, V, 64, top)
    logits = (4 * T * ((V + 7) // 8 * 8) + 255) // 256 * 256
    ws = torch.full((n // 4,), 3.0, device=DEV)
    ws[-(logits // 4):] = -1.0
    logp, words = scores_into(x, w, ids, top, ws.view(torch.uint8), -7777.0)
    assert G.device_status() == 4
    assert bool(((words >= 0) & (words < V)).all())
    assert not bool((logp == -7777.0).any())


def close_words(V, D, n, dtype, seed):
    """x of ones, and n words at random ids whose logits differ by multiples of
    2^-17 around 40: pairs of terms that cancel out, of sizes from 2^-6 to 2^7
    (bfloat16: 2^-9 to 2^10), so that sums in 32 bits are off by more than that
    (a partial sum of 500 or more has a last place of 2^-15 or more).  All
    other logits are below 20."""
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    w = (torch.randn(V, D, generator=gen, device=DEV) * 2 / D ** 0.5).to(dtype)
    at = torch.argsort(rand(V))[:n]
    half = (D - 2) // 2
    e = 6 if dtype == F16 else 9
    r = ((rand(n, half) + 1) * 2.0 ** torch.randint(
        -e, e + 1, (n, half), generator=gen, device=DEV)).to(dtype)
    pairs = torch.cat([r, -r], 1)
    rows = torch.zeros(n, D, dtype=dtype, device=DEV)
    rows[:, 2:2 + 2 * half] = pairs.gather(1, torch.argsort(rand(n, 2 * half), 1))
    rows[:, 0] = 40.0
    rows[:, 1] = torch.arange(n, device=DEV) * 2.0 ** -17
    w[at] = rows
    return torch.ones(1, D, dtype=dtype, device=DEV), w


@TYPES
@pytest.mark.parametrize("V,D,n,top", [
    (5000, 1024, 60, 5), (5000, 1024, 40, 20), (40000, 1024, 200, 1),
    (40000, 2048, 250, 64), (3000, 1000, 250, 200), (900, 520, 120, 10),
    (5000, 1001, 60, 5)])
def test_rank_of_many_words_that_rounding_would_exchange(V, D, n, top, dtype):
    """More words than are looked at beyond `top` lie within what a sum in 32
    bits may be off: the words are those of the operands all the same, and of
    batches of one token, a few tiles and many the same."""
    x, w = close_words(V, D, n, dtype, V + n)
    z = x.double() @ w.double().t()
    want = z.sort(dim=1, descending=True, stable=True).indices[:, :top]
    for T in (1, 200, 300, 1500):  # (blocks of every size)
        ids = torch.zeros(T, dtype=torch.int64, device=DEV)
        s = L.log_probs(x.repeat(T, 1), w, ids, top=top)
        assert torch.equal(s.top_ids, want.expand(T, top))
    assert G.device_status() == 0


def test_rank_among_the_first_words_is_not_enough():
    """The search must go below its first bound: words whose logits in 32 bits
    come out clearly lower than those of others, though theirs are larger."""
    x, w = close_words(6000, 4096, 500, BF16, 3)
    z = x.double() @ w.double().t()
    for top in (1, 3, 30, 100):
        want = z.sort(dim=1, descending=True, stable=True).indices[:, :top]
        for T in (2, 200, 900):
            ids = torch.zeros(T, dtype=torch.int64, device=DEV)
            s = L.log_probs(x.repeat(T, 1), w, ids, top=top)
            assert torch.equal(s.top_ids, want.expand(T, top))


@TYPES
@pytest.mark.parametrize("T", [3, 64, 128])
def test_gradients_of_near_certain_words(T, dtype):
    """1 - p of a word with p near 1 comes from the row's reference and sum,
    not from lse, whose last place is 8e-6 of logits around 80.  The logits are
    exact (small integers over 4), and of 128 tokens and fewer G is kept in two
    16-bit parts, so that what is off in a row of G is
      * at the word: a logarithm's error of 6e-7 (the exponentials, the sum of
        the others and its logarithm, as for logp), |a|·6e-7, and for the
        entropy's gradient 1e-5 of |b| (its own, ten times that);
      * elsewhere p's, a factor of 1 ± 4e-5 (lse's rounding) of |G|;
      * 2^-15 of |G| (binary16 and bfloat16 in two parts), and binary16's
        smallest step under the scale that brings the largest to 2^14.
    dX and dW add those up and round once."""
    V, D = 1000, 64
    u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -11
    gen = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randint(-1, 2, (T, D), generator=gen, device=DEV).to(dtype)
    w = (torch.randint(-4, 5, (V, D), generator=gen, device=DEV) / 4).to(dtype)
    ids = torch.arange(T, device=DEV)
    w[:T] = x / 2
    x[:, 0], w[:, 0] = 8.0, 8.0  # all logits 64 higher
    a = torch.rand(T, generator=gen, device=DEV) + 0.5
    b = 0.1 * torch.rand(T, generator=gen, device=DEV)
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, 1)
    log_p = z - lse[:, None]
    p = log_p.exp()
    H = -(p * log_p).sum(1)
    rows = torch.arange(T, device=DEV)
    some = (1 - p[rows, ids]) < 1e-2
    assert int(some.sum()) > T // 2 and float(lse.min()) > 64
    for with_b in (False, True):
        s = L.log_probs(x, w, ids, keep=True)
        dx, dw = L.log_probs_grad(x, w, ids, s, a, b if with_b else None)
        A = a.double()[:, None]
        B = b.double()[:, None] * with_b
        g = -p * (A + B * (log_p + H[:, None]))
        # (1 - p without the difference)
        rest = p.clone()
        rest[rows, ids] = 0.0
        g[rows, ids] = (A[:, 0] * rest.sum(1)
                        - B[:, 0] * (p[rows, ids] * (log_p[rows, ids] + H)))
        most = float((A + B * (0.4 + H[:, None])).max())
        wrong = g.abs() * (4e-5 + 2.0 ** -15) + p * B * 1e-5
        wrong[rows, ids] += A[:, 0] * 6e-7
        if dtype == F16:
            wrong += most * 2.0 ** -24 / 2.0 ** 13
        for got, left, other, dleft in (
                (dx, g, w.double(), wrong), (dw, g.t(), x.double(), wrong.t())):
            want = left @ other
            tol = (dleft @ other.abs() + u * want.abs()
                   + 1e-6 * (left.abs() @ other.abs())
                   + (2.0 ** -25 if dtype == F16 else 0.0))
            err = (got.double() - want).abs()
            assert bool((err <= tol).all()), float((err / tol).max())
    assert G.device_status() == 0


def test_checked_build_runs_clean():
    """The checked build, in a process of its own: no index leaves its buffer
    where many words are ranked, and where products gave up."""
    import os
    import subprocess
    import sys

    from dense_fp32_matrix_02_gb300 import build
    path = build.build(checked=True)
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k",
         "rank or certain or gave_up or maxima",
         os.path.join(here, "test_gpu_score_edges.py")],
        env=dict(os.environ, GEMM_F32_LIBRARY=path), cwd=here,
        capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
