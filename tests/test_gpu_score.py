"""Log probabilities, entropy, the likeliest words and their gradients on the
GPU against the definitions in float64 (tolerances: tests/score_reference.py).
The likeliest words have to be the same, rank by rank."""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import score_reference as ref  # noqa: E402
from dense_fp32_matrix_02_gb300 import gemm as G  # noqa: E402
from dense_fp32_matrix_02_gb300 import loss as L  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])


def matrix(rows, cols, dtype, seed, scale=1.0, pad=0, skew=0):
    """Rows cols + pad apart, `skew` elements into the storage; NaN around."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    store = torch.full((skew + rows * (cols + pad),), math.nan, dtype=dtype,
                       device=DEV)
    view = store[skew:].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.randn(rows, cols, generator=gen, device=DEV) * scale)
    return view


def case(T, V, D, dtype, seed=0, ignored=0.0, pad=0, skew=0):
    x = matrix(T, D, dtype, seed, 1.0, pad, skew)
    w = matrix(V, D, dtype, seed + 1, 2.0 / math.sqrt(D), pad, skew)
    gen = torch.Generator(device=DEV).manual_seed(seed + 2)
    ids = torch.randint(0, V, (T,), generator=gen, device=DEV)
    if ignored:
        out = torch.rand(T, generator=gen, device=DEV) < ignored
        ids = torch.where(out, torch.where(ids % 2 == 0, -100, V + ids), ids)
        x[out] = math.nan  # rows that are not scored are not read
    a = torch.randn(T, generator=gen, device=DEV)
    b = 0.3 * torch.randn(T, generator=gen, device=DEV)
    return x, w, ids, a, b


def check(got, want, names):
    for name in names:
        a, b, tol = got[name].double(), want[name], want[name + "_tol"]
        bad = ~((a - b).abs() <= tol)
        assert not bool(bad.any()), (
            f"{name}: {int(bad.sum())} of {bad.numel()} outside tolerance; "
            f"first at {bad.nonzero()[0].tolist()}: got "
            f"{float(a[bad][0])!r}, want {float(b[bad][0])!r}, tol "
            f"{float(tol[bad][0])!r}")
    torch.cuda.synchronize()
    assert G.device_status() == 0


NUMBERS = ("logp", "lse", "entropy")


def check_scores(x, w, ids, tau=1.0, top=0, **kw):
    s = L.log_probs(x, w, ids, top=top, temperature=tau, **kw)
    want = ref.scores(x, w, ids, tau, top)
    check(s._asdict(), want, NUMBERS)
    if top:
        check(s._asdict(), want, ("top_logp",))
        assert torch.equal(s.top_ids, want["top_ids"])
        # the given word among them has its own log probability, to the bit
        own = s.top_ids == ids[:, None]
        logp = s.logp[:, None].expand_as(s.top_logp)
        assert torch.equal(s.top_logp[own], logp[own])
    else:
        assert s.top_ids is None and s.top_logp is None
    return s


def check_step(x, w, ids, a, b, tau=1.0, **kw):
    s = check_scores(x, w, ids, tau, keep=True)
    dx, dw = L.log_probs_grad(x, w, ids, s, a, b, temperature=tau, **kw)
    check({"dx": dx, "dw": dw}, ref.gradients(x, w, ids, a, b, tau),
          ("dx", "dw"))
    return dx, dw


SIZES = [(1, 1, 1), (1, 1000, 64), (2, 5, 7), (63, 255, 63), (64, 256, 64),
         (65, 257, 65), (127, 511, 128), (128, 512, 200), (129, 513, 72),
         (255, 1000, 520), (256, 20000, 64), (257, 129, 264), (300, 4099, 96),
         (513, 70, 136), (1030, 300, 33), (3, 20011, 1000), (2100, 3001, 160)]


@TYPES
@pytest.mark.parametrize("T,V,D", SIZES)
def test_scores_sizes(T, V, D, dtype):
    x, w, ids, _, _ = case(T, V, D, dtype, seed=T + V)
    for top in (0, min(5, V)):
        check_scores(x, w, ids, 1.0, top)


@TYPES
@pytest.mark.parametrize("T,V,D", SIZES)
def test_step_sizes(T, V, D, dtype):
    x, w, ids, a, b = case(T, V, D, dtype, seed=T + V + 9)
    check_step(x, w, ids, a, b)


@TYPES
@pytest.mark.parametrize("ignored", [0.02, 0.5, 0.97, 1.0])
@pytest.mark.parametrize("T", [40, 700])
def test_unscored_tokens(T, ignored, dtype):
    x, w, ids, a, b = case(T, 900, 72, dtype, 5, ignored)
    a[ids < 0] = math.nan  # nothing of an unscored token counts
    check_scores(x, w, ids, 1.0, 7)
    dx, _ = check_step(x, w, ids, a, b)
    out = (ids < 0) | (ids >= 900)
    assert bool((dx[out] == 0).all())


@TYPES
@pytest.mark.parametrize("tau", [0.25, 0.7, 3.0])
def test_temperatures(tau, dtype):
    x, w, ids, a, b = case(300, 1500, 96, dtype, 6, 0.1)
    check_scores(x, w, ids, tau, 9)
    check_step(x, w, ids, a, b, tau)


@TYPES
@pytest.mark.parametrize("pad,skew", [(0, 1), (3, 0), (5, 2), (8, 8), (8, 4)])
def test_rows_off_boundaries(pad, skew, dtype):
    x, w, ids, a, b = case(150, 700, 61, dtype, 7, 0.1, pad, skew)
    check_scores(x, w, ids, 1.0, 6)
    check_step(x, w, ids, a, b)
    x, w, ids, a, b = case(20, 300, 67, dtype, 8, 0.0, pad, skew)
    dx = matrix(20, 67, dtype, 1, 1.0, 5, 1)
    dw = matrix(300, 67, dtype, 1, 1.0, 1, 3)
    check_step(x, w, ids, a, b, dx=dx, dw=dw)
    for m in (dx, dw):  # what lies between the rows is left as it was
        gap = m.as_strided((m.shape[0] - 1, m.stride(0) - m.shape[1]),
                           (m.stride(0), 1), m.storage_offset() + m.shape[1])
        assert bool(gap.isnan().all())


@TYPES
@pytest.mark.parametrize("D,pad,skew", [
    (505, 0, 0), (511, 0, 1), (512, 1, 2), (520, 3, 3), (1003, 0, 4),
    (1019, 2, 5), (1025, 0, 6), (1031, 1, 7), (2045, 0, 0), (2050, 0, 0)])
def test_long_rows_off_boundaries(D, pad, skew, dtype):
    """Rows long enough to be packed piece by piece, from every element of a
    16-byte boundary on; gradients in rows that start on even and odd
    elements."""
    for T in (3, 140):
        x, w, ids, a, b = case(T, 333, D, dtype, D, 0.0, pad, skew)
        check_scores(x, w, ids, 1.0, 4)
        dx = matrix(T, D, dtype, 1, 1.0, pad, skew)
        dw = matrix(333, D, dtype, 1, 1.0, pad, skew)
        check_step(x, w, ids, a, b, dx=dx, dw=dw)
        for m in (dx, dw) if pad else ():
            gap = m.as_strided((m.shape[0] - 1, pad), (m.stride(0), 1),
                               m.storage_offset() + D)
            assert bool(gap.isnan().all())


@pytest.mark.parametrize("top", [1, 2, 8, 31, 64, 100, 255, 256])
@pytest.mark.parametrize("T,V", [(3, 256), (5, 300), (40, 5000), (300, 40000),
                                 (500, 20000), (1100, 700), (1500, 40000)])
def test_numbers_of_words(T, V, top):
    """Vocabularies of fewer stretches than words asked for, of about as
    many, and of many more."""
    x, w, ids, _, _ = case(T, V, 48, BF16, top)
    check_scores(x, w, ids, 1.0, top)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 15, 16])
def test_all_words(V):
    x, w, ids, _, _ = case(33, V, 24, F16, V)
    check_scores(x, w, ids, 1.3, V)


def test_more_stretches_than_are_held():
    """Vocabularies whose stretches' maxima are read again from memory."""
    x, w, ids, _, _ = case(2, 300_007, 16, BF16, 3)
    check_scores(x, w, ids, 1.0, 20)
    x, w, ids, _, _ = case(300, 270_001, 16, BF16, 3)
    check_scores(x, w, ids, 1.0, 20)


def test_equal_logits_by_the_lower_id():
    """Small integers: logits are exact, and most are equal to others."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    for T, V in ((1, 3000), (9, 700), (300, 12000), (500, 3000), (500, 40000),
                 (1200, 700), (1200, 40000)):
        x = torch.randint(-1, 2, (T, 16), generator=gen, device=DEV).to(BF16)
        w = torch.randint(-1, 2, (V, 16), generator=gen, device=DEV).to(BF16)
        x[0] = 0  # every logit is 0
        w[V // 2:] = w[:V - V // 2].clone()
        ids = torch.randint(0, V, (T,), generator=gen, device=DEV)
        for top in (1, 5, 40, 256):
            check_scores(x, w, ids, 1.0, top)


def test_rank_is_before_rounding():
    """Logits that differ by less than fp32 sums of their size hold: the
    rank is the operands', whatever the batch's size."""
    D, V = 2048, 4000
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(1, D, generator=gen, device=DEV).to(BF16)
    row = torch.randn(1, D, generator=gen, device=DEV).to(BF16)
    w = row.repeat(V, 1)
    # one element of each row off by steps of its last place, at places where x
    # is small: logits some 1e-6 of their terms' sum apart
    at = x[0].float().abs().argsort()[64:64 + V % D + 1]
    for v in range(V):
        j = int(at[v % at.numel()])
        w[v, j] = w[v, j].float() * (1 + 2.0 ** -7 * (1 + v % 3))
    for T in (1, 300):
        xs = x.repeat(T, 1)
        ids = torch.zeros(T, dtype=torch.int64, device=DEV)
        z = xs[:1].double() @ w.double().t()
        s = L.log_probs(xs, w, ids, top=8)
        got = z[0][s.top_ids[0]]
        assert bool((got[:-1] >= got[1:]).all())
        assert torch.equal(s.top_ids, s.top_ids[:1].expand(T, 8))


@TYPES
def test_infinite_and_missing_logits(dtype):
    """Words whose row holds -Inf (masked): probability 0, ranked last; a
    row of x that holds NaN: NaN for that token alone."""
    x, w, ids, _, _ = case(70, 500, 40, dtype, 9)
    x.abs_().add_(0.125)
    w[100:499, 3] = -math.inf
    ids.remainder_(100)
    x[5, 7] = math.nan
    s = L.log_probs(x, w, ids, top=120)
    keep = torch.arange(70, device=DEV) != 5
    small = torch.cat([w[:100], w[499:]])
    want = ref.scores(x[keep], small, ids[keep], 1.0, 101)
    got = {n: getattr(s, n)[keep] for n in NUMBERS}
    check(got, want, NUMBERS)
    order = torch.where(want["top_ids"] == 100, 499, want["top_ids"])
    assert torch.equal(s.top_ids[keep][:, :101], order)
    assert bool((s.top_logp[keep][:, 101:] == -math.inf).all())
    last = torch.arange(100, 119, device=DEV)
    assert bool((s.top_ids[keep][:, 101:] == last).all())
    for n in NUMBERS:
        assert bool(getattr(s, n)[5].isnan())
    assert bool(((s.top_ids[5] >= 0) & (s.top_ids[5] < 500)).all())


@TYPES
def test_masked_words_gradients(dtype):
    """p = 0: no gradient reaches a word of logit -Inf by way of G."""
    x, w, ids, a, b = case(40, 300, 40, dtype, 11)
    x.abs_().add_(0.125)
    w[200:, 3] = -math.inf
    ids.remainder_(200)
    s = L.log_probs(x, w, ids, keep=True)
    _, dw = L.log_probs_grad(x, w, ids, s, a, b)
    assert bool((dw[200:] == 0).all())
    want = ref.gradients(x, w[:200], ids, a, b)
    check({"dw": dw[:200]}, want, ("dw",))


def test_sharp_and_flat_distributions():
    """A distribution that is one word (entropy near 0), and equal logits
    (entropy log V)."""
    D, V, T = 64, 4000, 30
    x, w, ids, a, b = case(T, V, D, BF16, 12)
    w[ids[0]] = 8 * x[0]
    x[1] = 0
    s = check_scores(x, w, ids, 1.0, 3)
    assert 0 <= float(s.entropy[0]) < 1e-6 and int(s.top_ids[0, 0]) == ids[0]
    assert abs(float(s.entropy[1]) - math.log(V)) < 1e-5
    check_step(x, w, ids, a, b)


@TYPES
def test_near_certain_words(dtype):
    """Log probabilities near 0 keep their own digits, not lse's.  The logits
    are exact (small integers over 4), so what is left is one exponential near
    1 (2^-22), the sum of the others (1e-6 of it), the rounding of a sum near
    1 and of its logarithm (2^-23 each): 6e-7, where lse's own rounding would
    be 2e-6 of logits of 20."""
    T, V, D = 64, 1000, 64
    gen = torch.Generator(device=DEV).manual_seed(33)
    x = torch.randint(-1, 2, (T, D), generator=gen, device=DEV).to(dtype)
    w = (torch.randint(-4, 5, (V, D), generator=gen, device=DEV) / 4).to(dtype)
    ids = torch.arange(T, device=DEV)
    w[:T] = x / 2
    s = L.log_probs(x, w, ids, top=3)
    want = ref.scores(x, w, ids, 1.0, 3)
    assert float(want["lse"].median()) > 18
    assert float(want["logp"].median()) > -0.02
    for got, exact in ((s.logp, want["logp"]), (s.entropy, want["entropy"]),
                       (s.top_logp[:, 0], want["top_logp"][:, 0])):
        close = want["logp"] > -0.05
        err = (got.double() - exact).abs()[close]
        assert int(close.sum()) > T // 2
        # (entropy: the others' terms, each log p ~ -10 of them)
        scale = 1.0 if got is not s.entropy else 10.0
        assert float(err.max()) <= 6e-7 * scale


@TYPES
def test_no_gradient_of_entropy(dtype):
    """None, zeros and cross entropy's gradient of the opposite sign."""
    x, w, ids, a, _ = case(300, 900, 72, dtype, 13, 0.2)
    s = L.log_probs(x, w, ids, keep=True)
    dx, dw = L.log_probs_grad(x, w, ids, s, a)
    check({"dx": dx, "dw": dw}, ref.gradients(x, w, ids, a), ("dx", "dw"))
    zero = torch.zeros(1, device=DEV).expand(300)
    dx2, dw2 = L.log_probs_grad(x, w, ids, s, a, zero)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    loss, lse = L.cross_entropy(x, w, ids)
    assert bool(((loss + s.logp).abs() <= 1e-5).all())
    assert bool(((lse - s.lse).abs() <= 1e-5).all())


def test_gradients_are_differences():
    """The slope of Σ a·logp + b·entropy along directions."""
    x, w, ids, a, b = case(60, 300, 64, BF16, 14)
    s = L.log_probs(x, w, ids, keep=True)
    dx, dw = L.log_probs_grad(x, w, ids, s, a, b)
    gen = torch.Generator(device=DEV).manual_seed(15)
    for g, m in ((dx, x), (dw, w)):
        for _ in range(3):
            way = torch.randn(m.shape, generator=gen, device=DEV).double()
            h, ends = 1e-4, []
            for sign in (h, -h):
                xs, ws = x.double(), w.double()
                if m is x:
                    xs = xs + sign * way
                else:
                    ws = ws + sign * way
                r = ref.scores(xs, ws, ids)
                ends.append((a * r["logp"] + b * r["entropy"]).sum())
            slope = float(ends[0] - ends[1]) / (2 * h)
            along = float((g.double() * way).sum())
            # G's and the results' roundings, one way at most as a sum
            tol = 2.0 ** -7 * float((g.double() * way).abs().sum())
            assert abs(slope - along) <= tol


@pytest.mark.parametrize("T", [300, 515])
def test_logits_of_some_tokens_at_a_time(T):
    """More logits than the workspace holds at once: several launches."""
    V = (1 << 22) + 77
    x, w, ids, _, _ = case(T, V, 16, BF16, 16, 0.05)
    # (256 tokens' logits and the statistics: less than all logits)
    assert L.score_workspace_size(T, V, 16, 4) < 4 * T * V
    s = L.log_probs(x, w, ids, top=4)
    for t0 in (0, 240, 256, T - 16):
        part = slice(t0, t0 + 16)
        want = ref.scores(x[part], w, ids[part], 1.0, 4)
        got = {n: v[part] for n, v in s._asdict().items() if v is not None}
        check(got, want, (*NUMBERS, "top_logp"))
        assert torch.equal(got["top_ids"], want["top_ids"])


def test_kept_logits_past_32_bits():
    """More kept logits than 2^31: the gradients of the last words and of the
    last tokens, from the definition."""
    T, V, D = 520, (1 << 22) + 77, 16
    x, w, ids, a, b = case(T, V, D, BF16, 35)
    ids[-8:] = torch.arange(V - 8, V, device=DEV)
    s = L.log_probs(x, w, ids, keep=True)
    dx, dw = L.log_probs_grad(x, w, ids, s, a, b)
    lse, H = s.lse.double(), s.entropy.double()

    def grads(rows, words):
        log_p = x[rows].double() @ w[words].double().t() - lse[rows][:, None]
        g = -log_p.exp() * (a[rows].double()[:, None] + b[rows].double()[:, None]
                            * (log_p + H[rows][:, None]))
        hit = ids[rows][:, None] == torch.arange(V, device=DEV)[words]
        return g + hit * a[rows].double()[:, None]

    u = 2.0 ** -8  # G's rounding and the result's; p's own error, 1e-4
    every, last = slice(0, T), slice(V - 300, V)
    g = grads(every, last)
    want = g.t() @ x.double()
    tol = (u + 1e-4) * (g.abs().t() @ x.double().abs()) + u * want.abs()
    assert bool(((dw[last].double() - want).abs() <= tol).all())
    rows = slice(T - 4, T)
    want = torch.zeros(4, D, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(want)
    for v in range(0, V, 1 << 20):
        g = grads(rows, slice(v, min(V, v + (1 << 20))))
        wv = w[v:v + (1 << 20)].double()
        want += g @ wv
        size += g.abs() @ wv.abs()
    tol = (u + 1e-4) * size + u * want.abs()
    assert bool(((dx[rows].double() - want).abs() <= tol).all())
    torch.cuda.synchronize()
    assert G.device_status() == 0


@pytest.mark.parametrize("T", [30, 600])
def test_pieces_of_the_vocabulary(T):
    """Gradients in several pieces of G (128 MB each)."""
    V = 300_001 if T < 100 else 150_001
    x, w, ids, a, b = case(T, V, 24, BF16, 17, 0.1)
    check_step(x, w, ids, a, b)


def test_gradients_want_what_was_kept():
    """Kept without a copy of w (its rows were aligned), gradients of the same
    values in rows that are not are refused: their copy is not there."""
    x, w, ids, a, b = case(70, 300, 64, BF16, 34)
    off = matrix(300, 64, BF16, 1, 1.0, 3, 1)
    off.copy_(w)
    s = L.log_probs(x, w, ids, keep=True)
    with pytest.raises(G.GemmError):
        L.log_probs_grad(x, off, ids, s, a, b)
    want = L.log_probs_grad(x, w, ids, s, a, b)
    s = L.log_probs(x, off, ids, keep=True)  # the other way round nothing lacks
    for wx in (off, w):
        for p, q in zip(L.log_probs_grad(x, wx, ids, s, a, b), want):
            assert torch.equal(p, q)


def test_large_gradients_and_none():
    x, w, ids, a, b = case(200, 400, 40, F16, 18)
    for scale in (1e-30, 1e4):
        s = L.log_probs(x, w, ids, keep=True)
        dx, dw = L.log_probs_grad(x, w, ids, s, a * scale, b * scale)
        if scale > 1:
            want = ref.gradients(x, w, ids, a * scale, b * scale)
            # (some are beyond 65520, which binary16 rounds to infinity by
            # definition: both sides end at its largest number)
            for name in ("dx", "dw"):
                want[name].clamp_(-65504.0, 65504.0)
            check({"dx": dx.clamp(-65504.0, 65504.0),
                   "dw": dw.clamp(-65504.0, 65504.0)}, want, ("dx", "dw"))
    dx, dw = L.log_probs_grad(x, w, ids, s, a * 0, b * 0)
    assert bool((dx == 0).all()) and bool((dw == 0).all())


def test_no_tokens():
    x, w, ids, a, b = case(4, 300, 40, BF16, 19)
    s = L.log_probs(x[:0], w, ids[:0], top=3, keep=True)
    assert s.logp.shape == (0,) and s.top_ids.shape == (0, 3)
    dx, dw = L.log_probs_grad(x[:0], w, ids[:0], s, a[:0], b[:0])
    assert dx.shape == (0, 40) and bool((dw == 0).all())


def test_same_bits_and_batches():
    """The same call gives the same bits, and workspaces need no values."""
    x, w, ids, a, b = case(700, 5000, 136, BF16, 20, 0.1)
    def run(**kw):
        s = L.log_probs(x, w, ids, top=5, keep=True, **kw)
        return (*s[:5], *L.log_probs_grad(x, w, ids, s, a, b, **kw))
    first = run()
    n = L.score_workspace_size(700, 5000, 136, 5, True, True)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)
    for got, want in zip(run(workspace=ws), first):
        assert torch.equal(got, want)


def test_graphs_share_a_workspace():
    """Forward and backward captured, beside another captured call on the
    same workspace, replayed in turn on changed inputs."""
    x, w, ids, a, b = case(260, 3000, 64, BF16, 21, 0.1)
    x2 = x.clone()
    n = L.score_workspace_size(260, 3000, 64, 5, False, True)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def step(x):
        s = L.log_probs(x, w, ids, top=5, keep=True, workspace=ws)
        return s, L.log_probs_grad(x, w, ids, s, a, b, workspace=ws)

    def score(x):
        return L.log_probs(x, w, ids, top=5, workspace=ws)

    want, want2 = step(x), score(x2)  # (and the one-time set-up)
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(x)
    with torch.cuda.graph(g2):
        got2 = score(x2)
    for _ in range(2):
        g.replay()
        g2.replay()
    torch.cuda.synchronize()
    pairs = [*zip(got[0][:5], want[0][:5]), *zip(got[1], want[1]),
             *zip(got2[:5], want2[:5])]
    for p, q in pairs:
        assert torch.equal(p.nan_to_num(9.0), q.nan_to_num(9.0))
    ids.copy_(ids.roll(1))
    x.copy_(x.roll(1, 0))
    g.replay()
    check(got[0]._asdict(), ref.scores(x, w, ids, 1.0, 5), NUMBERS)


def test_streams():
    x, w, ids, a, b = case(300, 3000, 64, BF16, 22)
    want = L.log_probs(x, w, ids, top=5, keep=True)
    wx, ww = L.log_probs_grad(x, w, ids, want, a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = L.log_probs(x, w, ids, top=5, keep=True, stream=side)
    dx, dw = L.log_probs_grad(x, w, ids, s, a, b, stream=side)
    side.synchronize()
    for p, q in zip((*s[:5], dx, dw), (*want[:5], wx, ww)):
        assert torch.equal(p, q)


def test_teacher_and_student():
    """The likeliest words of a teacher are what distillation learns from:
    a student with the teacher's own matrix has next to no loss."""
    x, w, ids, _, _ = case(200, 1000, 64, BF16, 23, 0.1)
    s = L.log_probs(x, w, ids, top=256)
    kd, _ = L.distill(x, w, s.top_logp, s.top_ids)
    rest = (1 - s.top_logp.exp().sum(1)).clamp_min(0)
    # the divergence is -log of the probability the entries hold
    want = torch.where(ids < 0, 0.0, -torch.log1p(-rest))
    want = torch.where(ids >= 1000, 0.0, want)
    assert bool(((kd - want).abs() <= 1e-4).all())


def test_policy_gradient_step():
    """A run as they are used together: scores, their gradients, clipped;
    the bound holds and the objective rises along the step."""
    from dense_fp32_matrix_02_gb300 import grads as C
    x, w, ids, a, b = case(400, 2000, 96, BF16, 24, 0.2)
    scored = (ids >= 0) & (ids < 2000)
    x = torch.where(scored[:, None], x, 0)
    s = L.log_probs(x, w, ids, keep=True)
    dx, dw = L.log_probs_grad(x, w, ids, s, a, b)
    want = math.sqrt(float((dx.double() ** 2).sum() + (dw.double() ** 2).sum()))
    norm = C.clip_([dx, dw], 0.5 * want)
    assert abs(float(norm) - want) <= 2e-6 * want
    half = math.sqrt(float((dx.double() ** 2).sum() + (dw.double() ** 2).sum()))
    assert abs(half - 0.5 * want) <= 2.0 ** -8 * want
    def value(x, w):
        r = ref.scores(x, w, ids)
        return float((a * r["logp"] + b * r["entropy"]).sum())
    h = 1e-4
    up = value(x.double() + h * dx.double(), w.double() + h * dw.double())
    assert up > value(x, w)


def test_refusals():
    x, w, ids, a, b = case(4, 30, 8, BF16, 25)
    for bad in (31, 257):
        with pytest.raises(G.GemmError):
            L.log_probs(x, w, ids, top=bad)
    with pytest.raises(ValueError, match="negative"):
        L.log_probs(x, w, ids, top=-1)
    for tau in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(G.GemmError):
            L.log_probs(x, w, ids, temperature=tau)
    s = L.log_probs(x, w, ids)
    with pytest.raises(ValueError, match="keep"):
        L.log_probs_grad(x, w, ids, s, a)
    s = L.log_probs(x, w, ids, keep=True)
    with pytest.raises(G.GemmError):
        L.log_probs_grad(x, w, ids, s._replace(kept=s.kept[:64]), a)
    with pytest.raises(ValueError, match="grad_logp"):
        L.log_probs_grad(x, w, ids, s, a[:3])
    with pytest.raises(TypeError):
        L.log_probs_grad(x, w, ids, s, a, b.double())
    with pytest.raises(ValueError, match="ids"):
        L.log_probs(x, w, ids[:3])


def test_checked_build_runs_clean():
    """The checked build, in a process of its own: no index leaves its
    buffer, and every result is in its tolerance."""
    import os
    import subprocess
    import sys

    from dense_fp32_matrix_02_gb300 import build
    path = build.build(checked=True)
    here = os.path.dirname(os.path.abspath(__file__))
    which = ("sizes or unscored or off_boundaries or numbers or all_words or held"
             " or lower or missing or masked or pieces or tokens_at_a_time")
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k", which,
         os.path.join(here, "test_gpu_score.py")],
        env=dict(os.environ, GEMM_F32_LIBRARY=path), cwd=here,
        capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]


def test_other_device_is_refused_or_used():
    """Operands of another device than the current one are worked on there;
    mixed devices are refused (here: the host beside the GPU)."""
    x, w, ids, a, _ = case(4, 30, 8, BF16, 26)
    with pytest.raises(ValueError, match="device"):
        L.log_probs(x, w, ids.cpu())
    with pytest.raises(ValueError):
        L.log_probs(x, w.cpu(), ids)
    s = L.log_probs(x, w, ids, keep=True)
    with pytest.raises(ValueError, match="device"):
        L.log_probs_grad(x, w, ids, s, a.cpu())
    with pytest.raises(ValueError, match="device"):
        L.log_probs_grad(x, w, ids, s._replace(kept=s.kept.cpu()), a)


def test_waits_that_run_out():
    """Products whose operands never come give up, report it and leave the
    device usable; what follows them works on whatever the workspace holds, here
    words' maxima that belong to no logits."""
    x, w, ids, a, b = case(300, 40000, 128, BF16, 36, 0.1)
    want = L.log_probs(x, w, ids, top=20, keep=True)
    grads = L.log_probs_grad(x, w, ids, want, a, b)
    torch.cuda.synchronize()
    n = L.score_workspace_size(300, 40000, 128, 20, False, False)
    gen = torch.Generator(device=DEV).manual_seed(37)
    old = G.set_wait_timeout_ns(20_000_000)
    G.set_debug_flags(G.DEBUG_STALL_PRODUCER)
    try:
        for _ in range(2):
            ws = torch.randint(0, 256, (n,), generator=gen, device=DEV,
                               dtype=torch.uint8)
            s = L.log_probs(x, w, ids, top=20, workspace=ws)
            torch.cuda.synchronize()
            assert G.device_status() == 4
            assert bool(((s.top_ids >= -1) & (s.top_ids < 40000)).all())
        L.log_probs_grad(x, w, ids, want, a, b)
        torch.cuda.synchronize()
        assert G.device_status() == 4
    finally:
        G.set_debug_flags(0)
        G.set_wait_timeout_ns(old)
    s = L.log_probs(x, w, ids, top=20, keep=True)
    got = L.log_probs_grad(x, w, ids, s, a, b)
    for p, q in zip((*s[:5], *got), (*want[:5], *grads)):
        assert torch.equal(p, q)
    assert G.device_status() == 0


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, do not meet."""
    cases = [case(300, 3000, 64, BF16, 30), case(77, 9000, 136, F16, 31)]
    streams = [torch.cuda.Stream() for _ in cases]
    want = [L.log_probs(x, w, ids, top=6, keep=True)
            for x, w, ids, _, _ in cases]
    grads = [L.log_probs_grad(x, w, ids, s, a, b)
             for s, (x, w, ids, a, b) in zip(want, cases)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for (x, w, ids, a, b), stream in zip(cases, streams):
            with torch.cuda.stream(stream):
                s = L.log_probs(x, w, ids, top=6, keep=True)
                got.append((s, L.log_probs_grad(x, w, ids, s, a, b)))
    torch.cuda.synchronize()
    for i, (s, g) in enumerate(got):
        for p, q in zip((*s[:5], *g), (*want[i % 2][:5], *grads[i % 2])):
            assert torch.equal(p, q)
