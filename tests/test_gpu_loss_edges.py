"""The vocabulary losses on the GPU at the ends of their ranges: sizes,
values and lengths at which counts overflow, terms vanish or sums run deep.

Tolerances follow tests/vocab_reference.py where a test does not derive its
own."""

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


def test_words_past_2_to_the_30():
    """2^30 + 300 words: a tile's two halves are counted past 2^31.

    All rows of w are 0 but a few, whose logits are 20 (a third of the
    probability) and -3.  Sums of ones are exact in fp32 here; lse is allowed
    1e-6 of itself and 2e-5, G one rounding to bfloat16 (2^-8) and lse's
    error, the products' results another 2^-8 and 1e-5."""
    V, D = 2**30 + 300, 8
    w = torch.zeros(V, D, dtype=BF16, device=DEV)
    hot = torch.tensor([3, 2**29 + 77, V - 1], device=DEV)
    w[hot[0]] = 2.5
    w[hot[1]] = -0.375
    w[hot[2]] = 2.5
    x = torch.ones(2, D, dtype=BF16, device=DEV)
    x[1] = -1.0  # logits of -20, 3 and -20
    y = torch.tensor([V - 1, 2**29 + 77], device=DEV)
    g = torch.tensor([1.0, 2.0], device=DEV)
    loss, lse = L.cross_entropy(x, w, y)
    dx, dw = L.cross_entropy_grad(x, w, y, lse, g)

    z = x.double() @ w[hot].double().t()
    want = torch.log(torch.exp(z).sum(1) + (V - 3))
    tol = 1e-6 * want + 2e-5
    assert bool(((lse.double() - want).abs() <= tol).all()), lse
    at = torch.stack([z[0, 2], z[1, 1]])
    assert bool(((loss.double() - (want - at)).abs() <= 2 * tol).all())
    p = torch.exp(z - want[:, None])
    Q = torch.zeros_like(p)
    Q[0, 2] = Q[1, 1] = 1.0
    P = g.double()[:, None] * (p - Q)
    dP = 2.0**-8 * P.abs() + g.double()[:, None] * p * (tol + 2e-5)[:, None]
    for got, dG, GG, other in ((dx, dP, P, w[hot].double()),
                               (dw[hot], dP.t(), P.t(), x.double())):
        ref = GG @ other
        lim = (dG @ other.abs() + (2.0**-8 + 1e-5) * ref.abs()
               + 1e-5 * (GG.abs() @ other.abs()))
        assert bool(((got.double() - ref).abs() <= lim).all()), (got, ref)
    base = g.double() / torch.exp(want)  # every other row of dw
    ref = (base[:, None] * x.double()).sum(0)
    lim = (base * (2.0**-7 + tol + 3e-5)).sum() + 2.0**-8 * ref.abs()
    cold = torch.tensor([0, 2**29, 2**30 + 17, V - 2], device=DEV)
    assert bool(((dw[cold].double() - ref).abs() <= lim).all())
    assert G.device_status() == 0


def test_a_launch_longer_than_a_wait_is_no_timeout():
    """One launch of about five seconds, 2.5 times the limit of any one wait:
    no wait of it lasts long, and none is reported.  All logits are 0, so
    that lse is log V, within 2 ulp."""
    n, D = 2**18, 49152
    x = torch.zeros(n, D, dtype=BF16, device=DEV)
    y = torch.zeros(n, dtype=torch.int64, device=DEV)
    loss, lse = L.cross_entropy(x, x, y)
    torch.cuda.synchronize()
    assert G.device_status() == 0
    want = math.log(n)
    assert bool(((loss.double() - want).abs() <= 2.0**-19).all())
    assert bool(((lse.double() - want).abs() <= 2.0**-19).all())


@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0, 2.0])
@pytest.mark.parametrize("T", [8, 300])
def test_teacher_logits_of_the_lowest_value(T, tau):
    """Masks that are the type's lowest value, not -inf: entries of weight 0
    beside others; alone in their row, equal ones.  (At a temperature below 1
    they overflowed and gave NaN, or took the token for one without entries.)
    One word's own logit is -inf where a teacher's weight is 0."""
    V, D = 300, 64
    gen = torch.Generator(device=DEV).manual_seed(T)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    x, w = normal(T, D).to(BF16), (normal(V, D) / 4).to(BF16)
    x[:, 0] = 1.0
    w[299] = 0
    w[299, 0] = -math.inf
    low = torch.finfo(torch.float32).min
    u = normal(T, 6)
    ids = torch.randint(0, 299, (T, 6), generator=gen, device=DEV)
    u[0::4, 2:] = low
    u[1::4] = low
    u[1, 3:] = -math.inf
    u[2::4, 1] = -2e5
    u[3::4, 5] = low
    ids[3::4, 5] = 299
    g = torch.rand(T, generator=gen, device=DEV) + 0.5

    loss, lse = L.distill(x, w, u, ids, tau)
    dx, dw = L.distill_grad(x, w, u, ids, lse, g, tau)
    live = w[:299]  # word 299 has no probability and no weight
    # (less each row's largest, beside which float64 would lose log 6)
    ud = u.double() - u.double().amax(1, keepdim=True)
    targets = ref.distill_targets(ud, ids.clamp(max=298), tau, 299)
    want = ref.loss_and_grads(x, live, *targets, tau, g)
    # its 0·(-Inf) in dx is no part of this: nor is it of the loss
    got = {"loss": loss, "lse": lse, "dw": dw[:299]}
    for name in got:
        a, b, tol = got[name].double(), want[name], want[name + "_tol"]
        assert bool(((a - b).abs() <= tol).all()), (name, a, b)
    assert G.device_status() == 0
    # and dx, without that word
    loss, lse = L.distill(x, live, u, ids.clamp(max=298), tau)
    dx, dw = L.distill_grad(x, live, u, ids.clamp(max=298), lse, g, tau)
    assert bool(((dx.double() - want["dx"]).abs() <= want["dx_tol"]).all())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,D", [(5, 4096), (64, 1024), (64, 4096),
                                 (600, 2048), (600, 4096)])
def test_gradients_of_tokens_learnt_by_heart(T, D, dtype):
    """G = p - 1 at the target of a token whose p is nearly 1 is the
    difference of a logit and lse: the two calls have to make the logits
    alike.  Seen in dw's row of each target (no two are the same), along its
    token's x.

    p's error: lse is rounded to fp32 below 32 (2^-20), and again where it is
    made of a power of 2 and where it is turned into one (2^-19 each); the
    exponential's argument (2^-19 of 32·log2 e < 64) and value (2^-22): 8e-6.
    Then G's rounding to 16 bits and dw's, u each, binary16's smallest step
    under the scale 2^14, and the other tokens' parts of the row, each rounded
    likewise."""
    V, u = 8000, 2.0**-8 if dtype == BF16 else 2.0**-11
    gen = torch.Generator(device=DEV).manual_seed(D + T)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    w = (normal(V, D) * 2 / math.sqrt(D)).to(dtype)
    y = torch.randperm(V, generator=gen, device=DEV)[:T]
    lean = 4.0 + 2.0 * torch.rand(T, 1, generator=gen, device=DEV)
    x = (normal(T, D) + lean * w[y].float()).to(dtype)
    g = torch.ones(T, device=DEV)
    _, lse = L.cross_entropy(x, w, y)
    _, dw = L.cross_entropy_grad(x, w, y, lse, g)

    X = x.double()
    z = X @ w.double().t()
    want = torch.logsumexp(z, 1)
    assert float(want.max()) < 32 and float(z.amax()) < 32
    P = (z - want[:, None]).exp()
    z.scatter_(1, y[:, None], -math.inf)
    left = torch.exp(torch.logsumexp(z, 1) - want)  # 1 - p, with all its bits
    assert bool((left < 1e-4).any())
    P.scatter_(1, y[:, None], -left[:, None])
    along = X / (X * X).sum(1, keepdim=True)
    cross = along @ X.t()
    mine = P[:, y]  # [token, target's row]
    ref_g = (mine.t() * cross).sum(1)
    got = (dw[y].double() * along).sum(1)
    step = 0.0 if dtype == BF16 else 2.0**-24 / 2.0**13
    dG = u * mine.abs() + step
    dG = dG + 8e-6 * torch.where(
        torch.eye(T, device=DEV, dtype=torch.bool), 1.0, mine.abs())
    row = mine.t() @ X  # dw's rows of the targets
    tol = ((dG.t() * cross.abs()).sum(1)
           + u * (row.abs() * along.abs()).sum(1) + 1e-5 * left)
    bad = ~((got - ref_g).abs() <= tol)
    assert not bool(bad.any()), (
        int(bad.sum()), (got - ref_g)[bad][:5], tol[bad][:5], left[bad][:5])
    assert G.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,V,D", [(65536, 2048, 64), (262144, 512, 64),
                                   (100_000, 1300, 600), (64, 262144, 4096)])
def test_deep_sums_of_the_gradients(T, V, D, dtype):
    """Many tokens (dW) and many words beside few tokens (dX): the depth of a
    sum does not show in the result, though the tensor cores drop bits at
    every step.  x has one sign, so that the roundings of a row of dw that is
    no target's all go one way.

    What they may add up to: a step of 64 terms is four additions, each short
    of less than two of the sum's last places (2^-23 of it and less; on
    average half of that, while the sum grows to its value from 0): over the
    256 steps of one sum 4·256·2^-23/2 = 6e-5 of it, twice that at most, as a
    mean over many sums.  Beside it stands the mean of the roundings to 16
    bits, which have no sign: none over more than 10^4 results, 1e-5 for
    bfloat16's 2^-9, and lse's own error, 1e-5."""
    gen = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, D, generator=gen, device=DEV)
    x = (x * 0.5 + 1.0).to(dtype)
    w = (torch.randn(V, D, generator=gen, device=DEV) * 2 / math.sqrt(D)).to(
        dtype)
    y = torch.randint(0, V // 8, (T,), generator=gen, device=DEV)
    g = torch.full((T,), 1024.0 / T, device=DEV)
    _, lse = L.cross_entropy(x, w, y)
    dx, dw = L.cross_entropy_grad(x, w, y, lse, g)
    assert G.device_status() == 0

    X = x.double()
    n = max(64, 2**28 // T)  # words at a time
    want = None
    for v in range(0, V, n):
        z = X @ w[v:v + n].double().t()
        part = torch.logsumexp(z, 1)
        want = part if want is None else torch.logaddexp(want, part)
    DX, DW = torch.zeros_like(X), torch.empty(V, D, dtype=torch.float64,
                                              device=DEV)
    for v in range(0, V, n):
        W = w[v:v + n].double()
        P = (X @ W.t() - want[:, None]).exp()
        t = ((y >= v) & (y < v + n)).nonzero()[:, 0]
        P[t, y[t] - v] -= 1.0
        P *= g[:, None].double()
        DX += P @ W
        DW[v:v + n] = P.t() @ X
    cold = DW[V // 8:]
    bias = float(((dw[V // 8:].double() - cold) * cold.sign()).sum()
                 / cold.abs().sum())
    assert abs(bias) <= 1.4e-4, bias
    # and in the norm: G's rounding and the result's (u/√3 each at worst,
    # their mean square), and that bias
    u = 2.0**-8 if dtype == BF16 else 2.0**-11
    for name, got, ref_ in (("dx", dx, DX), ("dw", dw, DW)):
        err = float((got.double() - ref_).norm() / ref_.norm())
        assert err <= 2 * u / math.sqrt(3.0) + 1.4e-4, (name, err)
