"""How near log probabilities, entropy and their gradients come to float64, at
the widths of real models: bounds on the error's norm and mean beside those on
elements, which are a worst case that hides a sum kept in fewer bits.

Where the bounds come from.  A logit is sums of 8 steps of 64 terms in the tensor
cores (4 steps up to 8 tokens): 32 (16) additions of 16 terms, each short of 0 to 1
last places (towards 0), half of one in the mean, of a sum that grows from 0.  A
last place is 2^-24 to 2^-23 of the sum, 2^-24/ln 2 in the mean over its
mantissas, so the logit is short of s = 32/2·2^-25/ln 2 = 6.9e-7 of itself
(3.4e-7).  Sums of 16 steps (they lose 9.6e-7, where 8 lose 4.7e-7) are outside
the bounds on the mean.  Then, p the distribution and E_p its mean,
  * lse is short of s·E_p|z|, logp of s·(|z_y| + E_p|z|);
  * the derivative of the entropy along the logits' size is the variance of the
    logits under p: s·Var_p(z);
  * the rest rounds without a side: an exponential (2^-22) and sums of them, a
    logarithm and the results' own place, 2^-22 of lse and of the logit each
    (their difference's), and 2^-21 of the entropy's two terms, log S and E/S,
    log V at most.  In the tokens' mean it falls by their number's root, and
    what is left is what all exponentials share, 2^-23 of S.
dX and dW: two roundings to 16 bits (G's and their own; of 128 tokens and fewer
the result's alone), each of a mean square of at most u/√3, u = 2^-8 or 2^-11.
"""

from __future__ import annotations

import math

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


def operands(T, V, D, dtype, seed, spread, lean=2.0):
    """Hidden states that lean towards their own word; logits of deviation
    `spread`."""
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    w = (normal(V, D) * spread / math.sqrt(D)).to(dtype)
    y = torch.randint(0, V, (T,), generator=gen, device=DEV)
    x = (normal(T, D) + lean * torch.rand(T, 1, generator=gen, device=DEV)
         * w[y].float()).to(dtype)
    return x, w, y, gen


def exactly(x, w, y, tau):
    z = x.double() @ w.double().t() / tau
    lse = torch.logsumexp(z, 1)
    log_p = z - lse[:, None]
    p = log_p.exp()
    at = z.gather(1, y[:, None])[:, 0]
    mean = (p * z).sum(1)
    return {"logp": at - lse, "lse": lse, "entropy": -(p * log_p).sum(1),
            "at": at, "size": (p * z.abs()).sum(1),
            "var": (p * (z - mean[:, None]) ** 2).sum(1),
            "log_p": log_p, "p": p}


def check_scores(s, want, T, V):
    short = (8 if T <= 8 else 16) * 2.0 ** -25 / math.log(2.0)
    size, at, var = want["size"], want["at"].abs(), want["var"]
    # what is lost on one side, and what rounds without one
    one = {"lse": short * size, "logp": short * (at + size),
           "entropy": short * var}
    two = {"lse": 2.0 ** -22 * want["lse"].abs(),
           "logp": 2.0 ** -22 * (want["lse"].abs() + at),
           "entropy": torch.full_like(var, 2.0 ** -21 * math.log(V))}
    for name in one:
        err = s[name].double() - want[name]
        norm, most = float(err.norm()), float((one[name] + two[name]).norm())
        assert norm <= most, (name, norm / most)
        mean = abs(float(err.mean()))
        most = float(one[name].mean() + 2.0 ** -23
                     + two[name].mean() * 3 / math.sqrt(T))
        if T >= 1000:
            assert mean <= most, (name, mean / most)


SIZES = [(1, 32000, 768), (7, 20011, 3000), (64, 32000, 4096),
         (300, 40000, 1100), (2045, 20021, 1000), (2000, 9000, 2048),
         (1500, 30000, 768)]


@TYPES
@pytest.mark.parametrize("tau", [1.0, 0.7])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_scores(T, V, D, tau, dtype):
    x, w, y, _ = operands(T, V, D, dtype, T, 2.0)
    s = L.log_probs(x, w, y, temperature=tau)
    check_scores(s._asdict(), exactly(x, w, y, tau), T, V)
    assert G.device_status() == 0


@pytest.mark.parametrize("D", [512, 1000, 2048, 4096])
def test_wide_distributions_lose_no_more_than_8_steps_do(D):
    """Logits of deviation 3.5, all of whose variance the entropy shows: sums
    that lose twice as much are outside."""
    T, V = 4000, 30000
    x, w, y, _ = operands(T, V, D, BF16, D, 3.5, 0.0)
    s = L.log_probs(x, w, y)
    want = exactly(x, w, y, 1.0)
    check_scores(s._asdict(), want, T, V)


@TYPES
@pytest.mark.parametrize("T,V,D", [(20, 9000, 2048), (128, 3001, 1000),
                                   (300, 20000, 1100), (1300, 2500, 1536)])
def test_gradients(T, V, D, dtype):
    x, w, y, gen = operands(T, V, D, dtype, T + 1, 2.0)
    a = torch.randn(T, generator=gen, device=DEV)
    b = 0.1 * torch.randn(T, generator=gen, device=DEV)
    s = L.log_probs(x, w, y, keep=True)
    want = exactly(x, w, y, 1.0)
    check_scores(s._asdict(), want, T, V)
    g = -want["p"] * (a.double()[:, None] + b.double()[:, None] * (
        want["log_p"] + want["entropy"][:, None]))
    g[torch.arange(T, device=DEV), y] += a.double()
    u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -11
    most = (1 if T <= 128 else 2) * u / math.sqrt(3.0) + 2e-5
    dx, dw = L.log_probs_grad(x, w, y, s, a, b)
    for got, exact in ((dx, g @ w.double()), (dw, g.t() @ x.double())):
        err = float((got.double() - exact).norm() / exact.norm())
        assert err <= most, err
    assert G.device_status() == 0
