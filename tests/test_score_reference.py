"""The float64 reference of the log probabilities, on the CPU: its gradients
against autograd's and against differences of its values."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import score_reference as ref  # noqa: E402


def case(T=5, V=11, D=7):
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(T, D, generator=gen, dtype=torch.float64)
    w = torch.randn(V, D, generator=gen, dtype=torch.float64)
    ids = torch.randint(0, V, (T,), generator=gen)
    ids[1] = -1
    a = torch.randn(T, generator=gen, dtype=torch.float64)
    b = torch.randn(T, generator=gen, dtype=torch.float64)
    return x, w, ids, a, b


def loss(x, w, ids, a, b, tau):
    s = ref.scores(x, w, ids, tau)
    return (a * s["logp"] + b * s["entropy"]).sum()


@pytest.mark.parametrize("tau", [1.0, 0.7, 2.0])
def test_gradients_are_autograds(tau):
    x, w, ids, a, b = case()
    x.requires_grad_(), w.requires_grad_()
    loss(x, w, ids, a, b, tau).backward()
    got = ref.gradients(x.detach(), w.detach(), ids, a, b, tau)
    assert torch.allclose(got["dx"], x.grad, rtol=0, atol=1e-12)
    assert torch.allclose(got["dw"], w.grad, rtol=0, atol=1e-12)


def test_gradients_are_differences():
    x, w, ids, a, b = case()
    got = ref.gradients(x, w, ids, a, b, 1.3)
    gen = torch.Generator().manual_seed(2)
    for name, m in (("dx", x), ("dw", w)):
        way = torch.randn(m.shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        ends = []
        for sign in (h, -h):
            xs, ws = (x + sign * way, w) if m is x else (x, w + sign * way)
            ends.append(loss(xs, ws, ids, a, b, 1.3))
        slope = (ends[0] - ends[1]) / (2 * h)
        assert abs(float(slope - (got[name] * way).sum())) < 1e-8


def test_top_and_unscored():
    x, w, ids, _, _ = case()
    w[4] = w[9]  # equal logits: the lower id first
    s = ref.scores(x, w, ids, 1.0, 11)
    assert s["top_ids"][1].tolist() == [-1] * 11
    assert float(s["logp"][1]) == 0.0
    for t in (0, 2, 3, 4):
        order = s["top_ids"][t].tolist()
        assert sorted(order) == list(range(11))
        assert order.index(9) == order.index(4) + 1
