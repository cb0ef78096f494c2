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
