"""What the log probabilities refuse, and what they need: host logic only."""

from __future__ import annotations

import math

import pytest

from test_abi import built_lib  # noqa: F401  (builds the library)

BAD, OK, NO = 1, 0, 2
P = 256  # an aligned address that is never read: the checks come first
MOST = 2**31 - 2**20


def score(lib, type_=0, T=4, V=8, D=8, X=P, ldx=8, W=P, ldw=8, ids=P, tau=1.0,
          top=0, logp=P, lse=P, entropy=P, tl=P, ti=P, kept=None, kn=0, ws=P,
          n=1 << 40):
    return lib.gemm_f32_vocab_score(type_, T, V, D, X, ldx, W, ldw, ids, tau,
                                    top, logp, lse, entropy, tl, ti, kept, kn,
                                    ws, n, None)


def grad(lib, T=4, V=8, D=8, ldx=8, ldw=8, ids=P, tau=1.0, lse=P, entropy=P,
         kept=P, kn=1 << 40, a=P, sa=1, b=P, sb=1, dX=P, lddx=8, dW=P, lddw=8,
         ws=P, n=1 << 40):
    return lib.gemm_f32_vocab_score_grad(
        0, T, V, D, P, ldx, P, ldw, ids, tau, lse, entropy, kept, kn, a, sa, b,
        sb, dX, lddx, dW, lddw, ws, n, None)


def test_forward_refusals(built_lib):  # noqa: F811
    from dense_fp32_matrix_02_gb300 import gemm
    lib = gemm.lib()
    for bad in (dict(type_=2), dict(type_=-1), dict(T=-1), dict(V=0),
                dict(D=0), dict(ldx=7), dict(ldw=7), dict(X=None),
                dict(W=None), dict(ids=None), dict(logp=None), dict(lse=None),
                dict(entropy=None), dict(tau=0.0), dict(tau=math.nan),
                dict(tau=math.inf), dict(top=-1), dict(top=9),
                dict(V=1000, top=257), dict(top=1, tl=None),
                dict(top=1, ti=None), dict(kept=P, kn=4 * 8 * 4 - 1),
                dict(kept=P + 8, kn=1 << 20), dict(kn=-1), dict(ws=None),
                dict(n=-1), dict(n=0), dict(ws=P + 8)):
        assert score(lib, **bad) == BAD, bad
    assert score(lib, T=0, X=None, ids=None, logp=None, lse=None, entropy=None,
                 ws=None, n=0) == OK


def test_gradient_refusals(built_lib):  # noqa: F811
    from dense_fp32_matrix_02_gb300 import gemm
    lib = gemm.lib()
    for bad in (dict(lse=None), dict(entropy=None), dict(kept=None),
                dict(kn=100), dict(kept=P + 4), dict(a=None), dict(sa=-1),
                dict(sb=-1), dict(dX=None), dict(dW=None), dict(lddx=7),
                dict(lddw=7), dict(ids=None), dict(tau=0.0), dict(ws=None),
                dict(n=16), dict(V=0)):
        assert grad(lib, **bad) == BAD, bad
    assert grad(lib, T=0, dW=None) == BAD  # dW = 0 is still written


@pytest.mark.parametrize("name", ["T", "V", "D"])
def test_sizes_past_the_limit(built_lib, name):  # noqa: F811
    from dense_fp32_matrix_02_gb300 import gemm
    lib = gemm.lib()
    size = lib.gemm_f32_vocab_score_workspace_size
    for n in (MOST + 1, 2**31):
        sizes = {"T": 4, "V": 8, "D": 8, name: n}
        wide = {"ldx": sizes["D"], "ldw": sizes["D"]}
        assert score(lib, **sizes, **wide) == NO
        assert grad(lib, **sizes, **wide, lddx=sizes["D"], lddw=sizes["D"],
                    kn=2**62) == NO
        assert size(sizes["T"], sizes["V"], sizes["D"], 0, 0, 0, 1) == -NO
    sizes = {"T": 4, "V": 8, "D": 8, name: MOST}
    for keep in (0, 1):
        for g in (0, 1):
            for top in (0, 8):
                got = size(sizes["T"], sizes["V"], sizes["D"], top, keep, g, 0)
                assert 0 < got < 2**50


def test_sizes(built_lib):  # noqa: F811
    from dense_fp32_matrix_02_gb300 import gemm
    lib = gemm.lib()
    size = lib.gemm_f32_vocab_score_workspace_size
    kept = lib.gemm_f32_vocab_score_kept_size
    assert kept(4, 9, 8, 1) == 4 * 16 * 4 and kept(0, 5, 8, 1) == 0
    assert kept(5, 9, 8, 1) == 512  # (a copy of W would start behind it)
    assert kept(4, 9, 9, 0) == 4 * 16 * 4 + 9 * 16 * 2  # with a copy of W
    assert kept(-1, 5, 8, 1) == -BAD and kept(4, 0, 8, 1) == -BAD
    assert kept(4, 5, 0, 1) == -BAD and kept(4, 5, 8, 2) == -BAD
    assert kept(2**31, 5, 8, 1) == -NO and kept(MOST, MOST, 1, 1) == -NO
    for bad in ((-1, 8, 8, 0, 0, 0, 1), (4, 0, 8, 0, 0, 0, 1),
                (4, 8, 0, 0, 0, 0, 1), (4, 8, 8, -1, 0, 0, 1),
                (4, 8, 8, 9, 0, 0, 1), (4, 999, 8, 257, 0, 0, 1),
                (4, 8, 8, 0, 2, 0, 1), (4, 8, 8, 0, 0, 2, 1),
                (4, 8, 8, 0, 0, 0, 2)):
        assert size(*bad) == -BAD, bad
    # the logits in the workspace: 4 GB at most, or 256 tokens' of them
    few = size(16384, 128000, 64, 0, 0, 0, 1)
    assert size(16384, 128000, 64, 5, 1, 0, 1) == few
    assert few < size(16384, 128000, 64, 5, 0, 0, 1) <= few + 2**32
    wide = size(8192, 2**23, 64, 5, 0, 0, 1) - size(8192, 2**23, 64, 0, 0, 0, 1)
    assert wide == 256 * 2**23 * 4
    for T, V in ((1, 1), (300, 900), (0, 100), (8192, 1000)):
        for al in (0, 1):
            assert size(T, V, 72, 1, 1, 1, al) >= size(T, V, 72, 1, 1, 0, al)


def test_binding_refusals(built_lib):  # noqa: F811
    torch = pytest.importorskip("torch")
    from dense_fp32_matrix_02_gb300 import loss as L
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    y = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        L.log_probs(x, x, y)
    with pytest.raises(TypeError):
        L.log_probs(x.float(), x.float(), y)
