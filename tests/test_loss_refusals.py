"""What the vocabulary losses refuse, and what they need: host logic only."""

from __future__ import annotations

import math

import pytest

from test_abi import built_lib  # noqa: F401  (builds the library)

torch = pytest.importorskip("torch")

BAD, OK, NO = 1, 0, 2
P = 256  # an aligned address that is never read: the checks come first


def ce(lib, type_=0, T=4, V=8, D=8, X=P, ldx=8, W=P, ldw=8, y=P, loss=P,
       lse=P, ws=P, n=1 << 30):
    return lib.gemm_f32_vocab_ce(type_, T, V, D, X, ldx, W, ldw, y, loss, lse,
                                 ws, n, None)


def ce_grad(lib, T=4, V=8, D=8, ldx=8, ldw=8, y=P, lse=P, g=P, gs=1, dX=P,
            lddx=8, dW=P, lddw=8, ws=P, n=1 << 30):
    return lib.gemm_f32_vocab_ce_grad(0, T, V, D, P, ldx, P, ldw, y, lse, g,
                                      gs, dX, lddx, dW, lddw, ws, n, None)


def kd(lib, top=2, u=P, ldt=2, ids=P, ldi=2, tau=1.0, n=1 << 30):
    return lib.gemm_f32_vocab_distill(0, 4, 8, 8, P, 8, P, 8, top, u, ldt,
                                      ids, ldi, tau, P, P, P, n, None)


def kd_grad(lib, top=2, tau=1.0, g=P):
    return lib.gemm_f32_vocab_distill_grad(0, 4, 8, 8, P, 8, P, 8, top, P, 2,
                                           P, 2, tau, P, g, 1, P, 8, P, 8, P,
                                           1 << 30, None)


def test_forward_refusals(built_lib):  # noqa: F811
    from dense_fp32_matrix_02_gb300 import gemm
    lib = gemm.lib()
    for bad in (dict(type_=2), dict(type_=-1), dict(T=-1), dict(V=0),
                dict(D=0), dict(ldx=7), dict(ldw=7), dict(X=None),
                dict(W=None), dict(y=None), dict(loss=None), dict(lse=None),
                dict(ws=None), dict(n=-1), dict(n=0), dict(ws=P + 8)):
        assert ce(lib, **bad) == BAD, bad
    assert ce(lib, T=1 << 31) == NO
    assert ce(lib, V=1 << 31) == NO
    # no tokens: nothing to do, nothing needed but W
    assert ce(lib, T=0, X=None, y=None, loss=None, lse=None, ws=None,
              n=0) == OK
    for bad in (dict(top=0), dict(top=257), dict(ldt=1), dict(ldi=1),
                dict(u=None), dict(ids=None), dict(tau=0.0), dict(tau=-1.0),
                dict(tau=math.inf), dict(tau=math.nan), dict(tau=1e-45)):
        assert kd(lib, **bad) == BAD, bad


def test_gradient_refusals(built_lib):  # noqa: F811
    from dense_fp32_matrix_02_gb300 import gemm
    lib = gemm.lib()
    for bad in (dict(lse=None), dict(g=None), dict(gs=-1), dict(dX=None),
                dict(dW=None), dict(lddx=7), dict(lddw=7), dict(y=None),
                dict(V=0), dict(ws=None), dict(n=16)):
        assert ce_grad(lib, **bad) == BAD, bad
    assert ce_grad(lib, T=0, dW=None) == BAD  # dW = 0 is still written
    for bad in (dict(top=0), dict(tau=0.0), dict(g=None)):
        assert kd_grad(lib, **bad) == BAD, bad


def test_binding_refusals(built_lib):  # noqa: F811
    from dense_fp32_matrix_02_gb300 import loss as L
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    y = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):  # host tensors
        L.cross_entropy(x, x, y)
    with pytest.raises(TypeError):  # 32-bit operands
        L.cross_entropy(x.float(), x.float(), y)
    with pytest.raises(ValueError, match="2-D"):
        L.cross_entropy(x[0], x, y)


def test_workspace_sizes_refuse(built_lib):  # noqa: F811
    from dense_fp32_matrix_02_gb300 import gemm
    lib = gemm.lib()
    size = lib.gemm_f32_vocab_workspace_size
    assert size(-1, 8, 8, 1, 0, 1) == -BAD
    assert size(4, 0, 8, 1, 0, 1) == -BAD
    assert size(4, 8, 0, 1, 0, 1) == -BAD
    assert size(4, 8, 8, 0, 0, 1) == -BAD
    assert size(4, 8, 8, 257, 0, 1) == -BAD
    assert size(4, 8, 8, 1, 2, 1) == -BAD
    assert size(4, 8, 8, 1, 0, 2) == -BAD
    assert size(1 << 31, 8, 8, 1, 0, 1) == -NO
