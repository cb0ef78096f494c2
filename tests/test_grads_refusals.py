"""What the global norm and clipping refuse: host logic only."""

from __future__ import annotations

import array
import math

import pytest

from test_abi import built_lib  # noqa: F401  (builds the library)

BAD, NO = 1, 2
P = 256  # an aligned address that is never read: the checks come first


def call(clip=True, data=P, out=P, rows=2, cols=4, ld=4, ld_out=4, type_=0,
         n=1, table=True, max_norm=1.0, norm=P, ws=P, size=0):
    """The status of a call that is refused: its workspace is too small
    where nothing else is wrong."""
    from dense_fp32_matrix_02_gb300 import gemm
    lib = gemm.lib()
    t = array.array("q", (data, out, rows, cols, ld, ld_out, type_))
    at = t.buffer_info()[0] if table else None
    if clip:
        return lib.gemm_f32_grad_clip(n, at, max_norm, norm, ws, size, None)
    return lib.gemm_f32_grad_norm(n, at, norm, ws, size, None)


def test_refusals(built_lib):  # noqa: F811
    for clip in (True, False):
        for bad in (dict(type_=3), dict(type_=-1), dict(rows=-1),
                    dict(cols=-1), dict(ld=3), dict(data=0), dict(data=P + 1),
                    dict(type_=2, data=P + 2), dict(n=-1), dict(table=False),
                    dict(norm=None), dict(ws=None), dict(size=-1),
                    dict(ws=P + 8, size=1 << 20)):
            assert call(clip, **bad) == BAD, bad
        for big in (dict(rows=2**31, cols=1, ld=1, ld_out=1),
                    dict(rows=2, cols=2**31, ld=2**31, ld_out=2**31),
                    dict(rows=1, cols=2**48 + 1),
                    dict(rows=2**20, ld=2**40, ld_out=2**40),
                    dict(n=2**31)):
            assert call(clip, **big) == NO, big
    for bad in (dict(out=0), dict(out=P + 1), dict(ld_out=3),
                dict(max_norm=-1.0), dict(max_norm=math.nan)):
        assert call(True, **bad) == BAD, bad
    # nothing is needed of a gradient without elements (the workspace is)
    assert call(True, data=0, out=0, rows=0, ld=0, ld_out=0) == BAD


def test_one_place_for_two_gradients(built_lib):  # noqa: F811
    from dense_fp32_matrix_02_gb300 import gemm
    lib = gemm.lib()
    one = (P, P, 1, 4, 4, 4, 0)
    for other in (one, (2 * P, P, 3, 5, 5, 5, 0)):
        t = array.array("q", one + (4 * P, 4 * P, 1, 1, 1, 1, 2) + other)
        assert lib.gemm_f32_grad_clip(3, t.buffer_info()[0], 1.0, P, P,
                                      1 << 20, None) == BAD


def test_workspace_size(built_lib):  # noqa: F811
    from dense_fp32_matrix_02_gb300 import gemm
    size = gemm.lib().gemm_f32_grad_workspace_size
    assert size(-1) == -BAD and size(2**31) == -NO
    assert 0 < size(0) == size(1) == size(520) < size(521) < size(2**31 - 1)


def test_binding_refusals(built_lib):  # noqa: F811
    torch = pytest.importorskip("torch")
    from dense_fp32_matrix_02_gb300 import grads as C
    with pytest.raises(ValueError, match="CUDA"):
        C.global_norm([torch.zeros(4)])
    with pytest.raises(TypeError):
        C.global_norm([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(TypeError):
        C.clip_([3.0], 1.0)
    with pytest.raises(ValueError, match="no gradients"):
        C.global_norm([])
