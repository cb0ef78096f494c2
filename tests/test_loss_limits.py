"""The largest sizes that the vocabulary losses take: host logic only."""

from __future__ import annotations

import pytest

from test_abi import built_lib  # noqa: F401  (builds the library)
from test_loss_refusals import NO, ce, ce_grad

MOST = 2**31 - 2**20


@pytest.mark.parametrize("name", ["T", "V", "D"])
def test_sizes_past_the_limit_are_unsupported(built_lib, name):  # noqa: F811
    """Rows and columns are counted in 32 bits, past the end of the matrix
    too: the sizes at which that would overflow are refused by every entry."""
    from dense_fp32_matrix_02_gb300 import gemm
    lib = gemm.lib()
    for n in (MOST + 1, 2**31 - 1, 2**31):
        sizes = {"T": 4, "V": 8, "D": 8, name: n}
        wide = {"ldx": sizes["D"], "ldw": sizes["D"]}
        assert ce(lib, **sizes, **wide) == NO, n
        assert ce_grad(lib, **sizes, **wide, lddx=sizes["D"],
                       lddw=sizes["D"]) == NO, n
        for grad in (0, 1):
            assert lib.gemm_f32_vocab_workspace_size(
                sizes["T"], sizes["V"], sizes["D"], 1, grad, 1) == -NO, n
    sizes = {"T": 4, "V": 8, "D": 8, name: MOST}
    for grad in (0, 1):
        assert lib.gemm_f32_vocab_workspace_size(
            sizes["T"], sizes["V"], sizes["D"], 1, grad, 1) > 0


def test_workspace_bytes_do_not_overflow(built_lib):  # noqa: F811
    """Operands of more than 2^48 elements are refused: their bytes of
    workspace, 2^64 and more, came out as small or negative numbers."""
    from dense_fp32_matrix_02_gb300 import gemm
    size = gemm.lib().gemm_f32_vocab_workspace_size
    for T, V, D in ((MOST, MOST, MOST), (MOST, 8, MOST), (8, MOST, MOST),
                    (2**30, 8, 2**19), (8, 2**30, 2**19)):
        for grad in (0, 1):
            for aligned in (0, 1):
                assert size(T, V, D, 256, grad, aligned) == -NO, (T, V, D)
        wide = {"ldx": D, "ldw": D}
        assert ce(gemm.lib(), T=T, V=V, D=D, n=2**62, **wide) == NO
        assert ce_grad(gemm.lib(), T=T, V=V, D=D, n=2**62, **wide, lddx=D,
                       lddw=D) == NO
    # the largest that are left: at least X's copy, W's and the targets'
    for T, V, D in ((2**30, 8, 2**18), (8, 2**30, 2**18), (MOST, MOST, 2**16),
                    (MOST, MOST, 1)):
        for grad in (0, 1):
            got = size(T, V, D, 256, grad, 0)
            assert 2 * (T + V) * D + 8 * T * 256 < got < 2**60, (T, V, D)


@pytest.mark.parametrize("T,V,D,top,most", [
    (8192, 1000, 512, 16, 100), (777, 9973, 521, 5, 130), (2, 5, 7, 1, 1),
    (300, 700, 96, 64, 2), (8192, 32000, 768, 1, 700)])
def test_workspace_holds_what_is_written(built_lib, T, V, D, top,  # noqa: F811
                                         most):
    """The gradients' workspace in MB: one buffer of G where the vocabulary
    is one piece, and no more fp32 slots than the steps of a tile of dX and
    the depth of dW can be cut into (it was 31 to 882 MB for these)."""
    from dense_fp32_matrix_02_gb300 import gemm
    assert gemm.lib().gemm_f32_vocab_workspace_size(
        T, V, D, top, 1, 1) <= most * 1_000_000


@pytest.mark.parametrize("T,V,D,top", [
    (1, 1, 1, 1), (300, 900, 72, 1), (2, 5, 7, 256), (2**20, 128000, 64, 1),
    (8192, 1000, 512, 16), (0, 100, 8, 1)])
def test_gradients_workspace_serves_the_forward_call(built_lib,  # noqa: F811
                                                     T, V, D, top):
    from dense_fp32_matrix_02_gb300 import gemm
    size = gemm.lib().gemm_f32_vocab_workspace_size
    for aligned in (0, 1):
        assert size(T, V, D, top, 1, aligned) >= size(T, V, D, top, 0, aligned)


def test_workspaces_that_hold_less_than_they_count(built_lib):  # noqa: F811
    """An expanded tensor counts elements that it has no memory for."""
    torch = pytest.importorskip("torch")
    from dense_fp32_matrix_02_gb300 import loss as L
    host, head = torch.device("cpu"), (0, 4, 8, 8)
    with pytest.raises(ValueError, match="contiguous"):
        L._scratch(torch.empty(1, dtype=torch.uint8).expand(1 << 20), head, 1,
                   0, 1, host, None)
    with pytest.raises(ValueError, match="contiguous"):
        L._scratch(torch.empty(1 << 10, 2, dtype=torch.uint8)[:, 0], head, 1,
                   0, 1, host, None)
    with pytest.raises(TypeError, match="tensor"):
        L._scratch(bytearray(1 << 20), head, 1, 0, 1, host, None)
    ws = torch.empty(64, 4, dtype=torch.float32)
    assert L._scratch(ws, head, 1, 0, 1, host, None) == (ws, ws.data_ptr(),
                                                         1024)
