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
