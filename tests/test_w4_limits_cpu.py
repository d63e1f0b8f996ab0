"""Refusals of 4-bit products beyond what their kernels count. No GPU."""
import ctypes

import pytest

from fine_grained_sparse_fp32_b200 import _build, kmoe

A = ctypes.c_void_p(1 << 20)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kmoe.load()


def test_rows_whose_cost_does_not_fit_are_refused(lib):
    """8192 columns with groups of 32: two tokens a unit at a cost of 4, so 2^30 rows make 2^31."""
    w = kmoe._W4Struct(A.value, A.value, None, 32)
    P = 1 << 30
    assert kmoe.moe_linear_w4_workspace_size(4, P, 1, 8192, group=32, y_dtype=kmoe.torch.float32) == 0
    st = lib.moe_linear_w4(A, 1, 4, P, 1, 8192, 1, A, None, ctypes.byref(w), A, 0, None, 0, None)
    assert st == kmoe.KMOE_ERR_UNSUPPORTED and b"rows" in lib.moe_last_error()
