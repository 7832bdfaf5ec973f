"""dw and dbias of the norm's backward are two arrays: sums written over each other are refused, on the CPU, before
any device work (the pointers are never dereferenced)."""

import ctypes

import pytest

from orthogonal_reparameterized_cnp_amd import binding as B

MB = 1 << 20


@pytest.mark.parametrize("T", [0, 4])
@pytest.mark.parametrize("off", [0, 4, -4, 63 * 4, -63 * 4])
def test_gradients_that_share_a_cell(T, off):
    dsc = B.norm_desc(64, "layer", "bf16")
    st = B.lib().poetx_norm_bwd(ctypes.byref(dsc), T, MB, 64, 2 * MB, 64, 3 * MB, 4 * MB, None, 64, 5 * MB, 64, 6 * MB,
                                6 * MB + off, 7 * MB, 1 << 30, None)
    assert st == B.POETX_E_SHAPE and "dbias" in B.poetx_last_error()
