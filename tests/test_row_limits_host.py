"""Limits of the row operators that need no GPU."""
import os

import pytest

import memory_bound_elementwise_gb300 as ew

pytestmark = pytest.mark.skipif(not os.path.exists(ew.LIB_PATH), reason="libew.so not built")

MOST = 2 ** 31 - 2 ** 16


@pytest.mark.parametrize("rows,cols,fits", [(MOST, 32768, True), (MOST, 32800, False), (32768, MOST, True), (MOST, MOST, False),
                                            (0, MOST, True), (1, MOST, True)])
def test_embedding_gradient_size(rows, cols, fits):
    """rows x cols up to 2^46: past it the call is refused before anything is launched."""
    need = ew.lib().ew_embed_grad_workspace(1000, rows, cols)
    assert (need >= 0) == fits
    if not fits:
        status = ew.lib().ew_embed_grad(ew.EW_F16, 0, 256, cols, 256, 1.0, ew.EW_F16, 256, 1000, cols, rows, cols, 0, 256,
                                        2 ** 62, None)
        assert ew.STATUS_NAMES[status] == "EW_ERR_INVALID_VALUE"
