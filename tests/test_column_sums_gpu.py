"""The sums of columns behind both norms' backward calls: one vector or two in a launch, in the same order."""
import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import EPS32, assert_within, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(9, 12000), (1, 300), (40, 1001), (700, 2048), (1300, 33)])
def test_one_vector_and_two(rows, cols):
    """rstd 1 and mean 0 make the layer norm's n, like the norm's, h itself: then dweight is the same sum in both, up to
    the order of a block's rows, and each norm's is the same with its other results wanted or not."""
    dy, h = randn((rows, cols), 1), randn((rows, cols), 2)
    one, zero = torch.ones(rows, device="cuda"), torch.zeros(rows, device="cuda")
    _, norm = ew.ew_rmsnorm_grad(dy, h, None, one)
    _, dw, db = ew.ew_layernorm_grad(dy, h, None, zero, one)
    want, size = (dy.double() * h.double()).sum(0), (dy.double() * h.double()).abs().sum(0)
    assert_within(norm, want, (rows + 16) * EPS32 * size, "the norm's dweight")
    assert_within(dw, want, (rows + 16) * EPS32 * size, "dweight")
    assert_within(db, dy.double().sum(0), (rows + 16) * EPS32 * dy.double().abs().sum(0), "dbias")
    L, stream = ew.lib(), torch.cuda.current_stream().cuda_stream
    size = L.ew_layernorm_grad_workspace(rows, cols)
    work, dx, alone = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty_like(dy), torch.empty_like(db)
    assert L.ew_layernorm_grad(0, dy.data_ptr(), cols, h.data_ptr(), cols, 0, None, zero.data_ptr(), one.data_ptr(), None, 0,
                               dx.data_ptr(), cols, None, alone.data_ptr(), rows, cols, work.data_ptr(), size, stream) == 0
    assert torch.equal(alone, db)  # the second vector alone: the first one's blocks leave
