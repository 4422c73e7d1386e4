"""The norm in place, and the backward call from what it returns."""
import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import TORCH, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 64), (5, 1001), (3, 20000), (700, 256)])
def test_h_is_kept_where_y_takes_its_place(dtype, rows, cols):
    x, w, dy = randn((rows, cols), 81, TORCH[dtype]), randn((cols,), 82), randn((rows, cols), 83, TORCH[dtype])
    before = x.clone()
    y, h, rstd = ew.ew_rmsnorm(x.clone(), w)
    place = x.clone()
    y2, h2, rstd2 = ew.ew_rmsnorm(place, w, y=place)
    assert y2 is place and torch.equal(y2, y) and torch.equal(rstd2, rstd)
    assert torch.equal(h2, before) and h2.data_ptr() != place.data_ptr()
    want, got = ew.ew_rmsnorm_grad(dy, h, w, rstd), ew.ew_rmsnorm_grad(dy, h2, w, rstd2)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_h_is_x_where_nothing_overwrites_it():
    x, w = randn((4, 96), 84), randn((96,), 85)
    assert ew.ew_rmsnorm(x, w)[1] is x
    assert ew.ew_rmsnorm(x, w, y=torch.empty_like(x))[1] is x
    assert ew.ew_rmsnorm_quant(x, w)[2] is x
    r = x.clone()
    y, h, _ = ew.ew_rmsnorm(x, w, residual=r, y=x)  # with a residual h is a tensor of its own
    assert y is x and torch.equal(h, r + r)
    y, h, _ = ew.ew_rmsnorm(r.clone(), w, h=r)
    assert h is r
    none = x[:0]
    assert ew.ew_rmsnorm(none, w, y=none)[1].shape == (0, 96)


def test_y_that_does_not_fit():
    x, w = randn((4, 96), 86), randn((96,), 87)
    with pytest.raises(TypeError):
        ew.ew_rmsnorm(x, w, y=3.0)
    with pytest.raises(ValueError):
        ew.ew_rmsnorm(x, w, y=x[:2])
    with pytest.raises(ValueError):
        ew.ew_rmsnorm(x, w, y=x.half())
