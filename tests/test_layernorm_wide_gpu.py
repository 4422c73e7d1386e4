"""Layer norm of many rows around the width that a block holds (64 tiles of 256 columns), on both sides of it."""
import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import TORCH, Guarded, randn
from tests.test_layernorm_gpu import check_backward, check_forward, make, statistics

pytestmark = pytest.mark.gpu

# rows, cols, pad, offset: more than 4 rows an SM; 64 tiles where rows start anywhere, the first column beyond, 65 and
# more, past 128 tiles, and aligned rows of as many
SHAPES = [(620, 16377, 0, 3), (620, 16378, 0, 3), (700, 16385, 0, 0), (640, 20001, 0, 0), (613, 50257, 0, 0),
          (620, 16384, 8, 0), (640, 20000, 0, 0)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_forward(dtype, rows, cols, pad, offset):
    x, r = make(rows, cols, dtype, pad, offset, 1), make(rows, cols, dtype, pad, offset, 2, 3.0, 0.5)
    y, h = (Guarded(rows, cols, TORCH[dtype], pad, offset) for _ in range(2))
    w, b = randn((cols,), 3), randn((cols,), 4)
    got = ew.ew_layernorm(x.t, w, b, residual=r.t, y=y.t, h=h.t)
    check_forward(got, x.t, r.t, w, b, 1e-5, dtype)
    assert all(m.intact() for m in (x, r, y, h))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [16384, 20000])
@pytest.mark.parametrize("given", ["weight", "bias"])
def test_aligned_rows_and_a_vector_that_starts_anywhere(dtype, cols, given):
    x = make(640, cols, dtype, 0, 0, 5)
    v = Guarded(1, cols, TORCH[dtype], 0, 3, randn((1, cols), 6, TORCH[dtype]))
    w, b = (v.t[0], None) if given == "weight" else (None, v.t[0])
    check_forward(ew.ew_layernorm(x.t, w, b), x.t, None, w, b, 1e-5, dtype)
    assert x.intact() and v.intact()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("form", ["y=x,h=residual", "y=residual,h=x"])
def test_in_place(dtype, form):
    rows, cols = 640, 20001
    x, r = make(rows, cols, dtype, 0, 0, 7), make(rows, cols, dtype, 0, 0, 8)
    want = ew.ew_layernorm(x.t.clone(), None, residual=r.t.clone())
    places = {"x": x.t, "residual": r.t}
    got = ew.ew_layernorm(x.t, None, residual=r.t, **{k: places[v] for k, v in (part.split("=") for part in form.split(","))})
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert x.intact() and r.intact()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [16378, 20000, 20001])
def test_backward(dtype, cols):
    dy, h, dh = (make(640, cols, dtype, 0, 0, k) for k in (9, 10, 11))
    w = randn((cols,), 12)
    mean, rstd = statistics(h.t)
    got = ew.ew_layernorm_grad(dy.t, h.t, w, mean, rstd, dh=dh.t)
    check_backward(got, dy.t, h.t, w, mean, rstd, dh.t, dtype)
