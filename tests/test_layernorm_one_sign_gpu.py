"""Layer norm of rows whose elements have one sign and a few of which stand out: as precise as a plain sum.

The bound does not know what the kernel compares elements with.  Let u = 2^-24 and A = mean(|h|).  A kernel that subtracts
some number L from the elements before it sums them, |L - mean| at most |mean|, is off by
    u |h| for h, u |h - L| for the difference, summed in 64 steps of u and multiplied: at most (64 + 4) u mean |h - L|,
and mean |h - L| <= A + 2 |mean| <= 3 A.  Parts of a row that have L of their own are joined in the same way, 8 steps of u of
at most 4 A.  That is 256 u A for the mean, and u (|h| + 2 |h - mean| + |mean|) more for one difference to it.
"""
import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import EPS32, TINY, TORCH, UNIT, Guarded, assert_within, randn
from tests.test_layernorm_gpu import STEPS

pytestmark = pytest.mark.gpu


def check(got, x, res, w, b, eps, dtype):
    y, h, mean, rstd = got
    want_h = x.double() + (res.double() if res is not None else 0.0)
    m = want_h.mean(1, keepdim=True)
    d = want_h - m
    var = (d * d).mean(1)
    want_r = 1.0 / torch.sqrt(var + eps)
    w, b = (v.double() if v is not None else k * torch.ones_like(d[0]) for v, k in ((w, 1.0), (b, 0.0)))
    want = d * want_r[:, None] * w + b
    mean_off = 256 * EPS32 * want_h.abs().mean(1, keepdim=True)
    off = EPS32 * (want_h.abs() + 2 * d.abs() + m.abs()) + mean_off
    rstd_off = STEPS + ((d.abs() * off).mean(1) + (off * off).mean(1)) / (var + eps)  # of itself
    y_off = want_r[:, None] * w.abs() * (off + d.abs() * (rstd_off[:, None] + 4 * EPS32)) + 2 * EPS32 * (want.abs() + b.abs())
    u, tiny = UNIT[dtype], TINY[dtype]
    assert_within(h, want_h, (u + EPS32) * want_h.abs() + tiny, "h")
    assert_within(mean, m[:, 0], mean_off[:, 0] + EPS32 * m[:, 0].abs(), "mean")
    assert_within(rstd, want_r, rstd_off * want_r, "rstd")
    assert_within(y, want, u * want.abs() + (1 + u) * y_off + tiny, "y")


# Columns that stand out, of a row of `cols`: the first, the first lane's, the lanes' first ones in a tile, the lanes of a
# tile moved by single elements, a tile, the last, and all but every 64th.
PLACES = {"first": lambda c: c == 0, "lane": lambda c: c < 8, "lanes": lambda c: (c % 8 == 0) & (c < 256),
          "singles": lambda c: c < 32, "tile": lambda c: c < 256, "last": lambda c: c == c[-1],
          "most": lambda c: c % 64 != 7}


def rows_of(rows, cols, dtype, place, size, pad=0, offset=0, sign=1.0):
    x = randn((rows, cols), 1).abs() + 0.01
    x[:, PLACES[place](torch.arange(cols, device="cuda"))] *= size
    return Guarded(rows, cols, TORCH[dtype], pad, offset, (sign * x).to(TORCH[dtype]))


# several rows to a warp by 8, 16 and 32 lanes, aligned and not; a warp a row; 1, 2 and 4 tiles a thread; blocks that walk;
# clusters of two blocks; rows too wide to hold; and, by padding that moves every row, rows by single elements
SHAPES = [(9, 64, 0, 0), (9999, 56, 0, 0), (9999, 57, 0, 0), (1003, 128, 0, 0), (10003, 121, 0, 1), (10000, 192, 0, 0),
          (10003, 249, 0, 3), (5, 201, 0, 0), (9, 1003, 0, 0), (9, 5120, 0, 0), (700, 4001, 0, 0), (700, 4096, 0, 0),
          (620, 16384, 0, 0), (3, 12480, 0, 0), (3, 12001, 0, 0), (700, 9001, 0, 0), (5, 33000, 0, 0), (5, 33001, 0, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("place", list(PLACES))
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_elements_that_stand_out(dtype, place, rows, cols, pad, offset):
    x = rows_of(rows, cols, dtype, place, 1e6, pad, offset, -1.0 if cols % 3 == 0 else 1.0)
    b = randn((cols,), 2)
    check(ew.ew_layernorm(x.t, None, b), x.t, None, None, b, 1e-5, dtype)


@pytest.mark.parametrize("place", list(PLACES))
@pytest.mark.parametrize("cols", [56, 57, 300, 1003, 4096, 12001, 20001])
def test_with_a_residual(place, cols):
    """16-bit matrices whose binary32 sum stands out."""
    x, r = rows_of(5, cols, "f16", place, 1e4), Guarded(5, cols, torch.float16, 0, 0, randn((5, cols), 3).abs().half())
    w = randn((cols,), 4)
    check(ew.ew_layernorm(x.t, w, None, residual=r.t), x.t, r.t, w, None, 1e-5, "f16")


@pytest.mark.parametrize("place", list(PLACES))
@pytest.mark.parametrize("cols", [61, 1003, 4096, 20001])
def test_rows_that_lie_apart(place, cols):
    x = rows_of(5, cols, "f32", place, 1e6)
    y = Guarded(5, cols, torch.float32, 0, 1)
    check(ew.ew_layernorm(x.t, None, y=y.t, h=torch.empty_like(x.t)), x.t, None, None, None, 1e-5, "f32")
    assert y.intact()


@pytest.mark.parametrize("cols", [56, 57, 201, 4096, 12001, 20001])
@pytest.mark.parametrize("at", [1e30, -3.0])
def test_rows_of_one_value_keep_it(cols, at):
    x = torch.full((5, cols), at, device="cuda")
    x[1] *= 3.0
    b = randn((cols,), 5)
    y, _, mean, rstd = ew.ew_layernorm(x, None, b)
    assert torch.equal(y, b.expand(5, cols)) and torch.equal(mean, x[:, 0])
    assert torch.equal(rstd, torch.full_like(rstd, 1e-5).rsqrt()) or float((rstd * 1e-5 ** 0.5 - 1).abs().max()) < 6 * EPS32


@pytest.mark.parametrize("cols", [56, 57, 201, 1003, 4096, 12001, 20001])
def test_a_row_does_not_depend_on_those_beside_it(cols):
    """The same bits beside rows of which something stands out as beside others: rows change places by eights, and so
    start as they did between multiples of 8 elements."""
    x = randn((24, cols), 6)
    x[8:] = x[8:].abs() + 0.01
    x[16:, 0], x[20, cols // 2] = 1e5, 1e6
    places = torch.arange(24, device="cuda").view(3, 8).clone()
    for k in range(8):
        places[:, k] = places[:, k].roll(k % 3)
    places = places.view(-1)
    want, got = ew.ew_layernorm(x, None), ew.ew_layernorm(x[places], None)
    for k in (0, 2, 3):
        assert torch.equal(got[k], want[k][places])


@pytest.mark.parametrize("cols", [56, 57, 201, 1003, 4096, 12001, 20001])
def test_variance_past_binary32(cols):
    """Elements that binary32 holds, but not their squares, of both signs and of one: rstd 0 and y the bias."""
    x = torch.full((2, cols), 2e30, device="cuda")
    x[0, ::2] = -2e30
    x[1, 3] = 1e25
    b = randn((cols,), 7)
    y, _, _, rstd = ew.ew_layernorm(x, None, b)
    assert not rstd.any() and torch.equal(y, b.expand(2, cols))
