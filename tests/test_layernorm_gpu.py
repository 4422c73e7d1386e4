"""Layer norm on the GPU: forward and backward against 64 bits."""
import math

import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import EPS32, TINY, TORCH, UNIT, Guarded, assert_within, generator, randn

pytestmark = pytest.mark.gpu

# binary32 steps between the inputs and a sum: at most 40 terms a thread, 10 levels of the tree, and a few single
# operations
STEPS = 64 * EPS32

# rows, cols, pad, offset: one element, less and more than a lane's 8, a warp's 256 columns from both sides, rows that
# start anywhere (runs of 8 that begin before the row, one tile more than the columns take), padded rows, one, two and
# four tiles a thread, many rows of one warp, more rows than blocks, rows too wide to hold
SHAPES = [(1, 1, 0, 0), (3, 7, 0, 0), (9, 3, 0, 5), (2, 8, 0, 0), (5, 255, 0, 0), (4, 256, 8, 0), (4, 257, 0, 0),
          (17, 256, 3, 7), (3, 1000, 0, 1), (2, 1001, 7, 3), (7, 5120, 0, 0), (2, 8192, 64, 8), (2, 8199, 0, 0),
          (3, 4096, 1, 2), (1, 16384, 0, 0), (2, 16390, 0, 0), (5, 16380, 3, 6), (700, 64, 0, 0), (701, 300, 4, 0),
          (700, 61, 0, 3), (650, 2048, 0, 0), (620, 4096, 0, 0), (613, 5001, 0, 0), (1, 40003, 0, 0), (3, 33001, 0, 3),
          (640, 1801, 0, 0), (3, 12480, 0, 0), (700, 9001, 0, 0), (613, 9344, 0, 0), (611, 12288, 8, 0), (700, 16384, 0, 0),
          (620, 16377, 0, 3), (3, 128, 0, 0), (1003, 64, 64, 0), (9999, 56, 0, 0), (9999, 100, 4, 0), (10001, 128, 0, 8),
          (9999, 250, 6, 0), (10000, 136, 0, 0), (5, 8, 0, 3), (9999, 57, 0, 0), (20001, 121, 0, 1), (10001, 101, 2, 0),
          (9999, 249, 0, 3)]


def make(rows, cols, dtype, pad, offset, seed, spread=1.0, at=0.0):
    return Guarded(rows, cols, TORCH[dtype], pad, offset, (randn((rows, cols), seed, torch.float32, spread) + at).to(TORCH[dtype]))


class Want:
    """The formula in 64 bits, and how far binary32 may be from it: a difference is off by a rounding of the sum h, two
    of its own and the mean's, the squares by theirs and the differences'."""

    def __init__(self, x, res, w, b, eps):
        self.h = x.double() + (res.double() if res is not None else 0.0)
        self.mean = self.h.mean(1)
        d = self.h - self.mean[:, None]
        var = (d * d).mean(1)
        self.rstd = 1.0 / torch.sqrt(var + eps)
        w = w.double() if w is not None else torch.ones_like(d[0])
        b = b.double() if b is not None else torch.zeros_like(d[0])
        self.y = d * self.rstd[:, None] * w + b
        away = (self.h - self.h[:, :1]).abs()
        off = EPS32 * (self.h.abs() + self.h[:, :1].abs() + 2 * away) + STEPS * away.mean(1, keepdim=True)
        self.mean_off = EPS32 * self.mean.abs() + off.mean(1)
        self.rstd_off = STEPS + ((d.abs() * off).mean(1) + (off * off).mean(1)) / (var + eps)  # of itself
        self.y_off = (self.rstd[:, None] * w.abs() * (off + d.abs() * (self.rstd_off[:, None] + 4 * EPS32))
                      + 2 * EPS32 * (self.y.abs() + b.abs()))


def check_forward(got, x, res, w, b, eps, dtype):
    y, h, mean, rstd = got
    want = Want(x, res, w, b, eps)
    u, tiny = UNIT[dtype], TINY[dtype]
    assert_within(h, want.h, (u + EPS32) * want.h.abs() + tiny, "h")
    assert_within(mean, want.mean, want.mean_off, "mean")
    assert_within(rstd, want.rstd, want.rstd_off * want.rstd, "rstd")
    assert_within(y, want.y, u * want.y.abs() + (1 + u) * want.y_off + tiny, "y")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_forward(dtype, rows, cols, pad, offset):
    x, r = make(rows, cols, dtype, pad, offset, 1), make(rows, cols, dtype, pad, offset, 2, 3.0, 0.5)
    y, h = (Guarded(rows, cols, TORCH[dtype], pad, offset) for _ in range(2))
    kind = TORCH[dtype] if rows % 2 else torch.float32
    w, b = randn((cols,), 3, kind), randn((cols,), 4, kind)
    got = ew.ew_layernorm(x.t, w, b, residual=r.t, y=y.t, h=h.t)
    assert got[0] is y.t and got[1] is h.t
    check_forward(got, x.t, r.t, w, b, 1e-5, dtype)
    assert all(m.intact() for m in (x, r, y, h))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [1001, 2048, 20001])
@pytest.mark.parametrize("places", [(0, 1, 0, 0), (3, 3, 3, 2), (1, 1, 4, 1), (5, 5, 5, 5)])
def test_matrices_whose_rows_lie_apart(dtype, cols, places):
    x, r = (make(5, cols, dtype, 0, o, 5 + k) for k, o in enumerate(places[:2]))
    y, h = (Guarded(5, cols, TORCH[dtype], 8 * k, o) for k, o in enumerate(places[2:]))
    w = Guarded(1, cols, TORCH[dtype], 0, places[0], randn((1, cols), 7, TORCH[dtype]))  # a weight that starts anywhere
    b = Guarded(1, cols, TORCH[dtype], 0, places[1] + 1, randn((1, cols), 8, TORCH[dtype]))
    got = ew.ew_layernorm(x.t, w.t[0], b.t[0], residual=r.t, y=y.t, h=h.t)
    check_forward(got, x.t, r.t, w.t[0], b.t[0], 1e-5, dtype)
    assert all(m.intact() for m in (x, r, y, h, w, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [96, 1001, 20000])
@pytest.mark.parametrize("given", ["", "w", "b"])
def test_no_residual(dtype, cols, given):
    x = make(3, cols, dtype, 0, 0, 9)
    w = randn((cols,), 10, TORCH[dtype]) if given == "w" else None
    b = randn((cols,), 11, torch.float32) if given == "b" else None
    got = ew.ew_layernorm(x.t, w, b, eps=0.0)
    assert got[1] is x.t
    check_forward(got, x.t, None, w, b, 0.0, dtype)


@pytest.mark.parametrize("cols", [61, 64, 201, 1003, 4096, 12000, 12001, 20001])
@pytest.mark.parametrize("at", [1e3, -1e6])
def test_mean_far_from_zero(cols, at):
    """Rows of spread 1 around a mean of up to 1e6: the elements hold the spread to 2^-5, and y loses no more."""
    x = make(5, cols, "f32", 0, 0, 12, 1.0, at)
    got = ew.ew_layernorm(x.t, None)
    want = Want(x.t, None, None, None, 1e-5)
    check_forward(got, x.t, None, None, None, 1e-5, "f32")
    # differences within a factor of two are exact, so nothing here grows with the mean
    assert float((got[0].double() - want.y).abs().max()) < 200 * EPS32 * float(want.y.abs().max() + 4)


@pytest.mark.parametrize("cols", [61, 64, 201, 1003, 12000, 12001, 20001])
def test_constant_and_outlying_rows(cols):
    x = torch.full((4, cols), 1234.567, device="cuda")
    x[1] = 0.0
    x[2] = randn((cols,), 13)
    x[2, 0] = 1e4  # the first element, which the others are compared with
    x[3] = randn((cols,), 14)
    x[3, cols // 2] = -1e6
    b = randn((cols,), 15)
    got = ew.ew_layernorm(x, None, b)
    assert torch.equal(got[0][:2], b.expand(2, cols))  # no spread: the bias alone
    assert torch.equal(got[2][:2], x[:2, 0])
    check_forward(got, x, None, None, b, 1e-5, "f32")


@pytest.mark.parametrize("cols", [57, 64, 121, 249, 320, 321, 12000, 12001, 20001])
def test_nan_and_infinity(cols):
    x = randn((4, cols), 16)
    x[0, 5], x[1, 0], x[2, cols - 1] = math.nan, math.inf, -math.inf
    y, _, _, rstd = ew.ew_layernorm(x, None)
    assert torch.isnan(y[:3]).all() and torch.isnan(rstd[:3]).all()
    assert torch.isfinite(y[3]).all() and torch.isfinite(rstd[3])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("rows,cols", [(5, 512), (5, 1003), (700, 40), (5, 33000), (3, 33001), (700, 9001), (700, 16000), (10003, 128), (10003, 192), (20003, 101), (30003, 50)])
@pytest.mark.parametrize("form", ["y=x,h=residual", "y=residual,h=x", "h=x", "y=x"])
def test_in_place(dtype, rows, cols, form):
    x, r = make(rows, cols, dtype, 0, 0, 17), make(rows, cols, dtype, 0, 0, 18)
    w = randn((cols,), 19, TORCH[dtype])
    want = ew.ew_layernorm(x.t.clone(), w, w, residual=r.t.clone())
    places = {"x": x.t, "residual": r.t}
    given = dict(part.split("=") for part in form.split(","))
    got = ew.ew_layernorm(x.t, w, w, residual=r.t, **{k: places[v] for k, v in given.items()})
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert x.intact() and r.intact()


def test_in_place_without_a_residual_h_is_a_copy():
    x = randn((7, 512), 20)
    before = x.clone()
    y, h, _, _ = ew.ew_layernorm(x, None, y=x)
    assert y is x and h is not x and torch.equal(h, before)


# ---------------------------------------------------------------- backward

def grads(dy, h, w, mean, rstd, dh):
    r = rstd.double()[:, None]
    n = (h.double() - mean.double()[:, None]) * r
    dy = dy.double()
    g = dy * (w.double() if w is not None else 1.0)
    dx = r * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True)) + (dh.double() if dh is not None else 0.0)
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + n.abs() * (g * n).abs().mean(1, keepdim=True))
    size = size + (dh.double().abs() if dh is not None else 0.0)
    return dx, size, (dy * n).sum(0), (dy * n).abs().sum(0), dy.sum(0), dy.abs().sum(0)


def statistics(h):
    mean = h.float().mean(1)
    return mean, torch.rsqrt((h.float() - mean[:, None]).square().mean(1) + 1e-5)


def check_backward(got, dy, h, w, mean, rstd, dh, dtype):
    dx, dw, db = got
    want, size, want_w, size_w, want_b, size_b = grads(dy, h, w, mean, rstd, dh)
    assert_within(dx, want, UNIT[dtype] * want.abs() + 80 * EPS32 * size + TINY[dtype], "dx")
    rows = dy.shape[0]
    assert_within(dw, want_w, (rows + 16) * EPS32 * size_w, "dweight")
    assert_within(db, want_b, (rows + 16) * EPS32 * size_b, "dbias")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES + [(3000, 96, 0, 0), (1300, 1000, 0, 0), (3001, 97, 0, 5),
                                                           (1301, 1003, 2, 1), (1400, 2049, 0, 0), (400, 8187, 0, 0),
                                                           (170, 12001, 0, 3), (400, 10240, 0, 0), (200, 16384, 8, 8),
                                                           (700, 400, 0, 0), (701, 509, 0, 0), (5000, 2041, 0, 0),
                                                           (10927, 248, 8, 0), (20003, 32, 0, 8), (9, 192, 0, 0)])
def test_backward(dtype, rows, cols, pad, offset):
    dy, h, dh = (make(rows, cols, dtype, pad, offset, k, s, m) for k, s, m in ((21, 1.0, 0.0), (22, 2.0, 0.7), (23, 0.5, 0.0)))
    w = randn((cols,), 24, TORCH[dtype] if rows % 2 else torch.float32)
    mean, rstd = statistics(h.t)
    given_dh = None if rows % 3 == 0 else dh.t
    dx, dw, db = Guarded(rows, cols, TORCH[dtype], pad, offset), Guarded(1, cols, torch.float32), Guarded(1, cols, torch.float32)
    ew.ew_layernorm_grad(dy.t, h.t, w, mean, rstd, dh=given_dh, dx=dx.t, dweight=dw.t.view(-1), dbias=db.t.view(-1))
    check_backward((dx.t, dw.t[0], db.t[0]), dy.t, h.t, w, mean, rstd, given_dh, dtype)
    assert all(m.intact() for m in (dy, h, dh, dx, dw, db))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(40, 1001), (700, 2048), (5, 20001)])
@pytest.mark.parametrize("places", [(0, 1, 0, 0), (3, 3, 3, 2), (1, 1, 4, 1), (5, 5, 5, 5)])
def test_backward_of_matrices_whose_rows_lie_apart(dtype, rows, cols, places):
    dy, h, dh = (make(rows, cols, dtype, 8 * k, o, 25 + k) for k, o in enumerate(places[:3]))
    dx = Guarded(rows, cols, TORCH[dtype], 0, places[3])
    w = Guarded(1, cols, TORCH[dtype], 0, 3, randn((1, cols), 28, TORCH[dtype]))
    mean, rstd = statistics(h.t)
    got = ew.ew_layernorm_grad(dy.t, h.t, w.t[0], mean, rstd, dh=dh.t, dx=dx.t)
    check_backward(got, dy.t, h.t, w.t[0], mean, rstd, dh.t, dtype)
    assert all(m.intact() for m in (dy, h, dh, dx, w))


@pytest.mark.parametrize("cols", [56, 64, 203, 300, 1003, 9000, 9001, 20001])
def test_backward_of_constant_rows_far_out(cols):
    """m r is past binary32, and no column of the row has it: dx = r (g - mean(g)), dweight = 0."""
    m, r = 2e36, 316.0
    h, dy = torch.full((5, cols), m, device="cuda"), randn((5, cols), 31)
    mean, rstd = (torch.full((5,), v, device="cuda") for v in (m, r))
    mean.copy_(h[:, 0])
    got = ew.ew_layernorm_grad(dy, h, None, mean, rstd)
    check_backward(got, dy, h, None, mean, rstd, None, "f32")
    assert not got[1].any()


@pytest.mark.parametrize("rows,cols", [(9, 64), (10003, 120), (10003, 101), (5003, 256), (9, 1003), (1300, 1003), (9, 8192), (200, 9001), (90, 16000), (9, 33001)])
@pytest.mark.parametrize("place", ["dy", "dh"])
def test_backward_in_place(rows, cols, place):
    dy, h, dh = (make(rows, cols, "bf16", 0, 0, k) for k in (29, 30, 31))
    mean, rstd = statistics(h.t)
    want = ew.ew_layernorm_grad(dy.t.clone(), h.t, None, mean, rstd, dh=dh.t.clone())
    got = ew.ew_layernorm_grad(dy.t, h.t, None, mean, rstd, dh=dh.t, dx={"dy": dy.t, "dh": dh.t}[place])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_backward_against_differences():
    """The gradient of sum(dy * y) + sum(dh * h) by central differences in 64 bits.  A step of 1e-5 leaves a truncation
    of about 1e-10 and a rounding of about 1e-11; the kernel adds binary32's own."""
    rows, cols, eps = 3, 37, 1e-3
    x, res, w, b = randn((rows, cols), 32), randn((rows, cols), 33), randn((cols,), 34), randn((cols,), 35)
    dy, dh = randn((rows, cols), 36), randn((rows, cols), 37)
    _, h, mean, rstd = ew.ew_layernorm(x, w, b, residual=res, eps=eps)
    got = ew.ew_layernorm_grad(dy, h, w, mean, rstd, dh=dh)

    def loss(x64, w64, b64):
        want = Want(x64, res, w64, b64, eps)
        return float((dy.double() * want.y).sum() + (dh.double() * want.h).sum())

    for by, d in enumerate(got):
        for k in range(0, d.numel(), 5):
            values = []
            for step in (1e-5, -1e-5):
                at = [x.double(), w.double(), b.double()]
                at[by] = at[by].clone()
                at[by].view(-1)[k] += step
                values.append(loss(*at))
            assert abs((values[0] - values[1]) / 2e-5 - float(d.view(-1)[k])) < 2e-5


@pytest.mark.parametrize("rows,cols", [(0, 40), (5, 40), (1300, 264), (3, 33000)])
def test_c_entry_leaves_out_what_is_null(rows, cols):
    """mean, rstd, h, dweight and dbias may each be null; a sum alone has the same bits as with the other."""
    L, stream = ew.lib(), torch.cuda.current_stream().cuda_stream
    x, dy = randn((rows, cols), 38), randn((rows, cols), 39)
    y = torch.empty_like(x)
    assert L.ew_layernorm(0, x.data_ptr(), cols, None, 0, 0, None, None, 1e-5, y.data_ptr(), cols, None, 0, None, None, rows,
                          cols, stream) == 0
    want_y, h, mean, rstd = ew.ew_layernorm(x, None)
    assert torch.equal(y, want_y)
    dx, dw, db = ew.ew_layernorm_grad(dy, h, None, mean, rstd)
    size = L.ew_layernorm_grad_workspace(rows, cols)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    for given in ((1, 0), (0, 1), (0, 0)):
        out = [torch.full((cols,), 7.0, device="cuda") for _ in range(2)]
        got = torch.empty_like(dx)
        p = [o.data_ptr() if g else None for o, g in zip(out, given)]
        assert L.ew_layernorm_grad(0, dy.data_ptr(), cols, h.data_ptr(), cols, 0, None, mean.data_ptr(), rstd.data_ptr(), None,
                                   0, got.data_ptr(), cols, p[0], p[1], rows, cols,
                                   work.data_ptr() if any(given) else None, size if any(given) else 0, stream) == 0
        assert torch.equal(got, dx)
        for o, g, want in zip(out, given, (dw, db)):
            assert torch.equal(o, want if g else torch.full_like(o, 7.0))
    if rows == 0:
        assert not dw.any() and not db.any()


def test_no_rows():
    x = torch.empty(0, 40, device="cuda")
    y, h, mean, rstd = ew.ew_layernorm(x, None)
    assert y.shape == (0, 40) and rstd.shape == (0,) and mean.shape == (0,)
    dw, db = torch.full((40,), 7.0, device="cuda"), torch.full((40,), 7.0, device="cuda")
    dx, _, _ = ew.ew_layernorm_grad(x, x, None, mean, rstd, dweight=dw, dbias=db)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()


@pytest.mark.parametrize("cols", [1024, 1001])
def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph(cols):
    dy, h = randn((3000, cols), 40, torch.bfloat16), randn((3000, cols), 41, torch.bfloat16)
    mean, rstd = statistics(h)
    want = ew.ew_layernorm_grad(dy, h, None, mean, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = ew.ew_layernorm_grad(dy, h, None, mean, rstd, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two captured calls of other inputs, each with its own workspace, replayed side by side
    graphs, outs, ins = [], [], []
    for k in range(2):
        x = randn((3000, cols), 42 + k, torch.bfloat16)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, hk, m, r = ew.ew_layernorm(x, None, residual=h)
            outs.append((y, hk, m, r, *ew.ew_layernorm_grad(dy, hk, None, m, r, dh=h)))
        graphs.append(g)
        ins.append(x)
    for k, x in enumerate(ins):
        x.copy_(randn(x.shape, 50 + k, torch.bfloat16))
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    for x, out in zip(ins, outs):
        y, hk, m, r = ew.ew_layernorm(x, None, residual=h)
        again = (y, hk, m, r, *ew.ew_layernorm_grad(dy, hk, None, m, r, dh=h))
        assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_more_than_2_to_the_31_elements():
    """Offsets past 32 bits: the last rows of a matrix of 4.4 billion bytes of bf16."""
    rows, cols = 270000, 8192
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=generator(44))
    y, h, mean, rstd = ew.ew_layernorm(x, None, y=x.clone())
    for a in (0, rows - 3):
        check_forward((y[a:a + 3], h[a:a + 3], mean[a:a + 3], rstd[a:a + 3]), x[a:a + 3], None, None, None, 1e-5, "bf16")
    dy = {a: y[a:a + 3].clone() for a in (0, rows - 3)}
    dx, dw, db = ew.ew_layernorm_grad(y, x, None, mean, rstd, dx=y)
    for a in (0, rows - 3):
        want, size, *_ = grads(dy[a], x[a:a + 3], None, mean[a:a + 3], rstd[a:a + 3], None)
        assert_within(dx[a:a + 3], want, UNIT["bf16"] * want.abs() + 80 * EPS32 * size, "dx")
    assert torch.isfinite(dw).all() and torch.isfinite(db).all()


def test_refusals():
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    s = torch.zeros(4, device="cuda")
    for call, error in ((lambda: ew.ew_layernorm(x.double(), w), TypeError), (lambda: ew.ew_layernorm(x.cpu(), w), ValueError),
                        (lambda: ew.ew_layernorm(x.t(), w), ValueError), (lambda: ew.ew_layernorm(x, w[:63]), ValueError),
                        (lambda: ew.ew_layernorm(x, w, w[:63]), ValueError), (lambda: ew.ew_layernorm(x, w.half()), TypeError),
                        (lambda: ew.ew_layernorm(x.half(), w.half(), w), TypeError),
                        (lambda: ew.ew_layernorm(x, w, residual=x[:, :32]), ValueError),
                        (lambda: ew.ew_layernorm(x, w, mean=s[:3]), ValueError),
                        (lambda: ew.ew_layernorm_grad(x, x, w, s, w), ValueError),
                        (lambda: ew.ew_layernorm_grad(x, x, w, w, s), ValueError),
                        (lambda: ew.ew_layernorm_grad(x, x.half(), w, s, s), ValueError)):
        with pytest.raises(error):
            call()
    with pytest.raises(ew.EwError, match="INVALID"):
        ew.ew_layernorm(x, w, eps=-1.0)
    with pytest.raises(ew.EwError, match="OVERLAP"):
        ew.ew_layernorm(x[:3], w, y=x[1:])
    with pytest.raises(ew.EwError, match="OVERLAP"):
        ew.ew_layernorm(x, w, mean=s, rstd=s)
    with pytest.raises(ew.EwError, match="OVERLAP"):
        ew.ew_layernorm_grad(x, torch.ones_like(x), w, s, s, dx=x, dweight=w)
