"""RMS norm on the GPU: forward, 8-bit output and backward against 64 bits."""
import math

import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import EPS32, TINY, TORCH, UNIT, Guarded, assert_within, generator, randn

pytestmark = pytest.mark.gpu

# binary32 steps between the inputs and a result, before its last rounding: at
# most 40 terms a thread, 10 levels of the tree, and a few single operations
STEPS = 64 * EPS32

# rows, cols, pad, offset: one element, less and more than a lane's 8, a warp's
# 256 columns from both sides, rows that start anywhere, padded rows, one, two
# and four tiles a thread, many rows of one warp, rows too wide to hold
SHAPES = [(1, 1, 0, 0), (3, 7, 0, 0), (2, 8, 0, 0), (5, 255, 0, 0), (4, 256, 8, 0), (4, 257, 0, 0), (3, 1000, 0, 1),
          (2, 1001, 7, 3), (7, 5120, 0, 0), (2, 8192, 64, 8), (2, 8199, 0, 0), (1, 16384, 0, 0), (2, 16390, 0, 0),
          (700, 64, 0, 0), (701, 300, 4, 0), (650, 2048, 0, 0), (620, 4096, 0, 0), (613, 5000, 0, 0), (1, 40003, 0, 0),
          (2, 33000, 0, 0)]


def make(rows, cols, dtype, pad, offset, seed, spread=1.0):
    return Guarded(rows, cols, TORCH[dtype], pad, offset, randn((rows, cols), seed, TORCH[dtype], spread))


def expected(x, res, w, eps):
    h = x.double() + (res.double() if res is not None else 0.0)
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None] * (w.double() if w is not None else 1.0)
    return y, h, rstd


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_forward(dtype, rows, cols, pad, offset):
    x, r = make(rows, cols, dtype, pad, offset, 1), make(rows, cols, dtype, pad, offset, 2, 3.0)
    y, h = (Guarded(rows, cols, TORCH[dtype], pad, offset) for _ in range(2))
    w = randn((cols,), 3, TORCH[dtype] if rows % 2 else torch.float32)
    got_y, got_h, rstd = ew.ew_rmsnorm(x.t, w, residual=r.t, y=y.t, h=h.t)
    assert got_y is y.t and got_h is h.t
    want_y, want_h, want_r = expected(x.t, r.t, w, 1e-6)
    u, tiny = UNIT[dtype], TINY[dtype]
    assert_within(h.t, want_h, (u + EPS32) * want_h.abs() + tiny, "h")
    assert_within(rstd, want_r, STEPS * want_r, "rstd")
    assert_within(y.t, want_y, (u + STEPS) * want_y.abs() + tiny, "y")
    assert all(m.intact() for m in (x, r, y, h))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [96, 1001, 20000])
def test_no_residual_no_weight(dtype, cols):
    x = make(3, cols, dtype, 0, 0, 4)
    y, h, rstd = ew.ew_rmsnorm(x.t, None, eps=0.0)
    assert h is x.t
    want_y, _, want_r = expected(x.t, None, None, 0.0)
    assert_within(rstd, want_r, STEPS * want_r, "rstd")
    assert_within(y, want_y, (UNIT[dtype] + STEPS) * want_y.abs() + TINY[dtype], "y")


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("cols", [512, 1003, 33000])
@pytest.mark.parametrize("form", ["y=x,h=residual", "y=residual,h=x", "h=x", "y=x"])
def test_in_place(dtype, cols, form):
    x, r = make(5, cols, dtype, 0, 0, 5), make(5, cols, dtype, 0, 0, 6)
    w = randn((cols,), 7, TORCH[dtype])
    want_y, want_h, _ = ew.ew_rmsnorm(x.t.clone(), w, residual=r.t.clone())
    places = {"x": x.t, "residual": r.t}
    given = dict(part.split("=") for part in form.split(","))
    y, h, _ = ew.ew_rmsnorm(x.t, w, residual=r.t, **{k: places[v] for k, v in given.items()})
    assert torch.equal(y, want_y) and torch.equal(h, want_h)
    assert x.intact() and r.intact()


def e4m3_half_step(v):
    """Half the distance of neighbouring e4m3 numbers around v (3 mantissa bits, least exponent -6)."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))) * 2.0 ** -4


@pytest.mark.parametrize("out", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("rows,cols,pad,offset",
                         [(1, 1, 0, 0), (3, 100, 0, 0), (4, 512, 8, 0), (3, 1000, 0, 1), (2, 777, 0, 0), (650, 520, 0, 0),
                          (2, 5120, 0, 0), (1, 16500, 0, 0), (1, 16501, 0, 0)])
def test_quant(out, dtype, group, rows, cols, pad, offset):
    x, r = make(rows, cols, dtype, pad, offset, 8), make(rows, cols, dtype, pad, offset, 9, 3.0)
    w = randn((cols,), 10, TORCH[dtype])
    if cols > 300:
        x.t[0, 256:320], r.t[0, 256:320] = 0.0, 0.0  # whole groups of zeros
    groups = -(-cols // group) if group else 1
    q, h = Guarded(rows, cols, out, pad, offset), Guarded(rows, cols, TORCH[dtype], pad, offset)
    scales = Guarded(rows, groups, torch.float32, pad)
    _, _, _, rstd = ew.ew_rmsnorm_quant(x.t, w, residual=r.t, group=group, q=q.t, scales=scales.t, h=h.t)
    y, want_h, want_r = expected(x.t, r.t, w, 1e-6)
    assert_within(h.t, want_h, (UNIT[dtype] + EPS32) * want_h.abs() + TINY[dtype], "h")
    assert_within(rstd, want_r, STEPS * want_r, "rstd")
    top = 127.0 if out == torch.int8 else 448.0
    parts = y.abs().split(group or cols, 1)
    want_s = torch.stack([p.amax(1) for p in parts], 1).clamp(min=2.0 ** -100) / top
    assert_within(scales.t, want_s, (STEPS + EPS32) * want_s, "scales")
    v = y / want_s.repeat_interleave(group or cols, 1)[:, :cols]
    step = torch.full_like(v, 0.5) if out == torch.int8 else e4m3_half_step(v)
    assert_within(q.t.double(), v, step * (1 + 2 * STEPS) + 4 * STEPS * v.abs(), "q")
    assert all(m.intact() for m in (x, r, q, h, scales))


@pytest.mark.parametrize("cols", [320, 321])
def test_quant_nan_infinity_and_zero_rows(cols):
    x = torch.zeros(4, cols, device="cuda")
    x[1, 5], x[2, 5] = math.nan, math.inf
    x[3] = 1e-30
    q, scales, _, rstd = ew.ew_rmsnorm_quant(x, None, group=64, eps=1e-6)
    assert torch.equal(scales[0], torch.full_like(scales[0], 2.0 ** -100) / 448.0) and not q[0].float().any()
    assert torch.isnan(scales[1]).all() and torch.isnan(q[1].float()).all()
    # infinity: rstd is 0, so the others are 0 and the infinity's own place 0 * inf
    assert rstd[2] == 0 and torch.isnan(scales[2, 0]) and not torch.isnan(scales[2, 1:]).any()
    # tiny values keep their scale: y = 1e-27 is above the floor of 2^-100
    assert_within(q[3].float() * scales[3, 0], torch.full((cols,), 1e-27, device="cuda").double(), 1e-32, "tiny")


def grads(dy, h, w, rstd, dh):
    n = h.double() * rstd.double()[:, None]
    g = dy.double() * (w.double() if w is not None else 1.0)
    c = (g * n).mean(1, keepdim=True)
    r = rstd.double()[:, None]
    dx = r * (g - n * c) + (dh.double() if dh is not None else 0.0)
    size = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True)) + (dh.double().abs() if dh is not None else 0.0)
    return dx, size, (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES + [(3000, 96, 0, 0), (1300, 1000, 0, 0)])
def test_backward(dtype, rows, cols, pad, offset):
    dy, h, dh = (make(rows, cols, dtype, pad, offset, k, s) for k, s in ((11, 1.0), (12, 2.0), (13, 0.5)))
    w = randn((cols,), 14, TORCH[dtype] if rows % 2 else torch.float32)
    rstd = torch.rsqrt(h.t.float().square().mean(1) + 1e-6)
    given_dh = None if rows % 3 == 0 else dh.t
    dx, dw = Guarded(rows, cols, TORCH[dtype], pad, offset), Guarded(1, cols, torch.float32)
    ew.ew_rmsnorm_grad(dy.t, h.t, w, rstd, dh=given_dh, dx=dx.t, dweight=dw.t.view(-1))
    want, size, want_w, size_w = grads(dy.t, h.t, w, rstd, given_dh)
    assert_within(dx.t, want, UNIT[dtype] * want.abs() + 80 * EPS32 * size + TINY[dtype], "dx")
    assert_within(dw.t[0], want_w, (rows + 16) * EPS32 * size_w, "dweight")
    assert all(m.intact() for m in (dy, h, dh, dx, dw))


@pytest.mark.parametrize("cols", [64, 1003, 8192, 33001])
@pytest.mark.parametrize("place", ["dy", "dh"])
def test_backward_in_place(cols, place):
    dy, h, dh = (make(9, cols, "bf16", 0, 0, k) for k in (15, 16, 17))
    rstd = torch.rsqrt(h.t.float().square().mean(1))
    want, want_w = ew.ew_rmsnorm_grad(dy.t.clone(), h.t, None, rstd, dh=dh.t.clone())
    dx, dw = ew.ew_rmsnorm_grad(dy.t, h.t, None, rstd, dh=dh.t, dx={"dy": dy.t, "dh": dh.t}[place])
    assert torch.equal(dx, want) and torch.equal(dw, want_w)


def test_backward_against_differences():
    """The gradient of sum(dy * y) + sum(dh * h) by central differences in 64 bits.  A step of 1e-5 leaves a
    truncation of about 1e-10 and a rounding of about 1e-11; the kernel adds binary32's own."""
    rows, cols, eps = 3, 37, 1e-3
    x, res, w = randn((rows, cols), 18), randn((rows, cols), 19), randn((cols,), 20)
    dy, dh = randn((rows, cols), 21), randn((rows, cols), 22)
    _, h, rstd = ew.ew_rmsnorm(x, w, residual=res, eps=eps)
    dx, dw = ew.ew_rmsnorm_grad(dy, h, w, rstd, dh=dh)

    def loss(x64, w64):
        y, h64, _ = expected(x64, res, w64, eps)
        return float((dy.double() * y).sum() + (dh.double() * h64).sum())

    for got, at, by in ((dx, x, 0), (dw, w, 1)):
        for k in range(0, at.numel(), 5):
            values = []
            for step in (1e-5, -1e-5):
                moved = at.double().clone()
                moved.view(-1)[k] += step
                values.append(loss(moved, w.double()) if by == 0 else loss(x.double(), moved))
            assert abs((values[0] - values[1]) / 2e-5 - float(got.view(-1)[k])) < 2e-5


def test_no_rows():
    x = torch.empty(0, 40, device="cuda")
    y, h, rstd = ew.ew_rmsnorm(x, None)
    assert y.shape == (0, 40) and rstd.shape == (0,)
    q, scales, _, _ = ew.ew_rmsnorm_quant(x, None, group=32)
    assert q.shape == (0, 40) and scales.shape == (0, 2)
    dw = torch.full((40,), 7.0, device="cuda")
    dx, _ = ew.ew_rmsnorm_grad(x, x, None, rstd, dweight=dw)
    assert dx.shape == (0, 40) and not dw.any()


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    dy, h = randn((3000, 1024), 23, torch.bfloat16), randn((3000, 1024), 24, torch.bfloat16)
    rstd = torch.rsqrt(h.float().square().mean(1))
    want = ew.ew_rmsnorm_grad(dy, h, None, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = ew.ew_rmsnorm_grad(dy, h, None, rstd, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, _, r = ew.ew_rmsnorm(dy, None, residual=h)
        dx, dw = ew.ew_rmsnorm_grad(dy, y, None, r)
    dy.copy_(randn(dy.shape, 25, torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    y2, _, r2 = ew.ew_rmsnorm(dy, None, residual=h)
    dx2, dw2 = ew.ew_rmsnorm_grad(dy, y2, None, r2)
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_more_than_2_to_the_31_elements():
    """Offsets past 32 bits: the last rows of a matrix of 4.4 billion bytes of bf16."""
    rows, cols = 270000, 8192
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=generator(26))
    y, _, rstd = ew.ew_rmsnorm(x, None, y=x.clone())
    for a in (0, rows - 3):
        want, _, _ = expected(x[a:a + 3], None, None, 1e-6)
        assert_within(y[a:a + 3], want, (UNIT["bf16"] + STEPS) * want.abs(), "rows from %d" % a)


def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(TypeError):
        ew.ew_rmsnorm(x.double(), w)
    with pytest.raises(ValueError):
        ew.ew_rmsnorm(x.cpu(), w)
    with pytest.raises(ValueError):
        ew.ew_rmsnorm(x.t(), w)
    with pytest.raises(ValueError):
        ew.ew_rmsnorm(x, w[:63])
    with pytest.raises(TypeError):
        ew.ew_rmsnorm(x, w.half())
    with pytest.raises(ValueError):
        ew.ew_rmsnorm(x, w, residual=x[:, :32])
    with pytest.raises(ValueError):
        ew.ew_rmsnorm(x, w, residual=x.half())
    with pytest.raises(ew.EwError, match="INVALID"):
        ew.ew_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(ew.EwError, match="OVERLAP"):
        ew.ew_rmsnorm(x[:3], w, y=x[1:])
    with pytest.raises(ew.EwError, match="INVALID"):
        ew.ew_rmsnorm_quant(x, w, group=48)
    with pytest.raises(TypeError):
        ew.ew_rmsnorm_quant(x, w, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ew.ew_rmsnorm_grad(x, x, w, w)
