"""Tokens sorted by expert and back on the GPU: the sort against lists, the moved rows bit for bit, sums against 64 bits."""
import math

import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import EPS32, TINY, TORCH, UNIT, Guarded, assert_within, generator, randn

pytestmark = pytest.mark.gpu


def choices(n, k, experts, seed, missing=0.1, skew=2.0):
    """Experts of n tokens, some popular, some ids outside the range, some named twice."""
    g = generator(seed)
    e = (torch.rand(n, k, generator=g, device="cuda") ** skew * experts).long()
    out = torch.rand(n, k, generator=g, device="cuda")
    e[out < missing] = -1
    e[out > 1 - missing / 2] = experts + 3
    return e


def sorted_by_lists(experts, n_experts, align, capacity):
    of = [[] for _ in range(n_experts)]
    for slot, e in enumerate(experts.reshape(-1).tolist()):
        if 0 <= e < n_experts:
            of[e].append(slot)
    positions, offsets, slots = [-1] * experts.numel(), [0], []
    for rows in of:
        for s in rows:
            positions[s] = len(slots)
            slots.append(s)
        slots += [-1] * (-len(slots) % align)
        offsets.append(len(slots))
    assert len(slots) <= capacity
    return positions, offsets, [len(r) for r in of], slots + [-1] * (capacity - len(slots))


def check_plan(plan, experts, n_experts, align):
    capacity = ew.lib().ew_expert_capacity(*experts.shape, n_experts, align)
    want = sorted_by_lists(experts, n_experts, align, capacity)
    for got, w, name in zip(plan, want, plan._fields):
        assert got.dtype == torch.int32 and got.reshape(-1).tolist() == w, name
    assert plan.positions.shape == experts.shape


# tokens, k, experts, align: single ones, one expert, more experts than slots, a block's slots from both sides, several
# blocks, the most experts
PLANS = [(1, 1, 1, 1), (1, 64, 1000, 16), (3, 2, 5, 1), (7, 8, 128, 128), (64, 8, 128, 16), (300, 1, 1, 8), (500, 4, 3, 7),
         (2048, 1, 100, 1), (2049, 1, 100, 1), (1000, 8, 256, 1), (341, 6, 60, 128), (3000, 64, 1024, 5), (20000, 8, 128, 128),
         (70000, 8, 17, 1), (600000, 1, 1024, 1)]


@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,k,experts,align", PLANS)
def test_sort(itype, n, k, experts, align):
    e = choices(n, k, experts, 1).to(itype)
    check_plan(ew.ew_expert_sort(e, experts, align=align), e, experts, align)


@pytest.mark.parametrize("how", ["none", "one", "last", "huge ids"])
@pytest.mark.parametrize("n", [5, 3000])
def test_sort_of_one_expert_or_none(how, n):
    e = torch.full((n, 3), {"none": -1, "one": 0, "last": 1023, "huge ids": 2 ** 40}[how], device="cuda")
    check_plan(ew.ew_expert_sort(e, 1024, align=64), e, 1024, 64)


def test_sort_of_a_view_of_wider_rows_and_of_top_alternatives():
    wide = choices(900, 12, 40, 2)
    check_plan(ew.ew_expert_sort(wide[:, 3:8], 40), wide[:, 3:8], 40, 1)
    ids = ew.ew_logprob(randn((900, 40), 3), None, top=6).top_ids
    check_plan(ew.ew_expert_sort(ids, 40, align=8), ids, 40, 8)


def test_sort_of_nothing():
    plan = ew.ew_expert_sort(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 9, align=16)
    assert plan.positions.shape == (0, 4) and plan.slots.shape == (0,)
    assert plan.offsets.tolist() == [0] * 10 and plan.counts.tolist() == [0] * 9
    x = torch.empty(0, 33, device="cuda")
    rows = ew.ew_expert_dispatch(x, plan)
    assert rows.shape == (0, 33) and ew.ew_expert_combine(rows, plan).shape == (0, 33)
    dy, dw = ew.ew_expert_combine_grad(x, rows, plan)
    assert dy.shape == (0, 33) and dw.shape == (0, 4)


def test_sort_into_more_rows_than_needed():
    """The C entry with a larger capacity: the rows behind are of no slot; a dispatch of no tokens clears all rows."""
    L, stream = ew.lib(), torch.cuda.current_stream().cuda_stream
    e = choices(50, 2, 6, 4).int()
    p, o, c = torch.empty(50, 2, dtype=torch.int32, device="cuda"), *(torch.empty(m, dtype=torch.int32, device="cuda") for m in (7, 6))
    slots = torch.full((1300,), 77, dtype=torch.int32, device="cuda")
    assert L.ew_expert_sort(0, e.data_ptr(), 2, 6, 1, p.data_ptr(), o.data_ptr(), c.data_ptr(), slots.data_ptr(), 1200, 50, 2,
                            None, 0, stream) == 0
    want = sorted_by_lists(e, 6, 1, 1200)
    assert slots[:1200].tolist() == want[3] and (slots[1200:] == 77).all() and p.reshape(-1).tolist() == want[0]
    out = torch.ones(40, 24, device="cuda")
    gone = torch.full((40,), -1, dtype=torch.int32, device="cuda")
    assert L.ew_expert_dispatch(0, None, 24, None, gone.data_ptr(), out.data_ptr(), 24, 40, 0, 2, 24, stream) == 0
    assert not out.any()


# ---------------------------------------------------------------- rows

# tokens, k, experts, align, cols, pad, offset: one element, less than a lane's 8, tiles from both sides, odd widths (rows
# that start anywhere), padded rows, many slots a token, few and many tokens
ROWS = [(1, 1, 1, 1, 1, 0, 0), (5, 3, 4, 1, 7, 0, 0), (9, 2, 3, 4, 8, 0, 0), (33, 8, 16, 8, 256, 8, 0), (20, 5, 8, 1, 257, 0, 0),
        (17, 33, 40, 16, 264, 0, 0), (6, 64, 100, 1, 100, 3, 1), (300, 8, 32, 128, 1000, 0, 0), (300, 2, 8, 1, 1001, 0, 3),
        (50, 4, 300, 16, 2048, 0, 8), (3, 8, 12, 1, 5003, 5, 2), (2500, 1, 7, 8, 4096, 0, 0), (1500, 6, 64, 16, 2056, 0, 0),
        (700, 2, 5, 3, 8191, 0, 0), (4000, 8, 64, 1, 65, 0, 0), (12, 16, 20, 8, 12000, 0, 0)]


def rows_of(n, cols, dtype, pad, offset, seed):
    return Guarded(n, cols, TORCH[dtype], pad, offset, randn((n, cols), seed, TORCH[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,experts,align,cols,pad,offset", ROWS)
def test_dispatch(dtype, n, k, experts, align, cols, pad, offset):
    plan = ew.ew_expert_sort(choices(n, k, experts, 5), experts, align=align)
    x = rows_of(n, cols, dtype, pad, offset, 6)
    x.t.view(torch.int32 if dtype == "f32" else torch.int16)[0, 0] = -1  # a NaN's bits are moved as they are
    out = Guarded(plan.slots.numel(), cols, TORCH[dtype], pad, offset)
    assert ew.ew_expert_dispatch(x.t, plan, out=out.t) is out.t
    token = plan.slots.long().clamp(min=0) // k
    want = torch.where(plan.slots[:, None] >= 0, x.t[token], torch.zeros_like(x.t[token]))
    bits = torch.int32 if dtype == "f32" else torch.int16
    assert torch.equal(out.t.contiguous().view(bits), want.view(bits))
    assert x.intact() and out.intact()


@pytest.mark.parametrize("weighted", [None, "own", "f32"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,experts,align,cols,pad,offset", ROWS)
def test_combine(dtype, weighted, n, k, experts, align, cols, pad, offset):
    plan = ew.ew_expert_sort(choices(n, k, experts, 7), experts, align=align)
    y = rows_of(plan.slots.numel(), cols, dtype, pad, offset, 8)
    residual = rows_of(n, cols, dtype, pad, offset, 9) if n % 2 else None
    w = randn((n, k), 10, torch.float32 if weighted == "f32" else TORCH[dtype]) if weighted else None
    out = Guarded(n, cols, TORCH[dtype], pad, offset)
    got = ew.ew_expert_combine(y.t, plan, w, residual=residual.t if residual else None, out=out.t)
    assert got is out.t
    check_combine(got, y.t, plan, w, residual.t if residual else None, dtype)
    assert y.intact() and out.intact() and (residual is None or residual.intact())


def check_combine(got, y, plan, w, residual, dtype):
    n, k = plan.positions.shape
    want = residual.double() if residual is not None else torch.zeros(n, y.shape[1], dtype=torch.float64, device="cuda")
    size = want.abs()
    for j in range(k):
        given = plan.positions[:, j] >= 0
        term = y.double()[plan.positions[:, j].long()[given]] * (w.double()[given, j, None] if w is not None else 1.0)
        want[given] += term
        size[given] += term.abs()
    assert_within(got, want, UNIT[dtype] * want.abs() + (k + 1) * EPS32 * size + TINY[dtype], "out")


@pytest.mark.parametrize("weighted", [None, "own", "f32"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,experts,align,cols,pad,offset", ROWS)
def test_combine_grad(dtype, weighted, n, k, experts, align, cols, pad, offset):
    plan = ew.ew_expert_sort(choices(n, k, experts, 11), experts, align=align)
    y, dout = rows_of(plan.slots.numel(), cols, dtype, pad, offset, 12), rows_of(n, cols, dtype, pad, offset, 13)
    w = randn((n, k), 14, torch.float32 if weighted == "f32" else TORCH[dtype]) if weighted else None
    dy = Guarded(plan.slots.numel(), cols, TORCH[dtype], pad, offset)
    dw = Guarded(n, k, torch.float32)
    ew.ew_expert_combine_grad(dout.t, y.t, plan, w, dy=dy.t, dweights=dw.t)
    check_combine_grad(dy.t, dw.t, dout.t, y.t, plan, w, dtype)
    assert all(m.intact() for m in (y, dout, dy, dw))


def check_combine_grad(dy, dw, dout, y, plan, w, dtype):
    k, slot = plan.positions.shape[1], plan.slots.long().clamp(min=0)
    given = plan.slots[:, None] >= 0
    factor = w.double().reshape(-1)[slot][:, None] if w is not None else 1.0
    want = torch.where(given, dout.double()[slot // k] * factor, 0.0)
    # a product in binary32, rounded again to the type
    assert_within(dy, want, (UNIT[dtype] + EPS32) * want.abs() * (1 + UNIT[dtype]) + TINY[dtype], "dy")
    assert not dy[plan.slots < 0].any()
    for j in range(k):
        there = plan.positions[:, j] >= 0
        terms = dout.double()[there] * y.double()[plan.positions[:, j].long()[there]]
        # a term goes through 4 sums in its tile, one more there, one a tile, 5 of lanes and up to 8 of warps
        steps = (y.shape[1] // 256 + 20) * EPS32
        assert_within(dw[there, j], terms.sum(1), steps * terms.abs().sum(1), "dweights")
        assert not dw[~there, j].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [40, 1001, 2048])
@pytest.mark.parametrize("places", [(0, 1, 2, 3), (4, 4, 0, 4), (1, 1, 1, 0)])
def test_matrices_whose_rows_lie_apart(dtype, cols, places):
    plan = ew.ew_expert_sort(choices(100, 3, 9, 15), 9, align=4)
    rows = plan.slots.numel()
    x, residual = (rows_of(100, cols, dtype, 8 * o, o, 16 + o) for o in places[:2])
    y = rows_of(rows, cols, dtype, 0, places[2], 20)
    w = randn((100, 3), 21)
    sorted_x, out = Guarded(rows, cols, TORCH[dtype], 0, places[3]), Guarded(100, cols, TORCH[dtype], 3, places[3])
    ew.ew_expert_dispatch(x.t, plan, out=sorted_x.t)
    token = plan.slots.long().clamp(min=0) // 3
    assert torch.equal(sorted_x.t, torch.where(plan.slots[:, None] >= 0, x.t[token], 0.0))
    ew.ew_expert_combine(y.t, plan, w, residual=residual.t, out=out.t)
    check_combine(out.t, y.t, plan, w, residual.t, dtype)
    dy = Guarded(rows, cols, TORCH[dtype], 1, places[3])
    _, dw = ew.ew_expert_combine_grad(x.t, y.t, plan, w, dy=dy.t)
    check_combine_grad(dy.t, dw, x.t, y.t, plan, w, dtype)
    assert all(m.intact() for m in (x, residual, y, sorted_x, out, dy))


@pytest.mark.parametrize("cols", [64, 1001])
def test_combine_in_place_and_what_belongs_to_no_slot(cols):
    e = choices(200, 4, 6, 22)
    e[7] = -1
    plan = ew.ew_expert_sort(e, 6, align=16)
    y, residual, w = randn((plan.slots.numel(), cols), 23), randn((200, cols), 24), randn((200, 4), 25)
    y[plan.slots < 0] = math.nan  # rows of no slot are not read
    w[plan.positions < 0] = math.inf  # and weights of slots without an expert do not count
    want = ew.ew_expert_combine(y, plan, w, residual=residual.clone())
    assert torch.isfinite(want).all() and torch.equal(want[7], residual[7])
    assert ew.ew_expert_combine(y, plan, w, residual=residual, out=residual) is residual and torch.equal(residual, want)
    dy, dw = ew.ew_expert_combine_grad(residual, y, plan, w)
    assert torch.isfinite(dy).all() and torch.isfinite(dw).all() and not dw[7].any()


@pytest.mark.parametrize("cols", [48, 1001])
def test_positions_outside_are_left_out(cols):
    plan = ew.ew_expert_sort(choices(60, 2, 5, 26), 5)
    moved = plan.positions.clone()
    moved[3, 0], moved[4, 1], moved[5, 0] = plan.slots.numel(), 2 ** 31 - 1, -2 ** 31
    gone = plan.positions.clone()
    gone[3, 0] = gone[4, 1] = gone[5, 0] = -1
    y, w = randn((plan.slots.numel(), cols), 27), randn((60, 2), 28)
    a, b = plan._replace(positions=moved), plan._replace(positions=gone)
    assert torch.equal(ew.ew_expert_combine(y, a, w), ew.ew_expert_combine(y, b, w))
    assert torch.equal(ew.ew_expert_combine_grad(y[:60].contiguous(), y, a, w)[1], ew.ew_expert_combine_grad(y[:60].contiguous(), y, b, w)[1])
    x = randn((60, cols), 29)
    out = Guarded(plan.slots.numel(), cols, torch.float32, fill=torch.zeros(plan.slots.numel(), cols, device="cuda"))
    ew.ew_expert_dispatch(x, a, out=out.t)
    want = torch.zeros_like(out.t)
    ew.ew_expert_dispatch(x, b, out=want)
    assert torch.equal(out.t, want) and out.intact()


def test_gradients_against_differences():
    """The gradient of sum(c * combine(dispatch(x) * s)) by central differences in 64 bits: linear in x and in the weights,
    so a step of 1e-3 leaves only rounding."""
    n, k, cols = 7, 3, 11
    plan = ew.ew_expert_sort(choices(n, k, 4, 30), 4, align=2)
    x, w, c = randn((n, cols), 31), randn((n, k), 32), randn((n, cols), 33)
    s = randn((plan.slots.numel(), 1), 34)  # stands for the experts
    y = ew.ew_expert_dispatch(x, plan) * s
    dy, dw = ew.ew_expert_combine_grad(c, y, plan, w)
    dx = ew.ew_expert_combine(dy * s, plan)

    def loss(x, w):
        total = 0.0
        for t in range(n):
            for j in range(k):
                p = int(plan.positions[t, j])
                if p >= 0:
                    total += float((c[t].double() * w[t, j] * x[t] * s[p].double()).sum())
        return total

    for by, d in ((0, dx), (1, dw)):
        for at in range(0, d.numel(), 3):
            values = []
            for step in (1e-3, -1e-3):
                moved = [x.double(), w.double()]
                moved[by] = moved[by].clone()
                moved[by].view(-1)[at] += step
                values.append(loss(*moved))
            assert abs((values[0] - values[1]) / 2e-3 - float(d.view(-1)[at])) < 1e-5


def test_c_entry_without_weight_gradients():
    """dweights null: y is not read and may be null."""
    L, stream = ew.lib(), torch.cuda.current_stream().cuda_stream
    plan = ew.ew_expert_sort(choices(90, 4, 6, 35), 6, align=8)
    dout, rows = randn((90, 72), 36), plan.slots.numel()
    want, _ = ew.ew_expert_combine_grad(dout, torch.zeros(rows, 72, device="cuda"), plan)
    dy = torch.full((rows, 72), 7.0, device="cuda")
    assert L.ew_expert_combine_grad(0, dout.data_ptr(), 72, None, 0, rows, plan.positions.data_ptr(), plan.slots.data_ptr(), 0,
                                    None, dy.data_ptr(), 72, None, 90, 4, 72, stream) == 0
    assert torch.equal(dy, want)


@pytest.mark.parametrize("n,cols", [(64, 512), (3000, 520), (3000, 333)])
def test_repeats_bit_for_bit_on_another_stream_and_in_graphs(n, cols):
    def step(e, x, w):
        plan = ew.ew_expert_sort(e, 32, align=16)
        y = ew.ew_expert_dispatch(x, plan)
        out = ew.ew_expert_combine(y, plan, w, residual=x)
        return (*plan, y, out, *ew.ew_expert_combine_grad(out, y, plan, w))

    def inputs(seed):
        return choices(n, 4, 32, seed), randn((n, cols), seed + 1, torch.bfloat16), randn((n, 4), seed + 2)

    case = inputs(40)
    want = step(*case)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            got = step(*case)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, cases, outs = [], [], []
    for seed in (50, 60):
        cases.append(inputs(seed))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*cases[-1]))
        graphs.append(g)
    for case, seed in zip(cases, (70, 80)):
        for held, new in zip(case, inputs(seed)):
            held.copy_(new)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    for case, out in zip(cases, outs):
        assert all(torch.equal(a, b) for a, b in zip(out, step(*case)))


def test_more_than_2_to_the_31_elements():
    """Offsets past 32 bits: 300000 sorted rows of 8192."""
    n, k, cols = 100000, 3, 8192
    e = choices(n, k, 50, 45, missing=0.02)
    plan = ew.ew_expert_sort(e, 50)
    x = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=generator(46))
    y = ew.ew_expert_dispatch(x, plan)
    end = int(plan.offsets[-1])
    for rows in (slice(0, 5), slice(end - 5, end)):
        assert torch.equal(y[rows], x[plan.slots[rows].long() // k])
    assert not y[end:].any()
    w = randn((n, k), 47)
    out = ew.ew_expert_combine(y, plan, w)
    dy, dw = ew.ew_expert_combine_grad(x, y, plan, w)
    for a in (0, n - 4):
        given = plan.positions[a:a + 4] >= 0
        total = torch.where(given, w[a:a + 4], 0.0).double()
        want = x[a:a + 4].double() * total.sum(1, keepdim=True)
        size = x[a:a + 4].double().abs() * total.abs().sum(1, keepdim=True)
        assert_within(out[a:a + 4], want, UNIT["bf16"] * want.abs() + 4 * EPS32 * size, "out")
        squares = x[a:a + 4].double().square().sum(1, keepdim=True) * given
        assert_within(dw[a:a + 4], squares, 160 * EPS32 * squares, "dweights")
    last = plan.slots[end - 1:end].long()
    want = x[last // k].double() * w.reshape(-1)[last].double()[:, None]
    assert_within(dy[end - 1:end], want, 2 * UNIT["bf16"] * want.abs(), "dy")


def test_refusals():
    e = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    plan = ew.ew_expert_sort(e, 3)
    y = torch.zeros(8, 64, device="cuda")
    for call, error in ((lambda: ew.ew_expert_sort(e.float(), 3), TypeError), (lambda: ew.ew_expert_sort(e.cpu(), 3), ValueError),
                        (lambda: ew.ew_expert_sort(e.t(), 3), ValueError),
                        (lambda: ew.ew_expert_dispatch(x[:3], plan), ValueError),
                        (lambda: ew.ew_expert_dispatch(x, plan[:2]), TypeError),
                        (lambda: ew.ew_expert_dispatch(x, e), TypeError),
                        (lambda: ew.ew_expert_dispatch(x.long(), plan), TypeError),
                        (lambda: ew.ew_expert_dispatch(x, plan._replace(slots=plan.slots.long())), ValueError),
                        (lambda: ew.ew_expert_dispatch(x, plan, out=y[:7]), ValueError),
                        (lambda: ew.ew_expert_combine(x, plan), ValueError),
                        (lambda: ew.ew_expert_combine(y, plan, torch.ones(4, device="cuda")), ValueError),
                        (lambda: ew.ew_expert_combine(y, plan, torch.ones(4, 2, device="cuda").half()), TypeError),
                        (lambda: ew.ew_expert_combine(y, plan, residual=x.half()), ValueError),
                        (lambda: ew.ew_expert_combine_grad(x, x, plan), ValueError),
                        (lambda: ew.ew_expert_combine_grad(y, y, plan), ValueError)):
        with pytest.raises(error):
            call()
    for args in ((0, 1), (1025, 1), (3, 0), (3, 65537)):
        with pytest.raises(ew.EwError, match="INVALID"):
            ew.ew_expert_sort(e, args[0], align=args[1])
    with pytest.raises(ew.EwError, match="INVALID"):
        ew.ew_expert_sort(torch.zeros(2, 65, dtype=torch.int32, device="cuda"), 3)
    with pytest.raises(ew.EwError, match="OVERLAP"):
        ew.ew_expert_dispatch(y[:4], plan, out=y)
    with pytest.raises(ew.EwError, match="OVERLAP"):
        ew.ew_expert_combine(y, plan, out=y[:4])
    with pytest.raises(ew.EwError, match="OVERLAP"):
        ew.ew_expert_combine_grad(x, y, plan, dy=y)
