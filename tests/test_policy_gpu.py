"""The clipped policy loss and its gradient on the GPU against 64 bits."""
import math

import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import EPS32, TINY, TORCH, UNIT, Guarded, assert_within, generator, randn
from tests.test_logits_gpu import Want, logits_of, special_rows

pytestmark = pytest.mark.gpu

# rows, cols, pad, offset: fewer than a chunk, rows that start anywhere, few and many rows (up to several for each block)
# of every size at which another kernel, block size or split is chosen
SHAPES = [(1, 1, 0, 0), (3, 5, 0, 1), (2, 8, 0, 0), (5, 100, 0, 0), (3, 1000, 24, 8), (4, 4097, 0, 0), (5, 8192, 0, 0),
          (3, 16387, 0, 3), (6, 50001, 0, 0), (1, 131072, 0, 0), (3, 150001, 0, 0), (400, 3001, 0, 0), (700, 12000, 8, 0),
          (330, 20001, 0, 0), (170, 33333, 0, 0), (165, 65536, 0, 0), (160, 100003, 5, 1), (320, 131071, 0, 0), (2, 400001, 0, 0)]
HOW = dict(clip_low=0.2, clip_high=0.3, kl=0.1)


def rounded(v):
    return float(torch.tensor(v, dtype=torch.float32))


class Case:
    """A policy's tokens: ratios on both sides of the clipping, none within 1e-2 of its borders, a third without a token."""

    def __init__(self, rows, cols, dtype, pad, offset, seed, scale=1.0, masked=0.33, x=None):
        self.dtype, self.scale = dtype, scale
        self.x = x if x is not None else logits_of(rows, cols, dtype, pad, offset, seed)
        if x is None and cols > 50:
            self.x.t[:, ::3] = -math.inf
        self.want = Want(self.x.t, rounded(scale))
        g = generator(seed + 1)
        tokens = torch.randint(0, max(1, cols // 3), (rows,), generator=g, device="cuda") * 3 + (1 if cols > 50 else 0)
        tokens = tokens.clamp(max=cols - 1 - (cols > 50 and (cols - 1) % 3 == 0))
        self.at = tokens.clone()
        gone = torch.rand(rows, generator=g, device="cuda") < masked
        tokens[gone] = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, -1, cols)[gone]
        self.tokens = tokens
        self.given = (tokens >= 0) & (tokens < cols)
        logp = self.want.logp.gather(1, self.at[:, None])[:, 0]
        moved = 0.3 * torch.randn(rows, generator=g, device="cuda").double()
        moved[::5] *= 10.0
        for border in (math.log(0.8), math.log(1.3)):
            moved = torch.where((moved - border).abs() < 0.02, moved + 0.05, moved)
        base = torch.where(torch.isfinite(logp), logp, 0.0)
        self.old = (base - moved).float()
        apart = torch.randn(rows, generator=g, device="cuda").double()
        apart[::4] *= 1e-3
        apart[1::7] *= 6.0
        self.ref = (base + apart).float()
        self.adv = torch.randn(rows, generator=g, device="cuda")
        self.adv[::11] = 0.0
        self.dloss = torch.randn(rows, generator=g, device="cuda")

    def expected(self, old=True, ref=True, logp=None):
        """Loss and slope in 64 bits with bounds: of logp's error, and of a few roundings of each term."""
        w = self.want
        if logp is None:
            logp = w.logp.gather(1, self.at[:, None])[:, 0]
            e = w.bound + 4 * EPS32 * logp.abs()
        else:
            logp, e = logp.double(), torch.zeros_like(logp, dtype=torch.float64)
        adv, d = self.adv.double(), self.dloss.double()
        low, high, kl = 1.0 - HOW["clip_low"], 1.0 + HOW["clip_high"], rounded(HOW["kl"])
        gap = logp - self.old.double() if old else torch.zeros_like(logp)
        ratio = gap.exp()
        free, bound = ratio * adv, ratio.clamp(low, high) * adv
        clipped = free > bound
        loss = -torch.where(clipped, bound, free)
        free_off = free.abs() * (torch.expm1(e if old else 0 * e) + EPS32 * (gap.abs() + 5))
        loss_off = torch.where(clipped, 4 * EPS32 * bound.abs(), free_off)
        slope, slope_off = -torch.where(clipped, 0.0, free), torch.where(clipped, 0.0, free_off)
        if ref:
            apart = self.ref.double() - logp
            one = torch.expm1(apart)
            loss = loss + kl * (one - apart)
            move = e + EPS32 * apart.abs()
            loss_off = loss_off + kl * (one.abs() * move + apart.exp() * move ** 2 + 8 * EPS32 * (one.abs() + apart.abs()) * (apart.abs() >= 0.49)
                                        + 16 * EPS32 * (one - apart).abs())
            slope = slope - kl * one
            slope_off = slope_off + kl * (apart.exp() * torch.expm1(move) + 6 * EPS32 * one.abs())
        loss_off = loss_off + 4 * EPS32 * loss.abs()
        slope_off = slope_off + 2 * EPS32 * slope.abs()
        factor, factor_off = d * slope * rounded(self.scale), d.abs() * rounded(self.scale) * slope_off
        factor_off = factor_off + 3 * EPS32 * factor.abs()
        g = self.given
        return [torch.where(g, v, 0.0) for v in (loss, loss_off, factor, factor_off)]

    def check_sums(self, loss, logp, lse, **how):
        want_loss, loss_off, _, _ = self.expected(**how)
        w, g = self.want, self.given
        at = w.logp.gather(1, self.at[:, None])[:, 0]
        assert_within(lse, torch.where(g, w.lse, 0.0), torch.where(g, w.bound + 2 * EPS32 * w.lse.abs(), 0.0), "lse")
        assert_within(logp, torch.where(g, at, 0.0), torch.where(g, w.bound + 4 * EPS32 * at.abs(), 0.0), "logp")
        assert_within(loss, want_loss, loss_off, "loss")

    def check_grad(self, d, more=0.0, **how):
        """more: how far p is off beside the sums' error."""
        _, _, f, off = (v[:, None] if v.dim() else v for v in self.expected(**how))
        p = self.want.p
        one = torch.zeros_like(p).scatter_(1, self.at[:, None], 1.0)
        want = f * (one - p)
        p_off = p * (self.want.bound[:, None] + 8 * EPS32 + more)
        bound = (off * (one - p).abs() + f.abs() * (p_off + 4 * EPS32 * one)) * (1 + UNIT[self.dtype])
        assert_within(d, want, UNIT[self.dtype] * want.abs() + bound + TINY[self.dtype], "dlogits")
        assert not d[~self.given].any()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_loss_gradient_and_both(dtype, rows, cols, pad, offset):
    scale = 1.0 if rows % 2 else 0.7
    c = Case(rows, cols, dtype, pad, offset, 1, scale)
    tokens = c.tokens.int() if cols % 2 else c.tokens
    how = dict(old_logp=c.old, ref_logp=c.ref, scale=scale, **HOW)
    loss, logp, lse = ew.ew_policy(c.x.t, tokens, c.adv, **how)
    c.check_sums(loss, logp, lse)
    out = Guarded(rows, cols, TORCH[dtype], pad, offset)
    step = ew.ew_policy_step(c.x.t, tokens, c.adv, c.dloss, dlogits=out.t, **how)
    assert step[3] is out.t
    assert all(torch.equal(a, b) for a, b in zip(step, (loss, logp, lse)))  # the same sums, the same bits
    c.check_grad(out.t)
    d = Guarded(rows, cols, TORCH[dtype], pad, offset)
    ew.ew_policy_grad(c.x.t, tokens, c.adv, logp, lse, c.dloss, dlogits=d.t, **how)
    c.check_grad(d.t, more=4 * EPS32 * c.want.lse.abs()[:, None])
    assert c.x.intact() and out.intact() and d.intact()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(4, 4097), (400, 3001), (330, 20001), (165, 65536), (3, 150001)])
@pytest.mark.parametrize("old,ref", [(False, False), (True, False), (False, True)])
def test_without_an_old_policy_or_a_reference(dtype, rows, cols, old, ref):
    c = Case(rows, cols, dtype, 0, 0, 3)
    how = dict(old_logp=c.old if old else None, ref_logp=c.ref if ref else None, **HOW)
    loss, logp, lse, d = ew.ew_policy_step(c.x.t, c.tokens, c.adv, c.dloss, **how)
    c.check_sums(loss, logp, lse, old=old, ref=ref)
    c.check_grad(d, old=old, ref=ref)
    # a weight of 0 is no term, whatever the reference is
    nan = torch.full_like(c.ref, math.nan)
    a = ew.ew_policy(c.x.t, c.tokens, c.adv, old_logp=how["old_logp"], ref_logp=nan, clip_low=0.2, clip_high=0.3, kl=0.0)
    b = ew.ew_policy(c.x.t, c.tokens, c.adv, old_logp=how["old_logp"], clip_low=0.2, clip_high=0.3)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(4, 4097), (3, 20001), (400, 3001), (330, 20001), (165, 65536), (160, 131072), (3, 150001),
                                       (2, 400001)])
def test_in_place_and_repeated(dtype, rows, cols):
    c = Case(rows, cols, dtype, 0, 0, 4)
    how = dict(old_logp=c.old, ref_logp=c.ref, **HOW)
    want = ew.ew_policy_step(c.x.t, c.tokens, c.adv, c.dloss, **how)
    place = c.x.t.clone()
    got = ew.ew_policy_step(place, c.tokens, c.adv, c.dloss, dlogits=place, **how)
    assert got[3] is place and all(torch.equal(a, b) for a, b in zip(got, want))
    d = ew.ew_policy_grad(c.x.t, c.tokens, c.adv, want[1], want[2], c.dloss, **how)
    place = c.x.t.clone()
    assert torch.equal(ew.ew_policy_grad(place, c.tokens, c.adv, want[1], want[2], c.dloss, dlogits=place, **how), d)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("cols", [5003, 40004, 100003])
@pytest.mark.parametrize("rows", [7, 200])
def test_outputs_whose_rows_lie_apart(dtype, cols, rows):
    """dlogits at another place between multiples of 16 bytes than the logits, and of another stride."""
    c = Case(rows, cols, dtype, 0, 0, 5)
    how = dict(old_logp=c.old, ref_logp=c.ref, **HOW)
    for pad, offset in ((3, 1), (0, 5)):
        out = Guarded(rows, cols, TORCH[dtype], pad, offset)
        ew.ew_policy_step(c.x.t, c.tokens, c.adv, c.dloss, dlogits=out.t, **how)
        c.check_grad(out.t)
        assert out.intact() and c.x.intact()


@pytest.mark.parametrize("rows,cols", [(200, 20000), (600, 70000), (1000, 4000), (9, 70000), (500, 131072)])
@pytest.mark.parametrize("how", ["none", "all but one", "prompts", "all"])
def test_rows_without_a_token_are_not_read(rows, cols, how):
    """Runs of rows without a token, longer than what is read ahead; NaN in them changes nothing."""
    c = Case(rows, cols, "bf16", 0, 0, 6, masked=0.0)
    t = c.tokens
    if how == "none":
        t[:] = -1
    elif how == "all but one":
        t[torch.arange(rows, device="cuda") != rows // 2] = -1
    elif how == "prompts":
        t[torch.arange(rows, device="cuda") % (rows // 2) < rows // 3] = -1
    c.given = t >= 0
    c.x.t[~c.given] = math.nan
    c.want = Want(torch.where(c.given[:, None], c.x.t, 0.0), 1.0)
    loss, logp, lse, d = ew.ew_policy_step(c.x.t, t, c.adv, c.dloss, old_logp=c.old, ref_logp=c.ref, **HOW)
    c.check_sums(loss, logp, lse)
    c.check_grad(d)
    d = ew.ew_policy_grad(c.x.t, t, c.adv, logp, lse, c.dloss, old_logp=c.old, ref_logp=c.ref, **HOW)
    c.check_grad(d, more=4 * EPS32 * c.want.lse.abs()[:, None])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [100, 4099, 20004, 70001])
@pytest.mark.parametrize("copies", [1, 30])
def test_special_rows(dtype, cols, copies):
    """Masked, broken and huge rows, beside one another and through every kernel."""
    x = special_rows(dtype, cols).repeat(copies, 1)
    rows = x.shape[0]
    kind = torch.arange(rows, device="cuda") % 12
    tokens = torch.full((rows,), cols // 2, dtype=torch.int64, device="cuda")
    tokens[kind == 5], tokens[kind == 6], tokens[kind == 8], tokens[kind == 10] = cols - 2, 0, 0, 3
    adv, dloss = randn((rows,), 7), randn((rows,), 8)
    old = randn((rows,), 9) - 3.0
    first = None
    for place in (False, True):
        y = x.clone()
        loss, logp, lse, d = ew.ew_policy_step(y, tokens, adv, dloss, old_logp=old, dlogits=y if place else None)
        sums = ew.ew_policy(x, tokens, adv, old_logp=old)
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(sums, (loss, logp, lse)))
        first = first or (loss, logp, lse, d.clone())
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(first, (loss, logp, lse, d)))
        want = ew.ew_logprob(x, tokens)
        fine = (kind != 3) & (kind != 4)
        for got, w in ((logp, want.logp), (lse, want.lse)):
            assert torch.isnan(got[~fine]).all() and torch.equal(torch.isinf(got[fine]), torch.isinf(w[fine]))
            there = fine & torch.isfinite(w)
            # the entropy's sums beside the others change an addition's order at most
            assert_within(got[there], w[there].double(), 600 * EPS32 * (1 + w[there].double().abs()), "logp, lse")
        assert torch.isnan(loss[~fine]).all() and torch.isnan(d[~fine]).all()
        assert not d[kind == 0].any()  # nothing but masked elements
        exact = Want(x[fine], 1.0)
        p = torch.where(exact.empty[:, None], 0.0, exact.p)
        ratio = torch.exp(exact.logp.gather(1, tokens[fine][:, None])[:, 0] - old[fine].double())
        free = torch.where(adv[fine] == 0, 0.0, ratio * adv[fine])
        clipped = free > ratio.clamp(0.8, 1.2) * adv[fine]
        near = ((ratio - 0.8).abs() < 1e-2) | ((ratio - 1.2).abs() < 1e-2)
        factor = -torch.where(clipped, 0.0, free) * dloss[fine]
        one = torch.zeros_like(p).scatter_(1, tokens[fine][:, None], 1.0)
        g = torch.where(exact.empty[:, None], 0.0, factor[:, None] * (one - p))
        size = exact.x.abs().amax(1).clamp(max=1e9)
        sound = ~near & torch.isfinite(factor) & (size < 1e3)  # a larger exponent has fewer digits
        e = 3 * exact.bound[sound] + 16 * EPS32
        bound = UNIT[dtype] * g[sound].abs() + 2 * factor[sound].abs()[:, None] * (p[sound] + one[sound]) * e[:, None] + TINY[dtype]
        assert_within(d[fine][sound], g[sound], bound, "dlogits")
        back = x.clone()
        again = ew.ew_policy_grad(back, tokens, adv, logp, lse, dloss, old_logp=old, dlogits=back if place else None)
        assert torch.isnan(again[~fine]).all() and not again[kind == 0].any()
        bound = bound + 2 * factor[sound].abs()[:, None] * p[sound] * (4 * EPS32 * exact.lse[sound].abs()[:, None])
        assert_within(again[fine][sound], g[sound], bound, "dlogits from lse")


def test_ends_of_the_terms():
    """A masked token, ratios past binary32, no advantage, a gradient that is not wanted, clipping at its ends."""
    x = torch.zeros(8, 64, device="cuda")
    x[0, 3] = -math.inf
    x[1, 3] = -200.0
    x[2, 3] = -200.0
    tokens = torch.full((8,), 3, device="cuda")
    old = torch.full((8,), -math.log(64.0), device="cuda")
    old[4] = old[5] = -200.0  # ratios of e^196
    adv = torch.tensor([2.0, 2.0, -2.0, 0.0, 1.0, -1.0, 0.0, 3.0], device="cuda")
    old[6] = -200.0
    one = torch.ones(8, device="cuda")
    loss, logp, _, d = ew.ew_policy_step(x, tokens, adv, one, old_logp=old)
    assert torch.isneginf(logp[0]) and loss[0] == 0 and not d[0].any()           # ratio 0, a gain: not clipped, no slope
    assert abs(float(loss[2]) - 1.6) < 1e-6 and not d[2].any()                    # ratio 0, a loss: clipped
    assert loss[3] == 0 and not d[3].any() and loss[6] == 0 and not d[6].any()    # no advantage
    assert abs(float(loss[4]) + 1.2) < 1e-6 and not d[4].any()                    # clipped above
    assert float(loss[5]) == math.inf                                            # a loss is not clipped above
    assert abs(float(loss[7]) + 3.0) < 1e-5 and abs(float(d[7, 3]) + 3.0 * 63 / 64) < 1e-5
    free = ew.ew_policy_step(x, tokens, adv, one, old_logp=old, clip_low=1.0, clip_high=math.inf)[0]
    assert free[2] == 0 and float(free[4]) == -math.inf
    none = ew.ew_policy_step(x, tokens, adv, 0.0 * one, old_logp=old)[3]
    assert not none.any()
    far = ew.ew_policy(x, tokens, adv, old_logp=old, ref_logp=old, kl=0.5)[0]
    assert float(far[0]) == math.inf and float(far[1]) == math.inf  # infinite, and e^196 / 2, past binary32
    assert torch.isfinite(far[7])
    # apart 0: no divergence
    same = ew.ew_policy(x[7:], tokens[7:], adv[7:], old_logp=logp[7:], ref_logp=logp[7:], kl=0.5)[0]
    assert float(same) == -3.0


def test_gradient_against_differences():
    """Central differences of the loss in 64 bits; ratios stay away from the borders.  A step of 1e-5 leaves a
    truncation of about 1e-10 and a rounding of about 1e-11; the kernel adds binary32's own."""
    c = Case(9, 41, "f32", 0, 0, 10, 0.7, masked=0.2)
    how = dict(old_logp=c.old, ref_logp=c.ref, scale=0.7, **HOW)
    d = ew.ew_policy_step(c.x.t, c.tokens, c.adv, c.dloss, **how)[3]

    def loss(x):
        moved = Case.__new__(Case)
        moved.__dict__.update(c.__dict__)
        moved.want = Want(x, rounded(0.7))
        return float((moved.expected()[0] * c.dloss.double()).sum())

    for k in list(range(0, d.numel(), 7)) + [int(r) * 41 + int(t) for r, t in enumerate(c.at)]:
        values = []
        for step in (1e-5, -1e-5):
            x = c.x.t.double().clone()
            x.view(-1)[k] += step
            values.append(loss(x))
        want = (values[0] - values[1]) / 2e-5
        assert abs(want - float(d.reshape(-1)[k])) < 2e-5 * (1 + abs(want))


@pytest.mark.parametrize("rows,cols", [(3, 9000), (700, 5000), (300, 40000)])
def test_another_stream_and_graphs(rows, cols):
    def step(x, tokens, adv, old, ref, dloss):
        a = ew.ew_policy_step(x, tokens, adv, dloss, old_logp=old, ref_logp=ref, **HOW)
        return (*a, ew.ew_policy_grad(x, tokens, adv, a[1], a[2], dloss, old_logp=old, ref_logp=ref, **HOW))

    def inputs(seed):
        c = Case(rows, cols, "bf16", 0, 0, seed)
        return c.x.t.contiguous(), c.tokens, c.adv, c.old, c.ref, c.dloss

    case = inputs(11)
    want = step(*case)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            got = step(*case)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, cases, outs = [], [], []
    for seed in (12, 13):
        cases.append(inputs(seed))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*cases[-1]))
        graphs.append(g)
    for case, seed in zip(cases, (14, 15)):
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
    rows, cols = 20000, 131072
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=generator(16))
    tokens = torch.randint(0, cols, (rows,), generator=generator(17), device="cuda")
    adv, one = randn((rows,), 18), torch.ones(rows, device="cuda")
    loss, logp, lse, d = ew.ew_policy_step(x, tokens, adv, one)
    for a in (0, rows - 2):
        part = slice(a, a + 2)
        want = Want(x[part], 1.0)
        at = want.logp.gather(1, tokens[part, None])[:, 0]
        assert_within(logp[part], at, want.bound + 4 * EPS32 * at.abs(), "logp")
        assert_within(loss[part], -adv[part].double(), 4 * EPS32 * adv[part].double().abs(), "loss")
        g = -adv[part].double()[:, None] * (torch.zeros_like(want.p).scatter_(1, tokens[part, None], 1.0) - want.p)
        off = adv[part].double().abs()[:, None] * want.p * (want.bound[:, None] + 16 * EPS32) + 8 * EPS32 * g.abs()
        assert_within(d[part], g, UNIT["bf16"] * g.abs() + 2 * off + TINY["bf16"], "dlogits")
    assert torch.isfinite(loss).all()


def test_more_rows_than_a_blocks_list_holds():
    """Rows of 24 KiB and more, 512 of them from each block at a time: three rounds of lists, rows without a token among
    them, whole lists of either kind."""
    rows, cols = 700000, 12300
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=generator(19))
    tokens = torch.randint(0, cols, (rows,), generator=generator(20), device="cuda", dtype=torch.int32)
    tokens[torch.rand(rows, generator=generator(21), device="cuda") < 0.5] = -1
    tokens[:300] = -1
    tokens[320000:330000] = 7
    adv, one = randn((rows,), 22), torch.ones(rows, device="cuda")
    given = tokens >= 0
    picked = torch.cat([torch.nonzero(given)[:3, 0], torch.nonzero(given)[-3:, 0], torch.tensor([320000, 329999], device="cuda")])
    before = x[picked].clone()
    loss, logp, lse, d = ew.ew_policy_step(x, tokens, adv, one, dlogits=x)
    assert not loss[~given].any() and not logp[~given].any() and not lse[~given].any()
    assert_within(loss[given], -adv[given].double(), 4 * EPS32 * adv[given].double().abs(), "loss")
    assert float(lse[given].min()) > 9.0 and float(lse[given].max()) < 11.0  # log(12300) + 1/2, give or take 0.02
    for part in torch.arange(rows, device="cuda").split(100000):  # a gradient's row adds up to nothing, and holds something
        sums, largest = d[part].float().sum(1), d[part].abs().amax(1).float()
        assert not largest[~given[part]].any() and (largest[given[part]] > 0.9 * adv[part][given[part]].abs()).all()
        assert (sums.abs() <= 2 * UNIT["bf16"] * 2 * adv[part].abs()).all()
    want = Want(before, 1.0)
    at = tokens[picked].long()[:, None]
    g = -adv[picked].double()[:, None] * (torch.zeros_like(want.p).scatter_(1, at, 1.0) - want.p)
    off = adv[picked].double().abs()[:, None] * want.p * (want.bound[:, None] + 16 * EPS32) + 8 * EPS32 * g.abs()
    assert_within(d[picked], g, UNIT["bf16"] * g.abs() + 2 * off + TINY["bf16"], "dlogits")


def test_no_rows():
    x, none = torch.empty(0, 40, device="cuda"), torch.empty(0, device="cuda")
    loss, logp, lse, d = ew.ew_policy_step(x, none.long(), none, none)
    assert loss.shape == (0,) and d.shape == (0, 40)
    assert ew.ew_policy_grad(x, none.long(), none, logp, lse, none).shape == (0, 40)


def test_refusals():
    x, t, f = torch.zeros(4, 64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    for call, error in ((lambda: ew.ew_policy(x.double(), t, f), TypeError), (lambda: ew.ew_policy(x, f, f), TypeError),
                        (lambda: ew.ew_policy(x, t[:3], f), ValueError), (lambda: ew.ew_policy(x, t, f[:3]), ValueError),
                        (lambda: ew.ew_policy(x, t, f.half()), ValueError), (lambda: ew.ew_policy(x.cpu(), t, f), ValueError),
                        (lambda: ew.ew_policy(x, t, f, old_logp=f[:2]), ValueError),
                        (lambda: ew.ew_policy(x, t, f, ref_logp=f.double()), ValueError),
                        (lambda: ew.ew_policy_step(x, t, f, None), TypeError),
                        (lambda: ew.ew_policy_grad(x, t, f, f, f, f, dlogits=x.half()), ValueError)):
        with pytest.raises(error):
            call()
    for how in (dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_high=-0.1), dict(clip_high=math.nan), dict(kl=-1.0),
                dict(kl=math.inf), dict(scale=0.0), dict(scale=2.0 ** 21)):
        with pytest.raises(ew.EwError, match="INVALID"):
            ew.ew_policy(x, t, f, **how)
    with pytest.raises(ew.EwError, match="OVERLAP"):
        ew.ew_policy_step(x[:3], t[:3], f[:3], f[:3], dlogits=x[1:])
