"""Rows of logits at the edges of binary32, through every kernel that a call may take."""
import math

import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import EPS32, TINY, TORCH, UNIT, assert_within, generator, randn
from tests.test_logits_gpu import Want

pytestmark = pytest.mark.gpu

# rows, columns and entries of a teacher that reach each of distillation's kernels: a row to 64 threads, a row to 256,
# a row split over a cluster, and rows in shared memory (one and several blocks a row)
KERNELS = [(200, 1000, 3), (3, 100, 3), (3, 4099, 300), (2, 70001, 300), (3, 70001, 3), (160, 70001, 3), (3, 5000, 3)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,k", KERNELS)
@pytest.mark.parametrize("scale,peak", [(1.0, 2.0 ** 127), (4.0, 2.0 ** 119), (0.125, 2.0 ** 127)])
def test_one_logit_near_the_end_of_binary32(dtype, rows, cols, k, scale, peak):
    """A peak whose exponent is finite, where the other elements' sums times their distance from it are not: p is 1
    at the peak and 0 elsewhere, lse is the peak's value (the others add less than 2^-1000 to the sum)."""
    if k > 3:
        peak /= 512.0  # the loss adds k terms of the peak's size
    x = randn((rows, cols), 31, TORCH[dtype])
    x[1] = 0.0         # large sums apart from the peak
    at = torch.randint(0, cols - k, (rows,), generator=generator(32), device="cuda")
    x[torch.arange(rows, device="cuda"), at] = peak
    ids = at[:, None] + torch.arange(k, device="cuda")
    t = randn((rows, k), 33)
    dloss = randn((rows,), 34)
    v = t.double() * scale
    logq = torch.log_softmax(v, 1)
    q = logq.exp()
    lse = torch.full((rows,), peak * scale, dtype=torch.float64, device="cuda")
    logp = x.double().gather(1, ids) * scale - lse[:, None]
    e_q = EPS32 * (k + 32 + 4 * v.abs().amax(1))
    want_loss = (q * (logq - logp)).sum(1)
    want_d = torch.zeros(rows, cols, dtype=torch.float64, device="cuda").scatter_(1, ids, -q)
    want_d[torch.arange(rows, device="cuda"), at] += 1.0
    bound_d = torch.zeros_like(want_d).scatter_(1, ids, (q + 1.0) * e_q[:, None])
    g = dloss.double()[:, None] * scale

    def check(loss, got_lse, d):
        # log2 e, ln 2 and two products are rounded
        assert_within(got_lse, lse, 4 * EPS32 * lse, "lse")
        assert_within(loss, want_loss, (e_q + 8 * EPS32) * want_loss.abs(), "loss")
        if d is not None:
            assert_within(d, g * want_d, UNIT[dtype] * (g * want_d).abs() + g.abs() * bound_d, "dlogits")

    first = ew.ew_distill_step(x, ids, t, dloss, scale=scale)
    check(*first)
    check(*ew.ew_distill(x, ids, t, scale=scale), None)
    place = x.clone()
    again = ew.ew_distill_step(place, ids, t, dloss, scale=scale, dlogits=place)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    got = ew.ew_logprob(x, at, top=2, scale=scale)
    assert_within(got.lse, lse, 4 * EPS32 * lse, "lse")
    assert not got.logp.any() and not got.entropy.any() and torch.equal(got.top_ids[:, 0].long(), at)


def test_ordinary_rows_beside_them():
    """The rows around a row with a peak keep their values."""
    x = randn((12, 100), 35)
    x[5, 7] = 2.0 ** 127
    ids, t = torch.tensor([[1, 2, 3]], device="cuda").repeat(12, 1), randn((12, 3), 36)
    rest = torch.arange(12, device="cuda") != 5
    want = Want(x[rest], 1.0)
    _, lse = ew.ew_distill(x, ids, t)
    assert_within(lse[rest], want.lse, want.bound + 2 * EPS32 * want.lse.abs(), "lse")


def far_rows(dtype, cols):
    """Rows whose lse is far from 0 or has no room for the logarithm of their number, and ordinary ones."""
    kind = TORCH[dtype]
    lowest, largest, far = torch.finfo(kind).min, torch.finfo(kind).max, 5e4 if dtype == "f16" else 5e5
    x = randn((12, cols), 41, kind)
    x[0] = lowest
    x[1] = -math.inf
    x[1, 0], x[1, cols - 1] = lowest, lowest
    x[2] = largest
    x[3] = far
    x[4] = randn((cols,), 42, torch.float32, 3.0) + 6000.0
    x[5] = randn((cols,), 43) * 8000.0
    x[6] = randn((cols,), 44, torch.float32, 3.0) + far / 5
    x[8] = randn((cols,), 45) - 20000.0
    x[8, ::3] = -math.inf
    x[9] = -math.inf
    x[10] = randn((cols,), 46) + 3000.0
    x[11, cols // 2] = largest / 8
    return x


class FarWant:
    """A row's softmax in 64 bits, relative to its largest element, and how far p may be off in parts of itself: the
    exponents up to 100 (beyond, p is below 2^-126) by three roundings, cols / 256 terms a thread and a tree; from a
    given lse below 4096, four roundings of its size more (lse itself, log2 e, ln 2 and the product)."""

    def __init__(self, x, scale, from_lse):
        z = x.double() * scale
        self.empty = torch.isneginf(z).all(1)
        top = torch.where(self.empty, 0.0, z.amax(1))
        away = z - top[:, None]
        log_s = torch.where(self.empty, 0.0, torch.logsumexp(torch.where(self.empty[:, None], 0.0, away), 1))
        self.logp = torch.where(self.empty[:, None], -math.inf, away - log_s[:, None])
        self.p = self.logp.exp()
        self.entropy = torch.special.entr(self.p).sum(1)
        self.lse = top + log_s
        spread = torch.where(torch.isfinite(away), -away, 0.0).clamp(max=100.0)
        self.e = EPS32 * (x.shape[1] / 256 + 64 + 6 * spread.amax(1))
        self.e_entropy = self.e * (3 + (self.p * spread).sum(1))
        if from_lse:
            self.e = self.e + torch.where(self.lse.abs() < 4096 * 1.001, 4 * EPS32 * self.lse.abs(), 0.0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("times,cols", [(1, 100), (1, 4099), (1, 70001), (1, 300000), (30, 70001), (60, 1000)])
@pytest.mark.parametrize("scale", [1.0, 2.0])
def test_logprob_gradient_far_from_zero(dtype, times, cols, scale):
    x = far_rows(dtype, cols).repeat(times, 1)
    rows = x.shape[0]
    tokens = torch.randint(0, cols, (rows,), generator=generator(47), device="cuda")
    tokens[1], tokens[8], tokens[11] = cols - 1, 1, cols // 2
    a, b = randn((rows,), 48), randn((rows,), 49)
    f = ew.ew_logprob(x, tokens, scale=scale)
    want = FarWant(x, scale, True)
    one = torch.zeros_like(want.p).scatter_(1, tokens[:, None], 1.0)
    away = torch.where(want.p > 0, want.logp + want.entropy[:, None], 0.0)
    for dent in (None, b):
        h = 0.0 if dent is None else b.double()[:, None]
        d = scale * (a.double()[:, None] * (one - want.p) - h * want.p * away)
        d = torch.where(want.empty[:, None], 0.0, d)
        size = scale * want.p * (a.double().abs()[:, None] + abs(h) * (away.abs() + 1))
        bound = (UNIT[dtype] * d.abs() + want.e[:, None] * size + scale * abs(h) * want.p * want.e_entropy[:, None]
                 + 4 * EPS32 * scale * a.double().abs()[:, None] * one
                 + scale * 2.0 ** -125 * (a.double().abs()[:, None] + 100 * abs(h)) + TINY[dtype])
        got = ew.ew_logprob_grad(x, tokens, f.lse, f.entropy, a, dent, scale=scale)
        assert_within(got, d, bound, "dlogits")
        apart = torch.empty(rows * cols + 1, dtype=x.dtype, device="cuda")[1:].view(rows, cols)
        assert torch.equal(ew.ew_logprob_grad(x, tokens, f.lse, f.entropy, a, dent, scale=scale, dlogits=apart), got)
        place = x.clone()
        ew.ew_logprob_grad(place, tokens, f.lse, f.entropy, a, dent, scale=scale, dlogits=place)
        assert torch.equal(place, got)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("times,cols,k", [(1, 100, 3), (1, 4099, 300), (1, 70001, 3), (1, 70001, 300), (30, 70001, 100),
                                          (60, 1000, 3)])
def test_distillation_gradient_far_from_zero(dtype, times, cols, k):
    """From a given lse, and from the sums of the same call: both within the bounds of the same values."""
    x = far_rows(dtype, cols).repeat(times, 1)
    rows, k, scale = x.shape[0], min(k, cols), 0.5
    ids = (torch.arange(rows, device="cuda")[:, None] + torch.arange(k, device="cuda") * (cols // k)) % cols
    ids[7, :] = -1
    t = randn((rows, k), 51)
    dloss = randn((rows,), 52)
    q = torch.softmax(t.double() * scale, 1)
    q[7] = 0.0
    g = dloss.double()[:, None] * scale
    e_q = EPS32 * (k + 32 + 4 * t.double().abs().amax(1, keepdim=True))
    for fused in (False, True):
        want = FarWant(x, scale, not fused)
        dense = torch.zeros_like(want.p).scatter_(1, ids.clamp(min=0), q)
        some = torch.ones_like(q[:, :1])
        some[7] = 0.0
        d = g * (want.p * some - dense)
        bound = (UNIT[dtype] * d.abs() + g.abs() * (want.p * want.e[:, None] + dense * e_q + 2.0 ** -125) + TINY[dtype])
        place = x.clone()
        if fused:
            _, _, got = ew.ew_distill_step(x, ids, t, dloss, scale=scale)
            ew.ew_distill_step(place, ids, t, dloss, scale=scale, dlogits=place)
        else:
            _, lse = ew.ew_distill(x, ids, t, scale=scale)
            got = ew.ew_distill_grad(x, ids, t, lse, dloss, scale=scale)
            ew.ew_distill_grad(place, ids, t, lse, dloss, scale=scale, dlogits=place)
        assert_within(got, d, bound, "step" if fused else "from lse")
        assert torch.equal(place, got)
        assert not got[7].any()


@pytest.mark.parametrize("rows,cols,k", [(2, 100, 100), (3, 5000, 64), (200, 1000, 64), (2, 70001, 1024)])
def test_loss_of_many_terms_near_the_end_of_binary32(rows, cols, k):
    """k equal terms of 1.5e38: their weighted mean is finite, their sum is not."""
    x = torch.zeros(rows, cols, device="cuda")
    x[:, cols - 1] = 1.5e38
    ids = torch.arange(k, device="cuda").repeat(rows, 1)
    ids[ids == cols - 1] = -1
    loss, _ = ew.ew_distill(x, ids, torch.zeros(rows, k, device="cuda"))
    want = torch.full((rows,), 1.5e38, dtype=torch.float64, device="cuda")
    assert_within(loss, want, (k + 40) * EPS32 * want, "loss")


# What distill_launch chooses: rows, columns and entries, and the threads of the block that it launches for
# step and loss (bf16 and f16; f32 at half the columns).  64 and 256: the row is read twice; 160, 320, 640: it is held
# in shared memory by 128, 256 or 512 streaming threads.
ROUTES = [(360, 1000, 3, 64), (360, 14000, 300, 64), (12, 100, 3, 256), (12, 4098, 300, 256), (12, 70002, 300, 256),
          (360, 50002, 300, 256), (360, 14002, 3, 160), (360, 14002, 60, 160), (360, 24002, 100, 320), (12, 10002, 3, 320),
          (360, 50002, 3, 640), (360, 50002, 250, 640), (12, 70002, 3, 640), (12, 70002, 100, 640), (24, 270000, 64, 640)]


def special_rows(dtype, times, cols):
    lowest, largest = torch.finfo(TORCH[dtype]).min, torch.finfo(TORCH[dtype]).max
    x = randn((12, cols), 61, TORCH[dtype])
    x[0] = -math.inf
    x[1] = lowest
    x[2] = -math.inf
    x[2, cols // 2] = 2.5
    x[3, cols // 3] = math.nan
    x[4, cols - 1] = math.inf
    x[5] = lowest
    x[5, 1], x[5, cols - 2] = 1.0, 2.0
    x[6] = -math.inf
    x[6, 0], x[6, cols - 1] = lowest, lowest
    x[7] = largest
    x[8, 0] = largest
    x[10] = -math.inf
    x[10, 3] = lowest
    return x.repeat(times, 1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,k,block", ROUTES)
def test_distillation_of_special_rows_by_every_kernel(dtype, rows, cols, k, block):
    cols, scale = cols // 2 if dtype == "f32" else cols, 0.5
    x = special_rows(dtype, rows // 12, cols)
    k = min(k, cols)
    g = generator(62)
    # among the ids the columns that special rows have left; some rows without a teacher
    ids = (torch.randint(0, cols, (rows, 1), generator=g, device="cuda") + torch.arange(k, device="cuda") * (cols // k)) % cols
    ids[2::12], ids[6::12, 1], ids[10::12] = cols // 2, cols - 1, 3  # one id k times in rows 2 and 10
    ids[9::24] = -1
    t, dloss = randn((rows, k), 63, TORCH[dtype]), randn((rows,), 64)
    broken = torch.zeros(rows, dtype=torch.bool, device="cuda")
    broken[3::12] = broken[4::12] = True
    want = FarWant(torch.where(broken[:, None], 0.0, x), scale, False)
    given = (ids >= 0)
    some = given[:, :1]
    logq = torch.where(given, torch.log_softmax(t.double() * scale, 1), 0.0)
    q = torch.where(given, logq.exp(), 0.0)
    at = ids.clamp(min=0)
    logp = want.logp.gather(1, at)
    want_loss = torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
    e_q = EPS32 * (k + 32 + 4 * t.double().abs().amax(1))
    size = (q * (logq.abs() + torch.where(torch.isfinite(logp), logp, 0.0).abs())).sum(1)
    loss_bound = want.e + e_q + (e_q + 8 * EPS32) * size
    want_lse = torch.where(want.empty, -math.inf, want.lse)
    lse_bound = want.e + 4 * EPS32 * want.lse.abs()
    gain = dloss.double()[:, None] * scale
    dense = torch.zeros_like(want.p).scatter_add_(1, at, q)
    want_d = gain * (want.p * some - dense)
    d_bound = (UNIT[dtype] * want_d.abs() + gain.abs() * (want.p * want.e[:, None] + dense * e_q[:, None] + 2.0 ** -125)
               + TINY[dtype])
    lse_d_bound = d_bound + gain.abs() * want.p * torch.where(want.lse.abs() < 4100, 4 * EPS32 * want.lse.abs(), 0.0)[:, None]
    nan = torch.full_like(want_loss, math.nan)
    want_loss, want_lse = torch.where(broken & some[:, 0], nan, want_loss), torch.where(broken, nan, want_lse)
    want_d = torch.where((broken & some[:, 0])[:, None], math.nan, want_d)

    place = x.clone()
    loss, lse, d = ew.ew_distill_step(x, ids, t, dloss, scale=scale)
    assert ew.last_launch()["block"] == block
    assert_within(lse, want_lse, lse_bound, "lse")
    assert_within(loss, want_loss, loss_bound, "loss")
    assert_within(d, want_d, d_bound, "dlogits")
    ew.ew_distill_step(place, ids, t, dloss, scale=scale, dlogits=place)
    assert same_bits(place, d)
    apart = torch.empty(rows * cols + 1, dtype=x.dtype, device="cuda")[1:].view(rows, cols)
    ew.ew_distill_step(x, ids, t, dloss, scale=scale, dlogits=apart)
    assert same_bits(apart, d)
    loss2, lse2 = ew.ew_distill(x, ids, t, scale=scale)
    assert ew.last_launch()["block"] == block and same_bits(loss, loss2) and same_bits(lse, lse2)
    d2 = ew.ew_distill_grad(x, ids, t, lse, dloss, scale=scale)
    assert_within(d2, want_d, lse_d_bound, "dlogits from lse")
    place = x.clone()
    ew.ew_distill_grad(place, ids, t, lse, dloss, scale=scale, dlogits=place)
    assert same_bits(place, d2)


def same_bits(a, b):
    """Equal, NaN with NaN."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a, nan=0.0), torch.nan_to_num(b, nan=0.0))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("times,cols", [(1, 100), (1, 4099), (1, 70001), (30, 1000), (30, 40001)])
@pytest.mark.parametrize("top", [20, 25, 64])
def test_alternatives_of_special_rows(dtype, times, cols, top):
    """Ties, few elements, NaN and infinities, with the bounds of few and of many groups."""
    x = special_rows(dtype, times, cols)
    got = ew.ew_logprob(x, None, top=top, scale=0.5)
    broken = torch.isnan(x).any(1) | torch.isposinf(x).any(1)
    clean = torch.where(broken[:, None], 0.0, x.double())
    best, ids = torch.sort(clean, dim=1, descending=True, stable=True)
    best, ids = best[:, :top], ids[:, :top]
    missing = torch.isneginf(best) | broken[:, None]
    assert torch.equal(got.top_ids.long(), torch.where(missing, -1, ids))
    want = FarWant(clean, 0.5, False)
    logp = torch.where(torch.isneginf(best), -math.inf, want.logp.gather(1, ids))
    size = torch.where(torch.isfinite(logp), logp.abs(), 0.0)
    assert_within(got.top_logp, torch.where(broken[:, None], math.nan, logp), want.e[:, None] + 6 * EPS32 * size, "top")
