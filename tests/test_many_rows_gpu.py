"""Row operators where another kernel, block size or ring is chosen: more rows than the device holds at a time, the
sizes on both sides of a choice."""
import math

import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests import test_embed_gpu as embed
from tests import test_logits_gpu as logits
from tests import test_norm_gpu as norm
from tests.rows_util import EPS32, TINY, TORCH, UNIT, Guarded, assert_within, randn

pytestmark = pytest.mark.gpu

ROWS = 700  # more than four blocks an SM of 152 or fewer


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols,pad,offset", [(5, 0, 0), (40, 0, 0), (1001, 3, 1), (2045, 0, 0), (4090, 6, 3)])
@pytest.mark.parametrize("top", [0, 1, 24, 25])
def test_logprob(dtype, cols, pad, offset, top):
    x = logits.logits_of(ROWS, cols, dtype, pad, offset, 31)
    x.t[:, ::3] = -math.inf
    x.t[3] = -math.inf
    x.t[4] = 0.25  # ties alone
    tokens = logits.some_tokens(ROWS, cols, 32)
    got = ew.ew_logprob(x.t, tokens, top=top)
    want = logits.Want(x.t, 1.0)
    full = ~want.empty
    assert torch.isneginf(got.lse[3]) and float(got.entropy[3]) == 0
    assert_within(got.lse[full], want.lse[full], (want.bound + 2 * EPS32 * want.lse.abs())[full], "lse")
    assert_within(got.entropy[full], want.entropy[full], (want.entropy_bound + 2 * EPS32 * want.entropy)[full], "entropy")
    given = (tokens >= 0) & (tokens < cols)
    at = torch.where(given, want.logp.gather(1, torch.where(given, tokens, 0)[:, None])[:, 0], 0.0)
    size = torch.where(torch.isneginf(at), 0.0, at.abs())
    assert_within(got.logp, at, (want.bound + 4 * EPS32 * size) * given, "logp")
    if top:
        logits.check_top(got, x.t, want, top)
    assert x.intact()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("how", ["rising", "constant", "few values"])
def test_top_of_short_rows_with_ties(dtype, how):
    cols = 2047
    j = torch.arange(cols, device="cuda", dtype=torch.float32)
    x = {"rising": j / cols * 8, "constant": torch.full_like(j, 1.5), "few values": (j * 7919 % 5).floor()}[how]
    x = x.to(TORCH[dtype]).repeat(ROWS, 1)
    for top in (1, 20):
        got = ew.ew_logprob(x, None, top=top)
        logits.check_top(got, x, logits.Want(x, 1.0), top)


# rows of 2, 26, 40, 47 and 80 KiB of 16-bit elements, the second at every start, with few and many teacher's entries
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols,pad,offset", [(7, 0, 0), (1000, 0, 0), (6701, 0, 0), (13401, 2, 5), (20480, 8, 0), (24001, 0, 0),
                                             (40000, 0, 0)])
@pytest.mark.parametrize("k", [8, 33, 64, 100])
def test_distill(dtype, cols, pad, offset, k):
    rows = ROWS if cols < 20000 else 200
    x = logits.logits_of(rows, cols, dtype, pad, offset, 41)
    ids, t = logits.teacher_case(rows, cols, k, TORCH[dtype], 42, torch.int64 if k % 2 else torch.int32)
    ids[5:, :] = torch.where(torch.arange(ids.shape[1], device="cuda") % 5 == 4, ids[5:, :1], ids[5:, :])  # one id many times
    scale, dloss = 0.5, randn((rows,), 44)
    out = Guarded(rows, cols, TORCH[dtype], pad, offset if cols % 2 else offset + 1)
    loss, lse, d = ew.ew_distill_step(x.t, ids, t, dloss, scale=scale, dlogits=out.t)
    want_loss, w, want_d, loss_bound, d_bound = logits.want_distill(x.t, ids, t, scale, dloss)
    assert_within(lse, w.lse, w.bound + 2 * EPS32 * w.lse.abs(), "lse")
    assert_within(loss, want_loss, loss_bound, "loss")
    assert_within(d, want_d, UNIT[dtype] * want_d.abs() + d_bound + TINY[dtype] * (want_d != 0), "dlogits")
    assert x.intact() and out.intact()
    loss2, lse2 = ew.ew_distill(x.t, ids, t, scale=scale)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    d2 = ew.ew_distill_grad(x.t, ids, t, lse, dloss, scale=scale)
    assert_within(d2, want_d, UNIT[dtype] * want_d.abs() + d_bound + TINY[dtype] * (want_d != 0), "dlogits from lse")
    ew.ew_distill_step(x.t, ids, t, dloss, scale=scale, dlogits=x.t)
    assert torch.equal(x.t, d)


# a writer's second, third and sixth row in the ring; widths of every number of tiles a thread; the last piece cut
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", [(5000, 64, 0, 0), (2500, 250, 6, 0), (900, 1001, 7, 0), (1300, 1984, 0, 0),
                                                  (1000, 4090, 6, 0), (700, 5056, 0, 0), (460, 8192, 0, 0), (310, 12296, 0, 0),
                                                  (200, 16384, 0, 0)])
def test_norm_grad(dtype, rows, cols, pad, offset):
    norm.test_backward(dtype, rows, cols, pad, offset)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [3, 700])
@pytest.mark.parametrize("cols,left", [(300, 300), (1000, 1000), (1500, 1500), (2000, 130), (9000, 700), (70000, 1400), (70000, 150)])
def test_top_where_few_threads_have_an_element(dtype, rows, cols, left):
    """Short rows, and rows masked but for a short part: more than 128 elements left, in fewer groups of threads than k."""
    rows = min(rows, 3 if cols > 9000 else rows)
    x = torch.full((rows, cols), -math.inf, device="cuda", dtype=TORCH[dtype])
    x[:, cols - left:] = randn((rows, left), 51, TORCH[dtype], 2.0)
    for top in (20, 24, 64):
        logits.check_top(ew.ew_logprob(x, None, top=top), x, logits.Want(x, 1.0), top)


@pytest.mark.parametrize("n", [2, 65, 511, 512, 513, 2049])
@pytest.mark.parametrize("how", ["uniform", "same", "falling"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_on_both_sides_of_the_sorts(n, how, accumulate):
    embed.grad_case(n, 600, 40, how, "bf16", "f32", accumulate=accumulate)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols,pad,offset", [(1, 0, 0), (7, 0, 0), (1981, 0, 0), (33, 2, 5)])
def test_zero_rows_that_start_anywhere(dtype, cols, pad, offset):
    embed.grad_case(3, 5000, cols, "uniform", dtype, dtype, pad, offset)
