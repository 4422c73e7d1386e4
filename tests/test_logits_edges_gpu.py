"""Rows of logits at the edges of binary32, through every kernel that a call may take."""
import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import EPS32, TORCH, UNIT, assert_within, generator, randn
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
