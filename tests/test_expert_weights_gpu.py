"""Weights and their gradient go with their plan: tokens x k, in that order."""
import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import randn

pytestmark = pytest.mark.gpu


def example(n, k):
    e = (torch.arange(n * k, device="cuda") * 7 % 5).view(n, k)
    plan = ew.ew_expert_sort(e, 5)
    return plan, randn((plan.slots.numel(), 24), 1), randn((n, 24), 2)


@pytest.mark.parametrize("n,k,shape", [(5, 2, (2, 5)), (2, 5, (5, 2)), (7, 64, (64, 7)), (7, 64, (2, 224)), (6, 4, (4, 6)),
                                       (6, 4, (3, 8)), (6, 4, (1, 4, 6, 1))])
def test_transposed_weights_are_refused(n, k, shape):
    plan, y, dout = example(n, k)
    wrong = torch.ones(shape, device="cuda")
    for call in (lambda: ew.ew_expert_combine(y, plan, wrong), lambda: ew.ew_expert_combine_grad(dout, y, plan, wrong),
                 lambda: ew.ew_expert_combine_grad(dout, y, plan, dweights=wrong)):
        with pytest.raises(ValueError, match="weights"):
            call()


@pytest.mark.parametrize("n,k", [(6, 4), (6, 1), (1, 6), (1, 1)])
def test_shapes_in_the_tokens_order_are_taken(n, k):
    plan, y, dout = example(n, k)
    w = randn((n, k), 3)
    want, (dy, dw) = ew.ew_expert_combine(y, plan, w), ew.ew_expert_combine_grad(dout, y, plan, w)
    shapes = [(n * k,), (n * k, 1), (1, n, k)] + ([(2, 3, k)] if n == 6 else []) + ([(k, n)] if 1 in (n, k) else []) + ([(2, 3)] if (n, k) == (6, 1) else [])
    for shape in shapes:
        assert torch.equal(ew.ew_expert_combine(y, plan, w.view(shape)), want)
        out = torch.full(shape, 7.0, device="cuda")
        got = ew.ew_expert_combine_grad(dout, y, plan, w.view(shape), dweights=out)
        assert torch.equal(got[0], dy) and got[1] is out and torch.equal(out.view(n, k), dw)
