"""Sizes at the ends of what the row operators take."""
import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import generator

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,accumulate", [(3, False), (40, False), (40, True)])
def test_embedding_gradient_of_many_columns(rows, accumulate):
    """More tiles of 256 columns than a grid's second dimension has; sums of small integers are exact."""
    cols = 65536 * 256 + 9
    tokens = torch.arange(rows, device="cuda") * 3 // rows * 2  # 0, 2 and 4: 1 and 3 are absent, runs cross chunks
    dout = torch.randint(-4, 5, (rows, cols), generator=generator(71), device="cuda", dtype=torch.int8).half()
    given = torch.full((5, cols), 7.0, dtype=torch.float16, device="cuda")
    got = ew.ew_embed_grad(dout, tokens, 5, dtable=given, accumulate=accumulate)
    for v in range(5):
        want = (dout[tokens == v].float().sum(0) + (7.0 if accumulate else 0.0)).half()
        assert torch.equal(got[v], want)
