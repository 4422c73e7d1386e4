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


@pytest.mark.parametrize("rows,cols", [(20000, 64), (20000, 300), (32768, 40), (32769, 40), (16384, 1024), (16353, 1001)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_gradient_on_both_sides_of_the_chunks_rule(rows, cols, accumulate):
    """Chunks of 8 and of 32 positions; sums of small integers are exact in binary32."""
    g = generator(72)
    tokens = (torch.rand(rows, generator=g, device="cuda") ** 4 * 700).long() - 1  # long runs and short ones, some absent
    dout = torch.randint(-4, 5, (rows, cols), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    given = torch.full((800, cols), 3.0, device="cuda")
    got = ew.ew_embed_grad(dout, tokens, 800, dtable=given, scale=0.5, accumulate=accumulate)
    want = torch.zeros(801, cols, dtype=torch.float64, device="cuda").index_add_(0, tokens % 801, dout.double())[:800] * 0.5
    assert torch.equal(got.double(), want + (3.0 if accumulate else 0.0))


@pytest.mark.parametrize("rows,launches", [(0, 2), (5, 2), (2000, 3)])
def test_launch_record_of_the_embedding_gradient(rows, launches):
    """The record's grid, block and shared memory are of one kernel, the sums' (which also clears the last, partial
    word of 32 rows)."""
    ew.ew_embed_grad(torch.zeros(rows, 64, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda"), 500)
    r = ew.last_launch()
    assert (r["launches"], r["block"], r["smem"]) == (launches, 256, 0)
