"""Embedding lookup and its gradient on the GPU against 64 bits."""
import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import EPS32, TINY, TORCH, UNIT, Guarded, assert_within, generator, randn

pytestmark = pytest.mark.gpu


def ids(n, vocab, how, seed, dtype=torch.int64):
    g = generator(seed)
    u = torch.rand(n, generator=g, device="cuda")
    if how == "uniform":
        t = (u * vocab).long()
    elif how == "skewed":
        t = (torch.exp(u * torch.log(torch.tensor(float(vocab)))).long() - 1) * 7 % vocab
    elif how == "same":
        t = torch.full((n,), vocab - 1, device="cuda")
    elif how == "falling":
        t = torch.arange(n, 0, -1, device="cuda") % vocab
    else:
        t = torch.full((n,), -1, device="cuda")
    t = t.clamp(max=vocab - 1)
    if how in ("uniform", "skewed") and n > 4:  # no token, and ids just outside the table
        t[1], t[n // 2], t[n - 1] = -1, vocab, vocab + 7
    return t.to(dtype)


def want_rows(table, tokens, scale):
    valid = (tokens >= 0) & (tokens < table.shape[0])
    rows = table.double()[torch.where(valid, tokens, 0).long()] * scale
    return torch.where(valid[:, None], rows, 0.0)


@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,vocab,cols,pad,offset",
                         [(1, 1, 1, 0, 0), (5, 10, 8, 0, 0), (33, 100, 257, 0, 0), (64, 1000, 4096, 0, 0), (700, 50, 1000, 8, 8),
                          (3, 9, 1001, 3, 1), (20000, 300, 256, 0, 0), (9000, 300, 520, 0, 0)])
def test_lookup(itype, dtype, n, vocab, cols, pad, offset):
    table = Guarded(vocab, cols, TORCH[dtype], pad, offset, randn((vocab, cols), 1, TORCH[dtype]))
    out = Guarded(n, cols, TORCH[dtype], pad, offset)
    tokens = ids(n, vocab, "uniform", 2, itype)
    for scale in (1.0, 11.3137085):
        got = ew.ew_embed(table.t, tokens, out=out.t, scale=scale)
        want = want_rows(table.t, tokens, float(torch.tensor(scale)))
        assert got is out.t
        assert_within(got, want, (UNIT[dtype] + 2 * EPS32) * want.abs() * (scale != 1.0) + TINY[dtype] * (scale != 1.0))
    assert table.intact() and out.intact()


def test_lookup_of_infinite_rows_and_no_token():
    table = torch.full((4, 64), float("inf"), device="cuda")
    out = ew.ew_embed(table, torch.tensor([[1, -1], [4, 2]], device="cuda"), scale=float("inf"))
    assert out.shape == (2, 2, 64)
    assert torch.isinf(out[0, 0]).all() and torch.isinf(out[1, 1]).all()
    assert not out[0, 1].any() and not out[1, 0].any()


def test_lookup_past_32_bit_offsets():
    table = torch.empty(1 << 20, 4104, dtype=torch.bfloat16, device="cuda").normal_(generator=generator(3))
    tokens = torch.tensor([0, (1 << 20) - 1, 523270, 777777], device="cuda")
    assert torch.equal(ew.ew_embed(table, tokens), table[tokens])


def grad_case(n, vocab, cols, how, dtype, gtype, pad=0, offset=0, accumulate=False, itype=torch.int64, scale=0.75):
    dout = Guarded(n, cols, TORCH[dtype], pad, offset, randn((n, cols), 4, TORCH[dtype]))
    old = randn((vocab, cols), 5, TORCH[gtype])
    dtable = Guarded(vocab, cols, TORCH[gtype], pad, offset, old)
    tokens = ids(n, vocab, how, 6, itype)
    got = ew.ew_embed_grad(dout.t, tokens, vocab, dtable=dtable.t, scale=scale, accumulate=accumulate)
    assert got is dtable.t
    valid = (tokens >= 0) & (tokens < vocab)
    at = torch.where(valid, tokens.long(), vocab)
    terms = dout.t.double() * scale
    want, size = (torch.zeros(vocab + 1, cols, dtype=torch.float64, device="cuda").index_add_(0, at, v)[:-1]
                  for v in (terms, terms.abs()))
    counts = torch.bincount(at, minlength=vocab + 1)[:-1, None]
    bound = (counts + 2) * EPS32 * size
    if accumulate:
        want = want + old.double()
        bound = bound + EPS32 * want.abs()
        named = counts[:, 0] > 0
        assert torch.equal(got[~named], old[~named])  # rows that no token names are not touched
        bound = torch.where(named[:, None], bound + UNIT[gtype] * want.abs() + TINY[gtype], bound)
    else:
        bound = bound + UNIT[gtype] * (want.abs() + bound) + TINY[gtype] * (counts > 0)
    assert_within(got, want, bound, "dtable")
    assert dout.intact() and dtable.intact()


@pytest.mark.parametrize("dtype,gtype", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n,vocab,cols,how",
                         [(1, 1, 1, "same"), (31, 7, 8, "uniform"), (32, 7, 64, "same"), (33, 40, 257, "same"),
                          (64, 3, 24, "falling"), (100, 1000, 1000, "uniform"), (1000, 33, 256, "skewed"),
                          (1025, 1024, 96, "skewed"), (5003, 32003, 100, "skewed"), (300, 5, 16, "none")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(dtype, gtype, n, vocab, cols, how, accumulate):
    grad_case(n, vocab, cols, how, dtype, gtype, accumulate=accumulate)


@pytest.mark.parametrize("n,vocab,cols,how",
                         [(70001, 70000, 40, "skewed"), (70000, 5, 8, "uniform"), (66000, 9, 300, "same"),
                          (5000, (1 << 20) + 5, 16, "skewed"), (40000, 1 << 20, 8, "falling"), (3, 1 << 22, 8, "uniform")])
def test_gradient_long(n, vocab, cols, how):
    grad_case(n, vocab, cols, how, "bf16", "f32")


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("pad,offset,itype", [(3, 1, torch.int32), (8, 8, torch.int32), (0, 3, torch.int64)])
def test_gradient_of_strided_rows(pad, offset, itype, accumulate):
    grad_case(777, 100, 520, "skewed", "f16", "f16", pad, offset, accumulate, itype)


def test_gradient_against_differences():
    """sum(dout * out) is linear in the table: its differences over a step of 2^-4 are exact up to 64-bit roundings."""
    table, dout = randn((6, 9), 7), randn((20, 9), 8)
    tokens = ids(20, 6, "uniform", 9)
    got = ew.ew_embed_grad(dout, tokens, 6, scale=0.5)

    def loss(t):
        return float((dout.double() * want_rows(t, tokens, 0.5)).sum())

    for k in range(0, 54, 7):
        moved = table.double().clone()
        moved.view(-1)[k] += 2.0 ** -4
        assert abs((loss(moved) - loss(table.double())) * 16 - float(got.view(-1)[k])) < 1e-5


def test_nothing_to_do():
    tokens = torch.empty(0, dtype=torch.int64, device="cuda")
    dout = torch.empty(0, 24, device="cuda")
    assert ew.ew_embed(torch.ones(3, 24, device="cuda"), tokens).shape == (0, 24)
    assert not ew.ew_embed_grad(dout, tokens, 70, dtable=torch.ones(70, 24, device="cuda")).any()
    kept = torch.ones(70, 24, device="cuda")
    assert ew.ew_embed_grad(dout, tokens, 70, dtable=kept, accumulate=True).all()


def test_repeats_bit_for_bit_and_in_a_graph():
    dout, tokens = randn((9000, 264), 10, torch.bfloat16), ids(9000, 500, "skewed", 11)
    want = ew.ew_embed_grad(dout, tokens, 500, dtable=torch.empty(500, 264, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = ew.ew_embed_grad(dout, tokens, 500, dtable=torch.empty(500, 264, device="cuda"), stream=side)
        side.synchronize()
        assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ew.ew_embed_grad(dout, tokens, 500, dtable=torch.empty(500, 264, device="cuda"))
    tokens.copy_(ids(9000, 500, "uniform", 12))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, ew.ew_embed_grad(dout, tokens, 500, dtable=torch.empty(500, 264, device="cuda")))


def test_refusals():
    table, tokens = torch.zeros(8, 64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    dout = torch.zeros(4, 64, device="cuda")
    with pytest.raises(TypeError):
        ew.ew_embed(table, tokens.short())
    with pytest.raises(ValueError):
        ew.ew_embed(table, tokens.cpu())
    with pytest.raises(TypeError):
        ew.ew_embed(table.long(), tokens)
    with pytest.raises(ew.EwError, match="OVERLAP"):
        ew.ew_embed(table, tokens, out=table[:4])
    with pytest.raises(ValueError):
        ew.ew_embed_grad(dout, tokens[:3], 8)
    with pytest.raises(ValueError):
        ew.ew_embed_grad(dout, tokens, 8, accumulate=True)
    with pytest.raises(TypeError):
        ew.ew_embed_grad(dout, tokens, 8, dtable=table.half())
    with pytest.raises(ValueError):
        ew.ew_embed_grad(dout, tokens, 9, dtable=table)
