"""Log probabilities, distillation and their gradients on the GPU against 64 bits."""
import math

import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import EPS32, TINY, TORCH, UNIT, Guarded, assert_within, generator, randn

pytestmark = pytest.mark.gpu

# rows, cols, pad, offset: fewer than a chunk, chunk edges, rows that start anywhere, a row to one block (many rows)
# and to clusters of 2 to 8 (few rows of at least 8192 columns), more than one turn of the stream
SHAPES = [(1, 1, 0, 0), (3, 5, 0, 1), (2, 8, 0, 0), (4, 100, 0, 0), (3, 1000, 24, 8), (2, 4097, 0, 0), (5, 8192, 0, 0),
          (3, 16387, 0, 3), (2, 50001, 0, 0), (1, 131072, 0, 0), (320, 3001, 0, 0), (310, 20000, 8, 0), (40, 33333, 0, 0)]


def logits_of(rows, cols, dtype, pad, offset, seed, spread=3.0):
    return Guarded(rows, cols, TORCH[dtype], pad, offset, randn((rows, cols), seed, TORCH[dtype], spread))


def some_tokens(rows, cols, seed, dtype=torch.int64):
    t = torch.randint(0, cols, (rows,), generator=generator(seed), device="cuda")
    if rows > 2:
        t[1], t[rows - 1] = -1, cols  # no token
    return t.to(dtype)


def sum_bound(x, scale):
    """Absolute error of a row's lse (relative error of its sum): exponents formed with two binary32 roundings of
    up to |x scale log2 e|, 2^-22 of the exponential, and cols / 512 terms a thread before a tree."""
    size = torch.where(torch.isfinite(x), x, 0.0).abs().amax(1) * scale
    return EPS32 * (x.shape[1] / 512 + 128 + 6 * size)


class Want:
    """A row's results in 64 bits."""

    def __init__(self, x, scale):
        self.x = x.double() * scale
        self.empty = torch.isneginf(self.x).all(1)
        self.lse = torch.logsumexp(self.x, 1)
        safe = torch.where(self.empty, 0.0, self.lse)
        self.logp = torch.where(self.empty[:, None], -math.inf, self.x - safe[:, None])
        self.p = torch.exp(self.logp)
        self.entropy = torch.special.entr(self.p).sum(1)
        self.bound = sum_bound(x.double(), scale)
        # the entropy's sum is of p times the distance to the largest element
        top = self.x.amax(1, keepdim=True)
        spread = torch.where(self.p > 0, self.p * (top - self.x), 0.0).sum(1)
        self.entropy_bound = self.bound * (3 + spread)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_logprob(dtype, rows, cols, pad, offset):
    x = logits_of(rows, cols, dtype, pad, offset, 1)
    if cols > 50:
        x.t[:, ::3] = -math.inf
    scale = 1.0 if rows % 2 else 0.7
    tokens = some_tokens(rows, cols, 2, torch.int32 if cols % 2 else torch.int64)
    top = (rows + cols) % 65
    got = ew.ew_logprob(x.t, tokens, top=top, scale=scale)
    want = Want(x.t, float(torch.tensor(scale)))
    assert_within(got.lse, want.lse, want.bound + 2 * EPS32 * want.lse.abs(), "lse")
    assert_within(got.entropy, want.entropy, want.entropy_bound + 2 * EPS32 * want.entropy, "entropy")
    given = (tokens >= 0) & (tokens < cols)
    at = want.logp.gather(1, torch.where(given, tokens, 0).long()[:, None])[:, 0]
    at = torch.where(given, at, 0.0)
    assert_within(got.logp, at, (want.bound + 4 * EPS32 * at.abs()) * given, "logp")
    check_top(got, x.t, want, top)
    assert x.intact()


def check_top(got, x, want, top):
    best, ids = torch.sort(x.double(), dim=1, descending=True, stable=True)
    best, ids = best[:, :top], ids[:, :top]
    missing = torch.isneginf(best)
    n = best.shape[1]
    assert torch.equal(got.top_ids[:, :n].long(), torch.where(missing, -1, ids))
    assert (got.top_ids[:, n:] == -1).all() and torch.isneginf(got.top_logp[:, n:]).all()
    logp = torch.where(missing, -math.inf, want.logp.gather(1, ids))
    assert_within(got.top_logp[:, :n], logp, want.bound[:, None] + 4 * EPS32 * torch.where(missing, 0.0, logp).abs(), "top")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(6, 70000), (320, 9001), (4, 300)])
@pytest.mark.parametrize("how", ["rising", "falling", "constant", "few values", "steps", "three left", "lowest"])
def test_top_with_ties_and_order(dtype, rows, cols, how):
    """Orders and ties that make many elements candidates at once."""
    j = torch.arange(cols, device="cuda", dtype=torch.float32)
    lowest = torch.finfo(TORCH[dtype]).min
    x = {"rising": j / cols * 8, "falling": -j / cols * 8, "constant": torch.full_like(j, 1.5),
         "few values": (j * 7919 % 5).floor(), "steps": (j / 3000).floor(),
         "three left": torch.where(j % (cols // 3) == 5, j / cols, -math.inf),
         "lowest": torch.where(j % (cols // 3) == 5, j / cols, lowest)}[how]
    x = x.to(TORCH[dtype]).repeat(rows, 1)
    for top in (1, 20, 64):
        got = ew.ew_logprob(x, None, top=top)
        assert got.logp is None
        want = Want(x, 1.0)
        want.bound = sum_bound(torch.where(x == lowest, 0.0, x.double()), 1.0)
        check_top(got, x, want, top) if how != "lowest" else check_top(got, x, lowest_kept(want, x, lowest), top)
        again = ew.ew_logprob(x, None, top=top)
        assert torch.equal(got.top_ids, again.top_ids) and torch.equal(got.lse, again.lse)


def lowest_kept(want, x, lowest):
    # log p of the type's lowest value is as large as the value itself: compared in its own size
    want.bound = want.bound + EPS32 * 4 * torch.where(x == lowest, x.double().abs(), 0.0).amax(1)
    return want


def special_rows(dtype, cols):
    lowest, largest = torch.finfo(TORCH[dtype]).min, torch.finfo(TORCH[dtype]).max
    x = randn((12, cols), 3, TORCH[dtype])
    x[0] = -math.inf
    x[1] = lowest
    x[2] = -math.inf
    x[2, cols // 2] = 2.5                     # a single element left
    x[3, cols // 3] = math.nan
    x[4, cols - 1] = math.inf
    x[5] = lowest
    x[5, 1], x[5, cols - 2] = 1.0, 2.0        # masked by the lowest value
    x[6] = -math.inf
    x[6, 0], x[6, cols - 1] = lowest, lowest  # uniform over two
    x[7] = largest
    x[8, 0] = largest                         # one huge value
    x[9] = 0.0
    x[10] = -math.inf
    x[10, 3] = lowest
    x[11] *= 30000.0 if dtype != "f16" else 1.0
    return x


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [100, 4099, 70001])
def test_special_rows(dtype, cols):
    x = special_rows(dtype, cols)
    tokens = torch.zeros(12, dtype=torch.int64, device="cuda")
    tokens[2], tokens[6], tokens[10] = cols // 2, cols - 1, 3
    got = ew.ew_logprob(x, tokens, top=3)
    n = math.log(cols)
    for row in (3, 4):
        assert all(torch.isnan(v[row]).all() for v in (got.logp, got.entropy, got.lse, got.top_logp))
        assert (got.top_ids[row] == -1).all()
    assert torch.isneginf(got.lse[0]) and torch.isneginf(got.logp[0]) and got.entropy[0] == 0
    assert (got.top_ids[0] == -1).all() and torch.isneginf(got.top_logp[0]).all()
    tol = 1e-4  # of values near log(cols); far above any rounding, far below a lost element
    for row in (1, 7, 9):  # uniform
        assert abs(float(got.logp[row]) + n) < tol and abs(float(got.entropy[row]) - n) < tol
        assert got.top_ids[row].tolist() == [0, 1, 2]
    for row in (2, 10):
        assert float(got.logp[row]) == 0 and abs(float(got.entropy[row])) < tol
        assert got.top_ids[row, 0] == tokens[row] and (got.top_ids[row, 1:] == -1).all()
    assert abs(float(got.entropy[5]) - 0.5822032) < tol and got.top_ids[5].tolist() == [cols - 2, 1, 0]
    assert abs(float(got.logp[6]) + math.log(2)) < tol and abs(float(got.entropy[6]) - math.log(2)) < tol
    assert float(got.logp[8]) == 0 and got.entropy[8] == 0
    want = Want(x[11:], 1.0)
    assert_within(got.lse[11:], want.lse, want.bound + 2 * EPS32 * want.lse.abs(), "spread row")


def check_logprob_grad(x, tokens, scale, dlogp, dent, got, dtype):
    want = Want(x, float(torch.tensor(scale)))
    given = (tokens >= 0) & (tokens < x.shape[1])
    a = torch.where(given, dlogp.double(), 0.0) if dlogp is not None else torch.zeros(x.shape[0], device="cuda").double()
    b = dent.double() if dent is not None else torch.zeros_like(a)
    one = torch.zeros_like(want.p)
    one[torch.arange(len(a), device="cuda")[given], tokens[given].long()] = 1.0
    away = torch.where(want.p > 0, want.logp + want.entropy[:, None], 0.0)
    d = scale * (a[:, None] * (one - want.p) - b[:, None] * want.p * away)
    # lse is given in binary32: its rounding and the exponent's make p relatively off by the bound
    e = (want.bound + 4 * EPS32 * want.lse.abs() + want.entropy_bound)[:, None]
    size = scale * want.p * (a.abs()[:, None] + b.abs()[:, None] * (away.abs() + 1))
    bound = UNIT[dtype] * d.abs() + e * size + 4 * EPS32 * scale * a.abs()[:, None] * one + TINY[dtype]
    assert_within(got, d, bound, "dlogits")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
@pytest.mark.parametrize("terms", ["both", "logp", "entropy"])
def test_logprob_gradient(dtype, rows, cols, pad, offset, terms):
    x = logits_of(rows, cols, dtype, pad, offset, 4)
    if cols > 50:
        x.t[:, ::3] = -math.inf
    tokens = some_tokens(rows, cols, 5)
    tokens[0] = cols - 1
    f = ew.ew_logprob(x.t, tokens, scale=0.8)
    dlogp = randn((rows,), 6) if terms != "entropy" else None
    dent = randn((rows,), 7) if terms != "logp" else None
    # the output starts elsewhere from 16 bytes than the input in half of the cases
    out = Guarded(rows, cols, TORCH[dtype], pad, offset if rows % 2 else offset + 1)
    got = ew.ew_logprob_grad(x.t, tokens, f.lse, f.entropy, dlogp, dent, scale=0.8, dlogits=out.t)
    assert got is out.t
    check_logprob_grad(x.t, tokens, 0.8, dlogp, dent, got, dtype)
    assert x.intact() and out.intact()
    kept = x.t.clone()
    ew.ew_logprob_grad(x.t, tokens, f.lse, f.entropy, dlogp, dent, scale=0.8, dlogits=x.t)  # in place
    assert torch.equal(x.t, got) and not torch.equal(x.t, kept)


def test_logprob_gradient_of_special_rows():
    x = special_rows("f32", 4099)
    tokens = torch.ones(12, dtype=torch.int64, device="cuda")
    f = ew.ew_logprob(x, tokens)
    one = torch.ones(12, device="cuda")
    d = ew.ew_logprob_grad(x, tokens, f.lse, f.entropy, one, one)
    assert not d[0].any()                                    # nothing depends on an empty row
    assert torch.isnan(d[3]).all() and torch.isnan(d[4]).all()
    for row in (2, 5, 6, 8, 9, 10, 11):
        assert torch.isfinite(d[row]).all()
    assert not d[5][2:4097].any()                            # masked elements have no gradient


def test_logprob_gradient_against_differences():
    """Central differences in 64 bits of sum(dlogp logp + dent H); step 1e-5, as precise as 1e-9."""
    x, tokens = randn((3, 21), 8), torch.tensor([0, 20, 7], device="cuda")
    dlogp, dent = randn((3,), 9), randn((3,), 10)
    f = ew.ew_logprob(x, tokens, scale=1.5)
    got = ew.ew_logprob_grad(x, tokens, f.lse, f.entropy, dlogp, dent, scale=1.5)

    def loss(v):
        w = Want(v, 1.5)
        return float((dlogp.double() * w.logp.gather(1, tokens[:, None])[:, 0] + dent.double() * w.entropy).sum())

    for k in range(0, 63, 4):
        up, down = x.double().clone(), x.double().clone()
        up.view(-1)[k] += 1e-5
        down.view(-1)[k] -= 1e-5
        assert abs((loss(up) - loss(down)) / 2e-5 - float(got.view(-1)[k])) < 1e-5


def teacher_case(rows, cols, k, dtype, seed, itype=torch.int64):
    k = min(k, cols)
    g = generator(seed)
    start = torch.randint(0, cols, (rows, 1), generator=g, device="cuda")
    ids = (start + torch.arange(k, device="cuda") * max(1, cols // k)) % cols
    if rows > 2 and k > 2:
        ids[0, k // 2:] = -1       # fewer than k
        ids[1] = -1                # none
        ids[2, 1], ids[2, k - 1] = cols + 3, ids[2, 0]  # outside, and one id twice
    t = randn((rows, k), seed + 1, dtype, 3.0)
    if rows > 3:
        t[3, 0] = -math.inf
    return ids.to(itype), t


def want_distill(x, ids, t, scale, dloss):
    w = Want(x, scale)
    rows, k = ids.shape
    given = (ids >= 0) & (ids < x.shape[1]) & ~torch.isneginf(t)
    v = torch.where(given, t.double() * scale, -math.inf)
    some = given.any(1)
    logq = torch.where(given, v - torch.where(some, torch.logsumexp(v, 1), 0.0)[:, None], 0.0)
    q = torch.where(given, torch.exp(logq), 0.0)
    at = torch.where(given, ids, 0).long()
    logp = w.logp.gather(1, at)
    terms = torch.where(q > 0, q * (logq - logp), 0.0)
    dense = torch.zeros_like(w.p).scatter_add_(1, at, q)
    g = dloss.double() * scale
    d = g[:, None] * (w.p * some[:, None] - dense)
    size_t = torch.where(given, v, 0.0).abs().amax(1)
    e_q = EPS32 * (k + 32 + 4 * size_t)
    loss_bound = w.bound + e_q * (1 + torch.where(q > 0, q * (logq.abs() + torch.nan_to_num(logp, neginf=0.0).abs()), 0.0).sum(1))
    d_bound = g.abs()[:, None] * (w.p * (w.bound + 4 * EPS32 * w.lse.abs())[:, None] + dense * e_q[:, None])
    return terms.sum(1), w, d, loss_bound * some, d_bound * some[:, None]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
@pytest.mark.parametrize("k", [1, 17, 300])
def test_distill(dtype, rows, cols, pad, offset, k):
    x = logits_of(rows, cols, dtype, pad, offset, 11)
    ids, t = teacher_case(rows, cols, k, TORCH[dtype] if k != 17 else torch.float32, 12, torch.int32 if k == 1 else torch.int64)
    scale, dloss = 0.5, randn((rows,), 14)
    out = Guarded(rows, cols, TORCH[dtype], pad, offset if cols % 2 else offset + 1)
    loss, lse, d = ew.ew_distill_step(x.t, ids, t, dloss, scale=scale, dlogits=out.t)
    want_loss, w, want_d, loss_bound, d_bound = want_distill(x.t, ids, t, scale, dloss)
    assert_within(lse, w.lse, w.bound + 2 * EPS32 * w.lse.abs(), "lse")
    assert_within(loss, want_loss, loss_bound, "loss")
    assert_within(d, want_d, UNIT[dtype] * want_d.abs() + d_bound + TINY[dtype] * (want_d != 0), "dlogits")
    assert x.intact() and out.intact()
    # the two halves alone: the same loss bit for bit, the gradient within the same bounds
    loss2, lse2 = ew.ew_distill(x.t, ids, t, scale=scale)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    d2 = ew.ew_distill_grad(x.t, ids, t, lse, dloss, scale=scale)
    assert_within(d2, want_d, UNIT[dtype] * want_d.abs() + d_bound + TINY[dtype] * (want_d != 0), "dlogits from lse")
    ew.ew_distill_grad(x.t.clone(), ids, t, lse, dloss, scale=scale)
    same = x.t.clone()
    ew.ew_distill_grad(same, ids, t, lse, dloss, scale=scale, dlogits=same)
    assert torch.equal(same, d2)
    ew.ew_distill_step(x.t, ids, t, dloss, scale=scale, dlogits=x.t)
    assert torch.equal(x.t, d)


@pytest.mark.parametrize("cols", [100, 70001])
def test_distill_special_rows(cols):
    x = special_rows("bf16", cols)
    ids = torch.tensor([[5, 9, -1]], device="cuda").repeat(12, 1)
    ids[2], ids[10] = cols // 2, 3  # one id three times
    t = torch.tensor([[1.0, 2.0, 3.0]], device="cuda").repeat(12, 1)
    one = torch.ones(12, device="cuda")
    for place in (None, x.clone()):
        if place is None:
            loss, lse, d = ew.ew_distill_step(x, ids, t, one)
        else:
            loss, lse, d = ew.ew_distill_step(place, ids, t, one, dlogits=place)
        q = 1 / (1 + math.e)
        assert torch.isneginf(lse[0]) and torch.isposinf(loss[0])  # the teacher's tokens are masked
        assert abs(float(d[0, 5]) + q) < 2e-3 and abs(float(d[0, 9]) + 1 - q) < 4e-3 and not d[0, 10:].any()
        assert torch.isnan(loss[3]) and torch.isnan(loss[4]) and torch.isnan(d[3]).all() and torch.isnan(d[4]).all()
        uniform = math.log(cols) + q * math.log(q) + (1 - q) * math.log(1 - q)
        for row in (1, 7, 9):
            assert abs(float(loss[row]) - uniform) < 1e-4
            assert abs(float(d[row, 20]) - 1 / cols) < 2.0 ** -8 / cols
        entropy = 0.8323956  # of softmax(1, 2, 3), each entry its own term: the loss is sum q log q, as log p = 0
        for row in (2, 10):
            assert abs(float(loss[row]) + entropy) < 1e-5 and float(d[row].abs().max()) < 1e-5
        assert torch.isfinite(d[5:]).all()


def test_distill_against_differences():
    x, dloss = randn((2, 30), 15), randn((2,), 16)
    ids, t = torch.tensor([[3, 4, 29], [0, -1, 7]], device="cuda"), randn((2, 3), 17)
    _, _, d = ew.ew_distill_step(x, ids, t, dloss, scale=0.5)

    def loss(v):
        return float((want_distill(v, ids, t, 0.5, dloss)[0] * dloss.double()).sum())

    for k in range(60):
        up, down = x.double().clone(), x.double().clone()
        up.view(-1)[k] += 1e-5
        down.view(-1)[k] -= 1e-5
        assert abs((loss(up) - loss(down)) / 2e-5 - float(d.view(-1)[k])) < 1e-5


def test_strided_teacher_and_no_rows():
    x = randn((4, 64), 18)
    ids, t = teacher_case(4, 64, 8, torch.float32, 19)
    wide_ids, wide_t = torch.full((4, 20), 7, device="cuda"), torch.full((4, 11), 50.0, device="cuda")
    wide_ids[:, 3:11], wide_t[:, 2:10] = ids, t
    a = ew.ew_distill(x, ids, t)
    b = ew.ew_distill(x, wide_ids[:, 3:11], wide_t[:, 2:10])
    assert torch.equal(a[0], b[0])
    none = x[:0]
    assert ew.ew_logprob(none, torch.empty(0, dtype=torch.int64, device="cuda"), top=4).top_ids.shape == (0, 4)
    assert ew.ew_distill(none, ids[:0], t[:0])[0].shape == (0,)


def test_past_32_bit_offsets():
    rows, cols = 17000, 131072
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = randn((cols,), 20, torch.bfloat16)
    tokens = torch.full((rows,), 5, device="cuda")
    got = ew.ew_logprob(x, tokens, top=2)
    want = Want(x[-1:], 1.0)
    assert_within(got.lse[-1:], want.lse, want.bound + 2 * EPS32 * want.lse.abs())
    f = ew.ew_logprob_grad(x, tokens, got.lse, None, torch.ones(rows, device="cuda"), dlogits=x)
    assert abs(float(f[-1, 5]) - (1 - float(want.p[0, 5]))) < 2.0 ** -7 and float(f[-1, 6]) < 0 and float(f[0, 5]) == 1


def test_repeats_bit_for_bit_and_in_a_graph():
    x = randn((33, 40000), 21, torch.bfloat16)
    tokens, dloss = some_tokens(33, 40000, 22), randn((33,), 23)
    ids, t = teacher_case(33, 40000, 64, torch.bfloat16, 24)

    def both():
        return (*ew.ew_logprob(x, tokens, top=20), *ew.ew_distill_step(x, ids, t, dloss))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*ew.ew_logprob(x, tokens, top=20, stream=side), *ew.ew_distill_step(x, ids, t, dloss, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both()
    x.copy_(randn(x.shape, 25, torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, both()))


def test_refusals():
    x, tokens = torch.zeros(4, 64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    each = torch.zeros(4, device="cuda")
    for bad in (0.0, -1.0, math.nan, math.inf, 2.0 ** 21, 2.0 ** -21):
        with pytest.raises(ew.EwError, match="INVALID"):
            ew.ew_logprob(x, tokens, scale=bad)
    with pytest.raises(ew.EwError, match="INVALID"):
        ew.ew_logprob(x, tokens, top=65)
    with pytest.raises(ValueError):
        ew.ew_logprob(x, tokens[:3])
    with pytest.raises(TypeError):
        ew.ew_logprob(x, tokens.float())
    with pytest.raises(ValueError):
        ew.ew_logprob_grad(x, tokens, each[:3], None, each)
    with pytest.raises(ew.EwError, match="OVERLAP"):
        ew.ew_logprob_grad(x[:3], tokens[:3], each[:3], None, each[:3], dlogits=x[1:])
    ids = torch.zeros(4, 3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        ew.ew_distill(x, ids, x[:, :2])
    with pytest.raises(TypeError):
        ew.ew_distill(x, ids, x[:, :3].half())
    with pytest.raises(ValueError):
        ew.ew_distill(x, ids[:2], x[:2, :3])
    with pytest.raises(ew.EwError, match="INVALID"):
        ew.ew_distill(x, torch.zeros(4, 1025, dtype=torch.int64, device="cuda"), torch.zeros(4, 1025, device="cuda"))
