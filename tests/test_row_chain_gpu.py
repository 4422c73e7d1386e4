"""Layer norm, routing and the policy loss one after another on a stream, with programmatic launch on and off, each on what
the one before has just written, and in a graph that is replayed on other inputs."""
import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import TORCH, generator, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def restored():
    yield
    ew.set_programmatic_launch(1)


def chain(s, between=lambda: None):
    out = []

    def step(*tensors):
        out.extend(t for t in tensors if t is not None)
        between()
        return tensors

    n, experts = s["x"].shape[0], s["router"].shape[1]
    y, h, mean, rstd = step(*ew.ew_layernorm(s["x"], s["weight"], s["bias"], residual=s["residual"]))
    scores = (y[:, :experts].float() * 0.3 + s["router"]).contiguous()
    best = ew.ew_logprob(scores, None, top=3)
    plan = ew.ExpertPlan(*step(*ew.ew_expert_sort(best.top_ids, experts, align=s["align"])))
    weights = best.top_logp.exp()
    rows, = step(ew.ew_expert_dispatch(y, plan))
    back, = step(ew.ew_expert_combine(rows, plan, weights, residual=h))
    logits = back.view(s["rows"], -1)
    loss, logp, lse, d = step(*ew.ew_policy_step(logits, s["picked"], s["advantage"], s["dloss"], old_logp=s["old"], ref_logp=s["ref"],
                                                 kl=0.1, scale=0.5))
    step(*ew.ew_policy(logits, s["picked"], s["advantage"], old_logp=logp, ref_logp=s["ref"], kl=0.1, scale=0.5))
    d2, = step(ew.ew_policy_grad(logits, s["picked"], s["advantage"], logp, lse, s["dloss"], old_logp=s["old"], scale=0.5))
    dout = d.view(n, -1)
    dy, dw = step(*ew.ew_expert_combine_grad(dout, rows, plan, weights))
    dx, = step(ew.ew_expert_combine(dy, plan, residual=d2.view(n, -1)))
    step(*ew.ew_layernorm_grad(dx, h, s["weight"], mean, rstd, dh=dout))
    return out


def inputs(dtype, rows, cols, per, seed):
    kind, n = TORCH[dtype], rows * per
    s = dict(rows=rows, align=8, x=randn((n, cols), seed, kind), residual=randn((n, cols), seed + 1, kind, 2.0),
             weight=randn((cols,), seed + 2), bias=randn((cols,), seed + 3), router=randn((n, 16), seed + 4),
             picked=torch.randint(0, cols * per, (rows,), generator=generator(seed + 5), device="cuda"),
             advantage=randn((rows,), seed + 6), dloss=randn((rows,), seed + 7), old=randn((rows,), seed + 8) - 9.0,
             ref=randn((rows,), seed + 9) - 9.0)
    s["picked"][::3] = -1
    return s


def same(got, want):
    return len(got) == len(want) and all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
                                         for a, b in zip(got, want))


# cols of each kind: aligned, anywhere, rows held in shared memory, several blocks a row
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,per", [(12, 512, 3), (700, 2048, 2), (64, 5001, 8), (200, 1003, 16)])
def test_chain_with_programmatic_launch_on_and_off(dtype, rows, cols, per):
    s = inputs(dtype, rows, cols, per, 200)
    ew.set_programmatic_launch(0)
    want = chain(s, torch.cuda.synchronize)
    torch.cuda.synchronize()
    for enabled in (0, 1):
        ew.set_programmatic_launch(enabled)
        for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
            stream.wait_stream(torch.cuda.current_stream())
            for _ in range(3):
                with torch.cuda.stream(stream):
                    got = chain(s)
                stream.synchronize()
                assert same(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_chain_in_a_graph(dtype):
    s = inputs(dtype, 64, 5001, 8, 220)
    chain(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain(s)
    for seed in (240, 260):
        for key, value in inputs(dtype, 64, 5001, 8, seed).items():
            if isinstance(value, torch.Tensor):
                s[key].copy_(value)
        for _ in range(2):
            g.replay()
            torch.cuda.synchronize()
            assert same(got, chain(s))


def test_calls_with_a_stream_argument():
    """The same by the calls' own stream argument, from another current stream."""
    s = inputs("bf16", 12, 512, 3, 280)
    want = chain(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, h, mean, rstd = ew.ew_layernorm(s["x"], s["weight"], s["bias"], residual=s["residual"], stream=side)
    side.synchronize()
    scores = (y[:, :16].float() * 0.3 + s["router"]).contiguous()
    best = ew.ew_logprob(scores, None, top=3)
    weights = best.top_logp.exp()
    torch.cuda.synchronize()
    plan = ew.ew_expert_sort(best.top_ids, 16, align=8, stream=side)
    rows = ew.ew_expert_dispatch(y, plan, stream=side)
    back = ew.ew_expert_combine(rows, plan, weights, residual=h, stream=side)
    logits = back.view(12, -1)
    how = dict(old_logp=s["old"], ref_logp=s["ref"], kl=0.1, scale=0.5, stream=side)
    loss, logp, lse, d = ew.ew_policy_step(logits, s["picked"], s["advantage"], s["dloss"], **how)
    again = ew.ew_policy(logits, s["picked"], s["advantage"], old_logp=logp, ref_logp=s["ref"], kl=0.1, scale=0.5, stream=side)
    d2 = ew.ew_policy_grad(logits, s["picked"], s["advantage"], logp, lse, s["dloss"], old_logp=s["old"], scale=0.5, stream=side)
    dout = d.view(36, -1)
    dy, dw = ew.ew_expert_combine_grad(dout, rows, plan, weights, stream=side)
    dx = ew.ew_expert_combine(dy, plan, residual=d2.view(36, -1), stream=side)
    last = ew.ew_layernorm_grad(dx, h, s["weight"], mean, rstd, dh=dout, stream=side)
    side.synchronize()
    assert same([y, h, mean, rstd, *plan, rows, back, loss, logp, lse, d, *again, d2, dy, dw, dx, *last], want)
