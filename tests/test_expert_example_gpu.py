"""The mixture of experts of the examples: its gradients against autograd in 64 bits, a run, and on a stream of its own."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("mixture_of_experts", os.path.join(ROOT, "examples", "mixture_of_experts.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def reference_loss(params, model, tokens, places, picked, advantage, old, ref, kl, low=0.2, high=0.2):
    """The same step by formulas in the parameters' type."""
    table, place_table, gain, bias = params[:4]

    def norm(h, g, b):
        d = h - h.mean(1, keepdim=True)
        return d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * g + b

    h = table[tokens] * model.scale + place_table[places]
    for i in range(len(model.blocks)):
        g, b, router, up, down = params[4 + 5 * i:9 + 5 * i]
        y = norm(h, g, b)
        scores, ids = (y @ router).topk(model.chosen, 1)
        weights = torch.softmax(scores, 1)
        total = h
        for j in range(model.chosen):
            hidden = torch.relu(torch.einsum("nd,ndh->nh", y, up[ids[:, j]]))
            total = total + weights[:, j, None] * torch.einsum("nh,nhd->nd", hidden, down[ids[:, j]])
        h = total
    every = torch.log_softmax(norm(h, gain, bias) @ table.t(), 1)
    given = picked >= 0
    logp = every.gather(1, picked.clamp(min=0)[:, None])[:, 0][given]
    ratio = torch.exp(logp - old.to(logp.dtype)[given])
    adv = advantage.to(logp.dtype)[given]
    gain_of = torch.minimum(ratio * adv, ratio.clamp(1 - low, 1 + high) * adv)
    apart = ref.to(logp.dtype)[given] - logp
    return (-gain_of + kl * (torch.exp(apart) - apart - 1)).mean()


@pytest.mark.parametrize("moved", [0.0, 0.4])
def test_gradients_against_autograd(example, moved):
    torch.backends.cuda.matmul.allow_tf32 = False
    model = example.Model(vocab=200, dim=96, hidden=64, experts=6, chosen=2, blocks=2, seed=1)
    tokens, places = example.batch(200, 300, 2)
    picked, advantage, old, _ = example.rollout(model, tokens, places, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    shift = moved * torch.randn(300, generator=g, device="cuda")
    for border in (-0.2231, 0.1823):  # log 0.8 and log 1.2: no ratio near where the gradient jumps
        shift = torch.where((shift - border).abs() < 0.01, shift + 0.02, shift)
    old, ref = old - shift, old + 0.3 * torch.randn(300, generator=g, device="cuda")
    params = [p.double().requires_grad_() for p in model.parameters()]
    want = reference_loss(params, model, tokens, places, picked, advantage, old, ref, 0.1)
    want.backward()
    before = [p.clone() for p in model.parameters()]
    loss = model.step(tokens, places, picked, advantage, old, ref, kl=0.1, rate=1.0)
    assert abs(float(loss) - float(want.detach())) < 1e-5 * (1 + abs(float(want.detach())))
    for old_p, new_p, p in zip(before, model.parameters(), params):
        got = (old_p - new_p).double()  # rate 1: the step is the gradient, less the parameter's rounding
        rounding = 2.0 ** -23 * float(old_p.abs().max())
        # binary32 products of up to 600 terms: 2e-4 of the gradient's size is far above their rounding
        assert float((got - p.grad).abs().max()) < 2e-4 * float(p.grad.abs().max()) + rounding


def test_runs_and_repeats(example):
    """A few updates of two equal models, one on another stream: finite, and the same bits."""
    models = [example.Model(seed=5), example.Model(seed=5)]
    side = torch.cuda.Stream()
    losses = []
    for model, stream in zip(models, (torch.cuda.current_stream(), side)):
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for i in range(3):
                tokens, places = example.batch(model.vocab, 512, i)
                picked, advantage, old, _ = example.rollout(model, tokens, places, 100 + i)
                for _ in range(2):
                    losses.append(model.step(tokens, places, picked, advantage, old, old))
        stream.synchronize()
    half = len(losses) // 2
    assert all(torch.isfinite(x) for x in losses)
    assert all(torch.equal(a, b) for a, b in zip(losses[:half], losses[half:]))
    assert all(torch.equal(a, b) for a, b in zip(models[0].parameters(), models[1].parameters()))
