"""The example's model: its gradients against autograd in 64 bits, training, scoring, on a stream of its own."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("small_language_model",
                                                  os.path.join(ROOT, "examples", "small_language_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def reference_loss(params, blocks, scale, tokens, ids, teacher, temperature):
    """The same step by formulas in the parameters' type."""
    table, gain = params[0], params[1]

    def norm(h, g):
        return h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * g

    h = table[tokens] * scale
    for b in range(blocks):
        g, up, down = params[2 + 3 * b:5 + 3 * b]
        h = h + torch.relu(norm(h, g) @ up) @ down
    logp = torch.log_softmax(norm(h, gain) @ table.t() / temperature, 1)
    given = ids >= 0
    rows = given.any(1)
    q = torch.softmax(torch.where(given, teacher.to(logp.dtype) / temperature, float("-inf"))[rows], 1)
    at = logp[rows].gather(1, ids.clamp(min=0)[rows])
    return torch.where(q > 0, q * (torch.log(q) - at), 0.0).sum(1).mean()


def test_gradients_against_autograd(example):
    torch.backends.cuda.matmul.allow_tf32 = False
    model = example.Model(vocab=300, dim=128, hidden=96, blocks=2, seed=1)
    tokens, ids, teacher = example.batch(300, 500, 8, 2)
    params = [p.double().requires_grad_() for p in model.parameters()]
    want = reference_loss(params, 2, model.scale, tokens, ids, teacher, 2.0)
    want.backward()
    before = [p.clone() for p in model.parameters()]
    loss = model.step(tokens, ids, teacher, temperature=2.0, rate=1.0)
    want = float(want.detach())
    assert abs(float(loss) - want) < 1e-5 * want
    for old, new, p in zip(before, model.parameters(), params):
        got = (old - new).double()  # rate 1: the step is the gradient, less the parameter's rounding
        rounding = 2.0 ** -23 * float(old.abs().max())
        # binary32 products of up to 500 terms: 1e-4 of the gradient's size is far above their rounding
        assert float((got - p.grad).abs().max()) < 1e-4 * float(p.grad.abs().max()) + rounding


def test_training_and_scoring(example):
    model = example.Model(seed=3)
    losses = [float(model.step(*example.batch(model.vocab, 2048, 8, i))) for i in range(60)]
    assert losses[-1] < 0.7 * losses[0]
    tokens, _, _ = example.batch(model.vocab, 64, 8, 999)
    following = (tokens + 1) % model.vocab
    got = model.score(tokens, following)
    assert got.top_ids.shape == (64, 5) and (got.logp <= 0).all() and (got.entropy >= 0).all()
    logits, _ = model.forward(tokens)
    exact = torch.log_softmax(logits.double(), 1).gather(1, following[:, None])[:, 0]
    # e4m3 leaves 2^-4 of each of 256 terms with a random sign: a few hundredths of a logit's spread
    assert float((got.logp.double() - exact).abs().max()) < 0.5


def test_on_another_stream(example):
    a, b = example.Model(seed=4), example.Model(seed=4)
    case = example.batch(a.vocab, 512, 8, 5)
    torch.cuda.synchronize()
    want = a.step(*case)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = b.step(*case)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(want, got)
