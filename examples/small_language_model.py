"""The row operators together: a small language model trained by distillation, then scored.

The model is an embedding, a few blocks of norm, two products and ReLU on the
residual stream, a last norm, and logits against the embedding table itself.
Its memory-bound steps run in this library: the lookup and its gradient, the
norms with the residual's addition and their gradients, ReLU, the distillation
loss with its gradient, and the update (SAXPY).  The products are torch's.

    python examples/small_language_model.py [--steps 60]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_bound_elementwise_gb300 as ew  # noqa: E402


class Model:
    def __init__(self, vocab=1000, dim=256, hidden=512, blocks=2, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, spread):
            return torch.randn(*shape, generator=g, device=device) * spread

        self.vocab, self.scale = vocab, math.sqrt(dim)
        self.table = normal(vocab, dim, spread=1.0 / self.scale)
        self.blocks = [dict(gain=torch.ones(dim, device=device), up=normal(dim, hidden, spread=dim ** -0.5),
                            down=normal(hidden, dim, spread=hidden ** -0.5)) for _ in range(blocks)]
        self.gain = torch.ones(dim, device=device)

    def parameters(self):
        return [self.table, self.gain] + [p for b in self.blocks for p in (b["gain"], b["up"], b["down"])]

    def forward(self, tokens):
        """Logits of each token, and what the backward pass needs."""
        x, residual, saved = ew.ew_embed(self.table, tokens, scale=self.scale), None, []
        for b in self.blocks:
            y, h, rstd = ew.ew_rmsnorm(x, b["gain"], residual=residual)
            a = ew.ew_relu(y @ b["up"])
            saved.append((y, h, rstd, a))
            x, residual = a @ b["down"], h
        y, h, rstd = ew.ew_rmsnorm(x, self.gain, residual=residual)
        return y @ self.table.t(), (saved, (y, h, rstd))

    def backward(self, tokens, dlogits, kept):
        """The parameters' gradients, in the order of parameters()."""
        saved, (y, h, rstd) = kept
        dtable = dlogits.t() @ y
        dh, dgain = ew.ew_rmsnorm_grad(dlogits @ self.table, h, self.gain, rstd)
        grads = []
        for b, (y, h, rstd, a) in zip(reversed(self.blocks), reversed(saved)):
            da = (dh @ b["down"].t()).masked_fill_(a == 0, 0.0)
            ddown, dup = a.t() @ dh, y.t() @ da
            # the residual's gradient joins the one through the norm
            dh, dg = ew.ew_rmsnorm_grad(da @ b["up"].t(), h, b["gain"], rstd, dh=dh)
            grads = [dg, dup, ddown] + grads
        # the table is the embedding too: its gradient is added to the logits'
        ew.ew_embed_grad(dh, tokens, self.vocab, dtable=dtable, scale=self.scale, accumulate=True)
        return [dtable, dgain] + grads

    def step(self, tokens, ids, teacher, temperature=2.0, rate=2.0):
        """One step of distillation on ``tokens``; returns the mean loss before it."""
        logits, kept = self.forward(tokens)
        given = (ids >= 0).any(1)
        dloss = given.float() / given.sum()
        # the gradient takes the logits' place
        loss, _, dlogits = ew.ew_distill_step(logits, ids, teacher, dloss, scale=1.0 / temperature, dlogits=logits)
        for p, g in zip(self.parameters(), self.backward(tokens, dlogits, kept)):
            ew.ew_saxpy(-rate, g, p)
        return (loss * dloss).sum()

    def score(self, tokens, following, top=5):
        """Log probabilities of the tokens that follow, the entropy and the likeliest alternatives.

        The last norm's output is taken in 8 bits, as a product in 8 bits would take it."""
        x, residual = ew.ew_embed(self.table, tokens, scale=self.scale), None
        for b in self.blocks:
            y, residual, _ = ew.ew_rmsnorm(x, b["gain"], residual=residual)
            x = ew.ew_relu(y @ b["up"]) @ b["down"]
        q, scales, _, _ = ew.ew_rmsnorm_quant(x, self.gain, residual=residual, group=64)
        y = (q.float().unflatten(1, (-1, 64)) * scales[:, :, None]).flatten(1)
        return ew.ew_logprob(y @ self.table.t(), following, top=top)


def batch(vocab, n, k, seed, device="cuda"):
    """Tokens, and a teacher that prefers the tokens after each one's; a tenth of the rows has none."""
    g = torch.Generator(device=device).manual_seed(seed)
    tokens = torch.randint(0, vocab, (n,), generator=g, device=device)
    ids = (tokens[:, None] + 1 + torch.arange(k, device=device)) % vocab
    ids[torch.rand(n, generator=g, device=device) < 0.1] = -1
    teacher = -torch.arange(k, device=device, dtype=torch.float32).repeat(n, 1)
    return tokens, ids, teacher


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=60)
    a = p.parse_args()
    model = Model()
    for i in range(a.steps):
        loss = model.step(*batch(model.vocab, 2048, 8, i))
        if i % 10 == 0 or i == a.steps - 1:
            print("step %3d  loss %.4f" % (i, float(loss)))
    tokens, ids, _ = batch(model.vocab, 4, 8, 10 ** 6)
    got = model.score(tokens, (tokens + 1) % model.vocab)
    for t, logp, h, alternatives in zip(tokens.tolist(), got.logp.tolist(), got.entropy.tolist(), got.top_ids.tolist()):
        print("after %4d: log p(%d) %.3f, entropy %.3f, likeliest %s" % (t, (t + 1) % model.vocab, logp, h, alternatives))


if __name__ == "__main__":
    main()
