"""A small mixture of experts tuned with rewards: layer norm, routing and the policy loss together.

The model is an embedding of tokens and places, a few blocks of layer norm and experts on the residual stream, a last
layer norm, and logits against the embedding table itself.  Of each token's experts the best few are taken (the top
alternatives of the router's logits), its row is laid out with those of the experts' other tokens, and their outputs
come back weighted, onto the residual stream.  A policy samples a token, a reward says how good it was, and the clipped
policy loss moves the model, held near a reference by its divergence.  All memory-bound steps run in this library; the
products are torch's.

    python examples/mixture_of_experts.py [--steps 40]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_bound_elementwise_gb300 as ew  # noqa: E402


class Model:
    def __init__(self, vocab=500, dim=128, hidden=256, experts=8, chosen=2, blocks=2, places=64, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, spread):
            return torch.randn(*shape, generator=g, device=device) * spread

        self.vocab, self.scale, self.chosen, self.experts = vocab, math.sqrt(dim), chosen, experts
        self.table, self.places = normal(vocab, dim, spread=1.0 / self.scale), normal(places, dim, spread=0.5)
        self.blocks = [dict(gain=torch.ones(dim, device=device), bias=torch.zeros(dim, device=device),
                            router=normal(dim, experts, spread=dim ** -0.5), up=normal(experts, dim, hidden, spread=dim ** -0.5),
                            down=normal(experts, hidden, dim, spread=hidden ** -0.5)) for _ in range(blocks)]
        self.gain, self.bias = torch.ones(dim, device=device), torch.zeros(dim, device=device)

    def parameters(self):
        return [self.table, self.places, self.gain, self.bias] + [b[k] for b in self.blocks
                                                                 for k in ("gain", "bias", "router", "up", "down")]

    def forward(self, tokens, places):
        """Logits of each token, and what the backward pass needs."""
        x, residual, saved = ew.ew_embed(self.table, tokens, scale=self.scale), ew.ew_embed(self.places, places), []
        for b in self.blocks:
            y, h, mean, rstd = ew.ew_layernorm(x, b["gain"], b["bias"], residual=residual)
            best = ew.ew_logprob(y @ b["router"], None, top=self.chosen)
            weights = torch.softmax(best.top_logp, 1)
            plan = ew.ew_expert_sort(best.top_ids, self.experts, align=8)
            rows = ew.ew_expert_dispatch(y, plan)
            ends = plan.offsets.tolist()  # the products of a small example, one for each expert
            active, outputs = rows.new_zeros(len(rows), b["up"].shape[2]), torch.zeros_like(rows)
            for e, (start, end) in enumerate(zip(ends, ends[1:])):
                active[start:end] = ew.ew_relu(rows[start:end] @ b["up"][e])
                outputs[start:end] = active[start:end] @ b["down"][e]
            saved.append((y, h, mean, rstd, best.top_ids, weights, plan, ends, rows, active, outputs))
            x, residual = ew.ew_expert_combine(outputs, plan, weights, residual=h), None
        y, h, mean, rstd = ew.ew_layernorm(x, self.gain, self.bias)
        return y @ self.table.t(), (saved, (y, h, mean, rstd))

    def backward(self, tokens, places, dlogits, kept):
        """The parameters' gradients, in the order of parameters()."""
        saved, (y, h, mean, rstd) = kept
        dtable = dlogits.t() @ y
        dh, dgain, dbias = ew.ew_layernorm_grad(dlogits @ self.table, h, self.gain, mean, rstd)
        grads = []
        for b, (y, h, mean, rstd, ids, weights, plan, ends, rows, active, outputs) in zip(reversed(self.blocks), reversed(saved)):
            doutputs, dweights = ew.ew_expert_combine_grad(dh, outputs, plan, weights)
            drows, dup, ddown = torch.zeros_like(rows), torch.empty_like(b["up"]), torch.empty_like(b["down"])
            for e, (start, end) in enumerate(zip(ends, ends[1:])):
                ddown[e] = active[start:end].t() @ doutputs[start:end]
                dactive = (doutputs[start:end] @ b["down"][e].t()).masked_fill_(active[start:end] == 0, 0.0)
                dup[e] = rows[start:end].t() @ dactive
                drows[start:end] = dactive @ b["up"][e].t()
            dchosen = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
            dscores = torch.zeros(len(tokens), self.experts, device=dh.device).scatter_(1, ids.long(), dchosen)
            # the router's gradient and the experts', which is the dispatch's
            dy = ew.ew_expert_combine(drows, plan, residual=dscores @ b["router"].t())
            drouter = y.t() @ dscores
            dh, dg, db = ew.ew_layernorm_grad(dy, h, b["gain"], mean, rstd, dh=dh)
            grads = [dg, db, drouter, dup, ddown] + grads
        dplaces = ew.ew_embed_grad(dh, places, self.places.shape[0])
        # the table is the embedding too: its gradient is added to the logits'
        ew.ew_embed_grad(dh, tokens, self.vocab, dtable=dtable, scale=self.scale, accumulate=True)
        return [dtable, dplaces, dgain, dbias] + grads

    def step(self, tokens, places, picked, advantage, old_logp, ref_logp, kl=0.02, rate=0.5):
        """One step of the policy's update on the picked tokens (-1 where none counts); returns the mean loss before it."""
        logits, kept = self.forward(tokens, places)
        counts = (picked >= 0).float()
        dloss = counts / counts.sum()
        # the gradient takes the logits' place
        loss, _, _, dlogits = ew.ew_policy_step(logits, picked, advantage, dloss, old_logp=old_logp, ref_logp=ref_logp, kl=kl,
                                                dlogits=logits)
        for p, g in zip(self.parameters(), self.backward(tokens, places, dlogits, kept)):
            ew.ew_saxpy(-rate, g.contiguous(), p)
        return (loss * dloss).sum()


def batch(vocab, n, seed, places=64, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    tokens = torch.randint(0, vocab, (n,), generator=g, device=device)
    return tokens, torch.arange(n, device=device) % places


def rollout(model, tokens, places, seed):
    """Tokens drawn from the policy, their log probabilities, and how good they are: those near the token are better.  A
    tenth of the places belong to prompts and hold none."""
    g = torch.Generator(device=tokens.device).manual_seed(seed)
    logits, _ = model.forward(tokens, places)
    picked = torch.multinomial(torch.softmax(logits, 1), 1, generator=g)[:, 0]
    picked[torch.rand(len(tokens), generator=g, device=tokens.device) < 0.1] = -1
    logp = ew.ew_logprob(logits, picked).logp
    reward = -((picked - tokens).abs().float() / model.vocab)
    given = picked >= 0
    mean, spread = reward[given].mean(), reward[given].std()
    return picked, torch.where(given, (reward - mean) / spread, 0.0), logp, mean


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=40)
    a = p.parse_args()
    model = Model()
    reference = Model()
    for i in range(a.steps):
        tokens, places = batch(model.vocab, 2048, i)
        picked, advantage, old, reward = rollout(model, tokens, places, 10 ** 6 + i)
        ref = ew.ew_logprob(reference.forward(tokens, places)[0], picked).logp
        for _ in range(2):  # the second time the policy has moved, and ratios are no longer 1
            loss = model.step(tokens, places, picked, advantage, old, ref)
        if i % 10 == 0 or i == a.steps - 1:
            print("step %3d  reward %.4f  loss %.4f" % (i, float(reward), float(loss)))


if __name__ == "__main__":
    main()
