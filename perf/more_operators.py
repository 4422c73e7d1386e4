"""Cases for layer norm, tokens sorted by expert and back, and the clipped policy loss.

Each case names an operator, its direction, the element type and the sizes.  ``prepare`` makes a case's inputs on
the GPU from a seed, ``run`` makes one pass: the operator's plain form in elementary torch operations in 32 bits,
or, where ``own`` is true, the calls of ``memory_bound_elementwise_gb300``.  ``work`` counts what a pass has to
read, write and compute, and ``exact`` gives the results in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ITYPES = {"i32": torch.int32, "i64": torch.int64}
EPS = 1e-5
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.05


def listed():
    return [
        # one decode step of 9 sequences: the residual's addition and the norm before a block
        dict(name="layernorm_decode", op="layernorm", dtype="bf16", wtype="bf16", rows=9, cols=5120),
        # the same for a prompt of 16384 tokens in a wide model
        dict(name="layernorm_prompt", op="layernorm", dtype="bf16", wtype="bf16", rows=16384, cols=8192),
        # the norm's backward in a training step, the residual stream's gradient added, single-precision weights
        dict(name="layernorm_grad_step", op="layernorm_grad", dtype="bf16", wtype="f32", rows=8192, cols=4096),
        # the same for a model of an odd width in half precision: rows start anywhere
        dict(name="layernorm_grad_odd", op="layernorm_grad", dtype="f16", wtype="f16", rows=3001, cols=2001),
        # a decode step of 64 sequences is sorted by expert and laid out for the experts' products
        dict(name="dispatch_decode", op="dispatch", dtype="bf16", itype="i32", n=64, k=8, experts=128, align=16, cols=4096),
        # a training step of 16384 tokens, each to 8 of 128 experts in tiles of 128 rows
        dict(name="dispatch_step", op="dispatch", dtype="bf16", itype="i64", n=16384, k=8, experts=128, align=128, cols=4096),
        # the experts' outputs back to their tokens, weighted, onto the residual stream
        dict(name="combine_step", op="combine", dtype="bf16", wtype="f32", n=16384, k=8, experts=128, align=128, cols=4096),
        # the gradients of the above in a small single-precision model of an odd width, two experts a token
        dict(name="combine_grad_odd", op="combine_grad", dtype="f32", wtype="f32", n=5003, k=2, experts=8, align=1, cols=1001),
        # a policy's update on 2048 tokens, a quarter of them of prompts: loss and gradient
        dict(name="policy_step", op="policy_step", dtype="bf16", itype="i64", rows=2048, cols=131072, pad=0, masked=0.25),
        # a small single-precision policy, an odd vocabulary in rows padded to whole lines
        dict(name="policy_step_odd", op="policy_step", dtype="f32", itype="i32", rows=97, cols=32003, pad=61, masked=0.0),
        # the loss alone, on held-out answers
        dict(name="policy_score", op="policy", dtype="bf16", itype="i64", rows=2048, cols=65536, pad=0, masked=0.5),
        # the gradient after it at an odd vocabulary: rows start anywhere
        dict(name="policy_grad_odd", op="policy_grad", dtype="f16", itype="i32", rows=1500, cols=50001, pad=0, masked=0.0),
    ]


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def size(lo, hi):
        v, how = log_uniform(lo, hi), rng.random()
        v = v // 64 * 64 if how < 0.4 else v // 8 * 8 if how < 0.6 else v | 1
        return max(lo, min(hi, v))

    op = rng.choice(("layernorm", "layernorm", "layernorm_grad", "layernorm_grad", "dispatch", "combine", "combine_grad",
                     "policy", "policy_grad", "policy_step", "policy_step"))
    c = dict(op=op, dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
    wide = 2 if c["dtype"] == "f32" else 1
    if op.startswith("layernorm"):
        c.update(wtype=rng.choice((c["dtype"], "f32")), cols=size(64, 16384))
        c["rows"] = min((1 << 27) // wide // c["cols"], log_uniform(1, 16384))
    elif op in ("dispatch", "combine", "combine_grad"):
        c.update(n=log_uniform(1, 16384), k=rng.choice((1, 2, 4, 6, 8, 8)), experts=log_uniform(8, 512),
                 align=rng.choice((1, 1, 8, 16, 128)), cols=size(64, 8192))
        c.update(dict(itype=rng.choice(("i32", "i64"))) if op == "dispatch" else dict(wtype=rng.choice((c["dtype"], "f32"))))
        c["cols"] = max(64, min(c["cols"], (1 << 28) // wide // _capacity(c)))
    else:
        c.update(itype=rng.choice(("i32", "i64")), cols=size(1000, 160000), pad=rng.choice((0, 0, 0, 1, 8, 61)),
                 masked=rng.choice((0.0, 0.0, 0.25, 0.5)))
        c["rows"] = min((1 << 27) // wide // c["cols"], log_uniform(1, 4096))
    return c


def _capacity(case):
    """Rows that the experts' segments take at most, each a multiple of ``align``."""
    slots, align = case["n"] * case["k"], case["align"]
    return (slots + min(case["experts"], slots) * (align - 1)) // align * align


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, g, dtype, spread=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * spread).to(dtype)


def _stream(rows, cols, g):
    """A residual stream: columns with a mean and a spread of their own, a few of them far out."""
    offset = 0.5 * torch.randn(cols, generator=g, device="cuda")
    offset[torch.randint(0, cols, (3,), generator=g, device="cuda")] = 30.0
    return 2.0 * torch.randn(rows, cols, generator=g, device="cuda") + offset


def _choices(case, g):
    """The experts of each token, distinct, some more popular than others, and their weights, which sum to 1; a
    fiftieth of the tokens fill up the batch and have none."""
    n, k = case["n"], case["k"]
    scores = torch.randn(n, case["experts"], generator=g, device="cuda")
    scores += 0.7 * torch.randn(case["experts"], generator=g, device="cuda")
    best = scores.topk(k, dim=1)
    weights = torch.softmax(best.values, 1)
    empty = torch.rand(n, 1, generator=g, device="cuda") < 0.02
    return torch.where(empty, -1, best.indices), torch.where(empty, 0.0, weights)


def _logits(case, g):
    """A view of rows in a buffer whose rows are ``pad`` elements longer; a few likely tokens stand out in each row."""
    rows, cols = case["rows"], case["cols"]
    buf = torch.empty(rows, cols + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")
    x = buf.normal_(0.0, 2.0, generator=g)[:, :cols]
    likely = torch.randint(0, cols, (rows, 1), generator=g, device="cuda")
    likely = (likely + torch.arange(8, device="cuda") * (cols // 8)) % cols
    peak = 6.0 + 6.0 * torch.rand(rows, 8, generator=g, device="cuda")
    return x.scatter_(1, likely, peak.to(x.dtype)), likely


def _plan(case, experts):
    """The plain form of the sort: places of the slots, the experts' first rows, counts, and the slots of the rows."""
    n, k, align = case["n"], case["k"], case["align"]
    flat = experts.reshape(-1).long()
    key = torch.where(flat >= 0, flat, case["experts"])
    order = torch.sort(key * (n * k) + torch.arange(n * k, device="cuda")).values % (n * k)
    counts = (key[None, :] == torch.arange(case["experts"], device="cuda")[:, None]).sum(1)
    ends = ((counts + align - 1) // align * align).cumsum(0)
    offsets = torch.cat((ends.new_zeros(1), ends))
    before = torch.cat((counts.new_zeros(1), counts.cumsum(0)))  # the experts' first slots in the sorted order
    picked = key[order]
    given = picked < case["experts"]
    place = offsets[picked] + torch.arange(n * k, device="cuda") - before[picked]
    positions = torch.empty_like(flat)
    positions[order] = torch.where(given, place, -1)
    slots = torch.full((_capacity(case) + 1,), -1, dtype=torch.int64, device="cuda")
    slots[torch.where(given, place, -1)] = torch.where(given, order, -1)  # those without an expert: one past the end
    return positions.view(n, k), offsets, counts, slots[:-1]


def prepare(case, seed):
    g, op, dt = _generator(seed), case["op"], DTYPES[case["dtype"]]
    s = dict(case=dict(case))
    if op.startswith("layernorm"):
        rows, cols = case["rows"], case["cols"]
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(DTYPES[case["wtype"]])
        if op == "layernorm_grad":
            h = _stream(rows, cols, g)
            s["h"] = h.to(dt)
            s["mean"] = h.mean(1)
            s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(1) + EPS)
            s["dy"] = _normal((rows, cols), g, dt, 1e-2)
            s["dh"] = _normal((rows, cols), g, dt, 1e-2)
        else:
            s["bias"] = _normal((cols,), g, DTYPES[case["wtype"]], 0.1)
            s["x"] = _normal((rows, cols), g, dt)
            s["residual"] = _stream(rows, cols, g).to(dt)
    elif op in ("dispatch", "combine", "combine_grad"):
        n, cols = case["n"], case["cols"]
        experts, weights = _choices(case, g)
        if op == "dispatch":
            s["experts"] = experts.to(ITYPES[case["itype"]])
            s["x"] = _normal((n, cols), g, dt)
            return s
        s["plan"] = [t.to(torch.int32) for t in _plan(case, experts)]  # the forward pass has sorted them
        s["weights"] = weights.to(DTYPES[case["wtype"]])
        s["y"] = _normal((_capacity(case), cols), g, dt)
        s["residual" if op == "combine" else "dout"] = _normal((n, cols), g, dt, 2.0 if op == "combine" else 1e-2)
    else:
        s["logits"], likely = _logits(case, g)
        rows = case["rows"]
        tokens = likely[:, 0].clone()
        x = s["logits"].float()
        lse = torch.logsumexp(x, 1)
        logp = x.gather(1, tokens[:, None])[:, 0] - lse
        # The policy that drew the tokens is some steps older, the reference older still.  A ratio on the border of
        # the clipping has two gradients: none comes closer to it than a rounding of the sums could carry it over.
        moved = 0.15 * torch.randn(rows, generator=g, device="cuda")
        for border in (math.log1p(-CLIP_LOW), math.log1p(CLIP_HIGH)):
            moved = torch.where((moved - border).abs() < 1e-3, moved + 2e-3, moved)
        s["old_logp"] = logp - moved
        s["ref_logp"] = logp + 0.1 * torch.randn(rows, generator=g, device="cuda")
        s["advantage"] = torch.randn(rows, generator=g, device="cuda")
        s["dloss"] = torch.ones(rows, device="cuda")
        tokens[torch.rand(rows, generator=g, device="cuda") < case["masked"]] = -1
        s["tokens"] = tokens.to(ITYPES[case["itype"]])
        if op == "policy_grad":
            s["logp"], s["lse"] = torch.where(tokens >= 0, logp, 0.0), torch.where(tokens >= 0, lse, 0.0)
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import memory_bound_elementwise_gb300 as ew
    op = s["case"]["op"]
    if op == "layernorm":
        y, h, mean, rstd = ew.ew_layernorm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS)
        return {"y": y, "h": h, "mean": mean, "rstd": rstd}
    if op == "layernorm_grad":
        dx, dweight, dbias = ew.ew_layernorm_grad(s["dy"], s["h"], s["weight"], s["mean"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "dispatch":
        plan = ew.ew_expert_sort(s["experts"], s["case"]["experts"], align=s["case"]["align"])
        return {**plan._asdict(), "rows": ew.ew_expert_dispatch(s["x"], plan)}
    if op in ("combine", "combine_grad"):
        plan = ew.ExpertPlan(*s["plan"])
        if op == "combine":
            return ew.ew_expert_combine(s["y"], plan, s["weights"], residual=s["residual"])
        dy, dweights = ew.ew_expert_combine_grad(s["dout"], s["y"], plan, s["weights"])
        return {"dy": dy, "dweights": dweights}
    how = dict(old_logp=s["old_logp"], ref_logp=s["ref_logp"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl=KL)
    if op == "policy":
        loss, logp, lse = ew.ew_policy(s["logits"], s["tokens"], s["advantage"], **how)
        return {"loss": loss, "logp": logp, "lse": lse}
    if op == "policy_grad":
        return ew.ew_policy_grad(s["logits"], s["tokens"], s["advantage"], s["logp"], s["lse"], s["dloss"], **how)
    loss, logp, lse, dlogits = ew.ew_policy_step(s["logits"], s["tokens"], s["advantage"], s["dloss"], **how)
    return {"loss": loss, "logp": logp, "lse": lse, "dlogits": dlogits}


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "layernorm":
        h = s["x"].float() + s["residual"].float()
        mean = h.mean(1)
        d = h - mean[:, None]
        rstd = torch.rsqrt((d * d).mean(1) + EPS)
        y = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
        return {"y": y.to(dt), "h": h.to(dt), "mean": mean, "rstd": rstd}
    if op == "layernorm_grad":
        r, dy = s["rstd"][:, None], s["dy"].float()
        hat = (s["h"].float() - s["mean"][:, None]) * r
        gain = dy * s["weight"].float()
        dx = r * (gain - gain.mean(1, keepdim=True) - hat * (gain * hat).mean(1, keepdim=True)) + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": (dy * hat).sum(0), "dbias": dy.sum(0)}
    if op == "dispatch":
        positions, offsets, counts, slots = _plan(case, s["experts"])
        rows = torch.where(slots[:, None] >= 0, s["x"][slots.clamp(min=0) // case["k"]], 0.0)
        out = {"positions": positions, "offsets": offsets, "counts": counts, "slots": slots}
        return {**{k: v.to(torch.int32) for k, v in out.items()}, "rows": rows.to(dt)}
    if op in ("combine", "combine_grad"):
        positions, _, _, slots = s["plan"]
        w = s["weights"].float()
        at, given = positions.clamp(min=0).long(), positions >= 0
        if op == "combine":
            out = s["residual"].float()
            for j in range(case["k"]):
                out = out + torch.where(given[:, j, None], w[:, j, None] * s["y"][at[:, j]].float(), 0.0)
            return out.to(dt)
        dout = s["dout"].float()
        products = [torch.where(given[:, j], (dout * s["y"][at[:, j]].float()).sum(1), 0.0) for j in range(case["k"])]
        slot = slots.clamp(min=0).long()
        dy = torch.where(slots[:, None] >= 0, w.view(-1)[slot][:, None] * dout[slot // case["k"]], 0.0)
        return {"dy": dy.to(dt), "dweights": torch.stack(products, 1)}
    x = s["logits"].float()
    given = s["tokens"] >= 0
    at = torch.where(given, s["tokens"], 0).long()[:, None]
    if op == "policy_grad":
        lse, logp = s["lse"], s["logp"]
    else:
        top = x.max(1, keepdim=True).values
        lse = torch.exp(x - top).sum(1).log() + top[:, 0]
        logp = x.gather(1, at)[:, 0] - lse
    # a token's few numbers in 64 bits: the clipping has a border, and the divergence is a small difference
    wide, adv = logp.double(), s["advantage"].double()
    ratio = torch.exp(wide - s["old_logp"].double())
    free, bound = ratio * adv, ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * adv
    apart = s["ref_logp"].double() - wide
    loss = -torch.minimum(free, bound) + KL * (torch.expm1(apart) - apart)
    loss, logp, lse = (torch.where(given, v, 0.0).float() for v in (loss, logp, lse))
    if op == "policy":
        return {"loss": loss, "logp": logp, "lse": lse}
    slope = -torch.where(free > bound, 0.0, free) - KL * torch.expm1(apart)
    slope = torch.where(given, slope * s["dloss"].double(), 0.0).float()[:, None]
    d = torch.where(given[:, None], -slope * torch.exp(x - lse[:, None]), 0.0).scatter_add_(1, at, slope).to(dt)
    return d if op == "policy_grad" else {"loss": loss, "logp": logp, "lse": lse, "dlogits": d}


def work(case):
    e, cols = DTYPES[case["dtype"]].itemsize, case["cols"]
    w = DTYPES[case["wtype"]].itemsize if "wtype" in case else 0
    i = ITYPES[case["itype"]].itemsize if "itype" in case else 0
    op = case["op"]
    if op.startswith("layernorm"):
        rows, n = case["rows"], case["rows"] * cols
        if op == "layernorm":
            return {"bytes": 4 * n * e + 2 * cols * w + 8 * rows, "flops": 8 * n}
        return {"bytes": 4 * n * e + cols * (w + 8) + 8 * rows, "flops": 14 * n}
    if "k" in case:
        n, slots, cap = case["n"], case["n"] * case["k"], _capacity(case)
        if op == "dispatch":
            return {"bytes": (n + cap) * cols * e + slots * (i + 4) + 4 * cap + 8 * case["experts"], "flops": slots}
        if op == "combine":
            return {"bytes": (slots + 2 * n) * cols * e + slots * (w + 4), "flops": (2 * slots + n) * cols}
        return {"bytes": (n + slots + cap) * cols * e + slots * (w + 8) + 4 * cap, "flops": 3 * slots * cols}
    rows, n = case["rows"], case["rows"] * cols
    read = round((1.0 - case["masked"]) * n)  # rows without a token need not be read
    if op == "policy":
        return {"bytes": read * e + rows * (i + 24), "flops": 4 * read}
    return {"bytes": (read + n) * e + rows * (i + 28), "flops": (4 if op == "policy_grad" else 7) * read}


def exact(case, seed):
    """What ``run`` returns for these inputs, in 64 bits and a block of rows at a time."""
    s = prepare(case, seed)
    op, cols = case["op"], case["cols"]
    if op == "dispatch":
        return _exact_dispatch(case, s)
    if op in ("combine", "combine_grad"):
        return _exact_experts(case, s)
    parts, block = [], max(1, (1 << 25) // cols)
    for a in range(0, case["rows"], block):
        v = {k: t[a:a + block].double() if t.is_floating_point() else t[a:a + block].long() for k, t in s.items()
             if isinstance(t, torch.Tensor) and k not in ("weight", "bias")}
        parts.append((_exact_norm if op.startswith("layernorm") else _exact_policy)(case, s, v))
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0] if k not in ("dweight", "dbias")}
    out.update({k: torch.stack([p[k] for p in parts]).sum(0) for k in ("dweight", "dbias") if k in parts[0]})
    return out["dlogits"] if op == "policy_grad" else out


def _exact_norm(case, s, v):
    cols, w = case["cols"], s["weight"].double()
    if case["op"] == "layernorm":
        h = v["x"] + v["residual"]
        mean = torch.einsum("rc->r", h) / cols
        away = torch.linalg.vector_norm(h - mean[:, None], dim=1)
        rstd = (away ** 2 / cols + EPS) ** -0.5
        return {"y": torch.addcmul(s["bias"].double(), torch.einsum("rc,r->rc", h - mean[:, None], rstd), w), "h": h,
                "mean": mean, "rstd": rstd}
    r, hat = v["rstd"], torch.einsum("rc,r->rc", v["h"] - v["mean"][:, None], v["rstd"])
    first = torch.einsum("rc,c->r", v["dy"], w) / cols
    second = torch.einsum("rc,c,rc->r", v["dy"], w, hat) / cols
    dx = torch.einsum("rc,c,r->rc", v["dy"], w, r) - (r * first)[:, None] - (r * second)[:, None] * hat + v["dh"]
    return {"dx": dx, "dweight": torch.einsum("rc,rc->c", v["dy"], hat), "dbias": torch.einsum("rc->c", v["dy"])}


def _exact_dispatch(case, s):
    """Token by token on the host: the experts' rows as lists."""
    k, align = case["k"], case["align"]
    of = [[] for _ in range(case["experts"])]
    for slot, expert in enumerate(s["experts"].reshape(-1).tolist()):
        if expert >= 0:
            of[expert].append(slot)
    offsets, slots, positions = [0], [], [-1] * (case["n"] * k)
    for rows in of:
        for slot in rows:
            positions[slot] = len(slots)
            slots.append(slot)
        slots += [-1] * (-len(slots) % align)
        offsets.append(len(slots))
    slots += [-1] * (_capacity(case) - len(slots))

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    at = torch.tensor(slots, device="cuda")
    padded = torch.cat((s["x"], s["x"].new_zeros(1, case["cols"])))  # a slot of -1 picks the row of zeros at the end
    return {"positions": whole(positions).view(-1, k), "offsets": whole(offsets), "counts": whole([len(r) for r in of]),
            "slots": whole(slots), "rows": padded[torch.div(at, k, rounding_mode="floor")]}


def _exact_experts(case, s):
    """A block of tokens at a time, by the rows that their slots have."""
    n, cols = case["n"], case["cols"]
    positions, w = s["plan"][0].long(), s["weights"].double()
    block = max(1, (1 << 25) // (cols * case["k"]))
    if case["op"] == "combine":
        out = s["residual"].double()
    else:
        out = {"dy": torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda"), "dweights": torch.zeros_like(w)}
    for a in range(0, n, block):
        token, j = torch.nonzero(positions[a:a + block] >= 0, as_tuple=True)
        token = token + a
        row = positions[token, j]
        if case["op"] == "combine":
            out.index_put_((token,), torch.einsum("sc,s->sc", s["y"][row].double(), w[token, j]), accumulate=True)
        else:
            dout = s["dout"][token].double()
            out["dy"][row] = torch.einsum("sc,s->sc", dout, w[token, j])
            out["dweights"][token, j] = torch.einsum("sc,sc->s", dout, s["y"][row].double())
    return out


def _exact_policy(case, s, v):
    row = torch.arange(v["logits"].shape[0], device="cuda")
    given, at = v["tokens"] >= 0, v["tokens"].clamp(min=0)
    if case["op"] == "policy_grad":
        lse, logp, p = v["lse"], v["logp"], torch.exp(v["logits"] - v["lse"][:, None])
    else:
        lse = torch.logsumexp(v["logits"], 1)
        every = torch.log_softmax(v["logits"], 1)
        logp, p = every[row, at], every.exp()
    ratio, adv = (logp - v["old_logp"]).exp(), v["advantage"]
    # the clipping takes effect where it makes the surrogate smaller: above for gains, below for losses
    stopped = torch.where(adv >= 0, ratio > 1.0 + CLIP_HIGH, ratio < 1.0 - CLIP_LOW)
    reached = torch.where(stopped, torch.where(adv >= 0, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW), ratio)
    other = (v["ref_logp"] - logp).exp()
    loss = KL * (other - 1.0 - (v["ref_logp"] - logp)) - reached * adv
    slope = KL * (1.0 - other) - torch.where(stopped, 0.0, ratio * adv)
    slope = torch.where(given, slope * v["dloss"], 0.0)
    d = torch.einsum("rc,r->rc", p, -slope)
    d[row, at] += slope
    d[~given] = 0.0
    return {**{k: torch.where(given, t, 0.0) for k, t in (("loss", loss), ("logp", logp), ("lse", lse))},
            **({"dlogits": d} if case["op"] != "policy" else {})}
