"""Cases for the language-model operators: embedding, RMS norm, token log probabilities, distillation.

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
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # a group's scale is never zero
EPS = 1e-6


def listed():
    return [
        # the next token of 64 sequences enters a decode step
        dict(name="embed_decode", op="embed", dtype="bf16", itype="i64", n=64, vocab=131072, cols=4096),
        # the embedding table's gradient in a training step of 16384 tokens, the dense table written whole
        dict(name="embed_grad_step", op="embed_grad", dtype="bf16", itype="i64", n=16384, vocab=131072, cols=2048),
        # a small single-precision model with an odd vocabulary and batch
        dict(name="embed_grad_odd", op="embed_grad", dtype="f32", itype="i32", n=5003, vocab=32003, cols=1000),
        # one decode step of 7 sequences: residual, norm and 8-bit activations for the next product
        dict(name="norm_q_decode", op="norm_q", dtype="bf16", wtype="bf16", rows=7, cols=5120, group=128),
        # the same for a prompt of 16384 tokens in a wide model
        dict(name="norm_q_prompt", op="norm_q", dtype="bf16", wtype="bf16", rows=16384, cols=8192, group=128),
        # the norm's backward in a training step, the residual stream's gradient added, single-precision weights
        dict(name="norm_grad_step", op="norm_grad", dtype="bf16", wtype="f32", rows=8192, cols=4096),
        # the same for a small single-precision model with an odd width
        dict(name="norm_grad_odd", op="norm_grad", dtype="f32", wtype="f32", rows=1023, cols=1001),
        # decode: the sampled tokens' log probabilities with 20 alternatives, half of the vocabulary masked out
        dict(name="logprob_decode", op="logprob", dtype="bf16", itype="i64", rows=5, cols=131072, pad=0, top=20, masked=0.5),
        # scoring a prompt of 2048 tokens with 5 alternatives a token
        dict(name="logprob_score", op="logprob", dtype="bf16", itype="i64", rows=2048, cols=131072, pad=0, top=5, masked=0.0),
        # the gradient of log probability and entropy (a policy's update) at an odd vocabulary: rows start anywhere
        dict(name="logprob_grad_odd", op="logprob_grad", dtype="f16", itype="i32", rows=1500, cols=50001, pad=0),
        # distillation of 4096 tokens from a teacher's 64 top logits: loss and gradient
        dict(name="distill_step", op="distill", dtype="bf16", itype="i32", rows=4096, cols=65536, pad=0, teacher=64, temperature=2.0),
        # a small single-precision student, an odd vocabulary in rows padded to whole lines
        dict(name="distill_odd", op="distill", dtype="f32", itype="i64", rows=97, cols=32003, pad=61, teacher=17, temperature=1.0),
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        how = rng.random()
        v = v // 64 * 64 if how < 0.4 else v // 8 * 8 if how < 0.6 else v | 1
        return max(lo, min(hi, v)) + (v == 3072)

    op = rng.choice(("embed", "embed_grad", "norm", "norm_q", "norm_grad", "logprob", "logprob_grad", "distill"))
    c = dict(op=op, dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
    if op in ("embed", "embed_grad"):
        c.update(itype=rng.choice(("i32", "i64")), n=int(round(math.exp(rng.uniform(0, math.log(16384))))),
                 vocab=size(1000, 131072), cols=size(64, 4096))
        c["cols"] = min(c["cols"], max(64, (1 << 28) // 4 * 4 // c["vocab"])) if op == "embed_grad" else c["cols"]
        if op == "embed_grad" and c["dtype"] == "f32":
            c["cols"] = max(64, c["cols"] // 2)
    elif op in ("norm", "norm_q", "norm_grad"):
        c.update(wtype=rng.choice((c["dtype"], "f32")), cols=size(64, 16384))
        most = (1 << 26) // c["cols"]
        c["rows"] = min(most, int(round(math.exp(rng.uniform(0, math.log(16384))))))
        if op == "norm_q":
            c["group"] = rng.choice((0, 32, 64, 128, 256))
    else:
        c.update(itype=rng.choice(("i32", "i64")), cols=size(1000, 160000), pad=rng.choice((0, 0, 0, 1, 8, 61)))
        most = (1 << (26 if c["dtype"] == "f32" else 27)) // c["cols"]
        c["rows"] = min(most, int(round(math.exp(rng.uniform(0, math.log(4096))))))
        if op == "logprob":
            c.update(top=rng.choice((0, 1, 5, 20)), masked=rng.choice((0.0, 0.0, 0.5, 0.9)))
        if op == "distill":
            c.update(teacher=rng.choice((8, 17, 64, 100, 256)), temperature=rng.choice((1.0, 2.0, 4.0)))
    return c


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, g, dtype, spread=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * spread).to(dtype)


def _tokens(n, vocab, g, itype, skipped):
    """Token ids as text has them: log-uniform ranks (a few tokens make up much of the text), scattered over the
    vocabulary; a share of ``skipped`` positions holds no token (-1)."""
    rank = torch.exp(torch.rand(n, generator=g, device="cuda") * math.log(vocab)).to(torch.int64) - 1
    ids = (rank.clamp(0, vocab - 1) * 7919 + 17) % vocab
    ids[torch.rand(n, generator=g, device="cuda") < skipped] = -1
    return ids.to(ITYPES[itype])


def _logits(case, g):
    """A view of rows in a buffer whose rows are ``pad`` elements longer; a few likely tokens stand out in each row."""
    rows, cols = case["rows"], case["cols"]
    buf = torch.empty(rows, cols + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")
    x = buf.normal_(0.0, 2.0, generator=g)[:, :cols]
    likely = torch.randint(0, cols, (rows, 1), generator=g, device="cuda")
    likely = (likely + torch.arange(8, device="cuda") * (cols // 8)) % cols
    peak = 6.0 + 6.0 * torch.rand(rows, 8, generator=g, device="cuda")
    return x.scatter_(1, likely, peak.to(x.dtype)), likely


def prepare(case, seed):
    g, op, dt = _generator(seed), case["op"], DTYPES[case["dtype"]]
    s = dict(case=dict(case))
    if op in ("embed", "embed_grad"):
        s["tokens"] = _tokens(case["n"], case["vocab"], g, case["itype"], 0.02)
        if op == "embed":
            s["table"] = _normal((case["vocab"], case["cols"]), g, dt, 0.02)
            s["scale"] = math.sqrt(case["cols"])
        else:
            s["dout"] = _normal((case["n"], case["cols"]), g, dt, 1e-2)
            s["scale"] = math.sqrt(case["cols"])
    elif op in ("norm", "norm_q", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(DTYPES[case["wtype"]])
        if op == "norm_grad":
            h = 3.0 * torch.randn(rows, cols, generator=g, device="cuda")
            s["h"] = h.to(dt)
            s["rstd"] = torch.rsqrt(h.square().mean(1) + EPS)
            s["dy"] = _normal((rows, cols), g, dt, 1e-2)
            s["dh"] = _normal((rows, cols), g, dt, 1e-2)
        else:
            s["x"] = _normal((rows, cols), g, dt)
            s["residual"] = _normal((rows, cols), g, dt, 3.0)
    else:
        s["logits"], likely = _logits(case, g)
        rows, cols = s["logits"].shape
        if op in ("logprob", "logprob_grad"):
            s["tokens"] = likely[:, 0].clone()
            s["tokens"][torch.rand(rows, generator=g, device="cuda") < 0.05] = -1  # no token was given here
            s["tokens"] = s["tokens"].to(ITYPES[case["itype"]])
        if op == "logprob" and case["masked"]:
            out = torch.rand(rows, cols, generator=g, device="cuda") < case["masked"]
            s["logits"].masked_fill_(out.scatter_(1, likely, False), -math.inf)
        if op == "logprob_grad":
            x = s["logits"].float()
            s["lse"] = torch.logsumexp(x, 1)
            p = torch.exp(x - s["lse"][:, None])
            s["entropy"] = s["lse"] - (p * x).sum(1)
            s["dlogp"] = torch.randn(rows, generator=g, device="cuda")
            s["dentropy"] = 0.01 * torch.randn(rows, generator=g, device="cuda")
        if op == "distill":
            k = case["teacher"]
            # the teacher's top tokens are distinct: a stride over the vocabulary from a likely one
            step = cols // k
            ids = (likely[:, :1] + torch.arange(k, device="cuda") * step) % cols
            few = torch.randint(k // 2, k + 1, (rows, 1), generator=g, device="cuda")  # some give fewer than k
            given = torch.rand(rows, 1, generator=g, device="cuda") >= 0.1  # a prompt's tokens are not distilled
            ids[(torch.arange(k, device="cuda") >= few) | ~given] = -1
            s["ids"] = ids.to(ITYPES[case["itype"]])
            top = torch.randn(rows, k, generator=g, device="cuda").mul_(3.0).sort(1, descending=True).values
            s["teacher"] = (top + 8.0).to(dt)
            s["dloss"] = torch.full((rows,), 1.0 / rows, device="cuda")
            s["scale"] = 1.0 / case["temperature"]
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import memory_bound_elementwise_gb300 as ew
    op = s["case"]["op"]
    if op == "embed":
        return ew.ew_embed(s["table"], s["tokens"], scale=s["scale"])
    if op == "embed_grad":
        return ew.ew_embed_grad(s["dout"], s["tokens"], s["case"]["vocab"], scale=s["scale"])
    if op == "norm":
        y, h, rstd = ew.ew_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        return {"y": y, "h": h, "rstd": rstd}
    if op == "norm_q":
        q, scales, h, rstd = ew.ew_rmsnorm_quant(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                                                 group=s["case"]["group"])
        return {"q": q, "scales": scales, "h": h, "rstd": rstd}
    if op == "norm_grad":
        dx, dweight = ew.ew_rmsnorm_grad(s["dy"], s["h"], s["weight"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dweight": dweight}
    if op == "logprob":
        return ew.ew_logprob(s["logits"], s["tokens"], top=s["case"]["top"])._asdict()
    if op == "logprob_grad":
        return ew.ew_logprob_grad(s["logits"], s["tokens"], s["lse"], s["entropy"], s["dlogp"], s["dentropy"])
    loss, lse, dlogits = ew.ew_distill_step(s["logits"], s["ids"], s["teacher"], s["dloss"], scale=s["scale"])
    return {"loss": loss, "lse": lse, "dlogits": dlogits}


def _lse(x):
    top = x.max(1, keepdim=True).values
    return (torch.exp(x - top).sum(1, keepdim=True).log() + top)


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "embed":
        valid = (s["tokens"] >= 0) & (s["tokens"] < case["vocab"])
        rows = s["table"][torch.where(valid, s["tokens"], 0).long()].float() * s["scale"]
        return torch.where(valid[:, None], rows, 0.0).to(dt)
    if op == "embed_grad":
        valid = s["tokens"] >= 0
        rows = torch.where(valid[:, None], s["dout"].float() * s["scale"], 0.0)
        dtable = torch.zeros(case["vocab"], case["cols"], device="cuda")
        return dtable.index_add_(0, torch.where(valid, s["tokens"], 0).long(), rows).to(dt)
    if op in ("norm", "norm_q"):
        h = s["x"].float() + s["residual"].float()
        rstd = torch.rsqrt((h * h).mean(1) + EPS)
        y = h * rstd[:, None] * s["weight"].float()
        out = {"h": h.to(dt), "rstd": rstd}
        if op == "norm":
            return {"y": y.to(dt), **out}
        rows, cols = y.shape
        group = case["group"] or cols
        groups = -(-cols // group)
        wide = torch.zeros(rows, groups * group, device="cuda")
        wide[:, :cols] = y
        wide = wide.view(rows, groups, group)
        scales = wide.abs().amax(2).clamp(min=AMAX_FLOOR) / E4M3_MAX
        q = (wide / scales[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, -1)[:, :cols]
        return {"q": q.to(torch.float8_e4m3fn), "scales": scales, **out}
    if op == "norm_grad":
        r, h, dy = s["rstd"][:, None], s["h"].float(), s["dy"].float()
        gain = dy * s["weight"].float()
        hat = h * r
        dx = r * (gain - hat * (gain * hat).mean(1, keepdim=True)) + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": (dy * hat).sum(0)}
    x = s["logits"].float()
    if op == "logprob":
        lse = _lse(x)
        logp = x - lse
        p = torch.exp(logp)
        valid = s["tokens"] >= 0
        at = logp.gather(1, torch.where(valid, s["tokens"], 0).long()[:, None])[:, 0]
        out = {"logp": torch.where(valid, at, 0.0), "entropy": -torch.where(p > 0, p * logp, 0.0).sum(1), "lse": lse[:, 0]}
        # the largest first, equal ones by index: the value's bits in whole-number order above the reversed index
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long()
        key = order * 2 ** 32 + (2 ** 32 - 1 - torch.arange(x.shape[1], device="cuda"))
        best = 2 ** 32 - 1 - key.topk(case["top"], dim=1).values % 2 ** 32
        return {**out, "top_logp": logp.gather(1, best), "top_ids": best.to(torch.int32)}
    if op == "logprob_grad":
        logp = x - s["lse"][:, None]
        p = torch.exp(logp)
        d = -p * (s["dlogp"][:, None] + s["dentropy"][:, None] * torch.where(p > 0, logp + s["entropy"][:, None], 0.0))
        valid = s["tokens"] >= 0
        d = torch.where(valid[:, None], d, d + p * s["dlogp"][:, None])
        at = torch.where(valid, s["tokens"], 0).long()[:, None]
        return d.scatter_add_(1, at, torch.where(valid, s["dlogp"], 0.0)[:, None]).to(dt)
    x = x * s["scale"]
    lse = _lse(x)
    valid = s["ids"] >= 0
    given = valid.any(1, keepdim=True)
    at = torch.where(valid, s["ids"], 0).long()
    t = torch.where(valid, s["teacher"].float() * s["scale"], -math.inf)
    logq = torch.where(valid, t - torch.where(given, _lse(torch.where(given, t, 0.0)), 0.0), 0.0)
    q = torch.where(valid, torch.exp(logq), 0.0)
    loss = (q * (logq - (x.gather(1, at) - lse))).sum(1)
    d = torch.where(given, torch.exp(x - lse), 0.0).scatter_add_(1, at, -q)
    return {"loss": loss, "lse": lse[:, 0], "dlogits": (d * (s["dloss"] * s["scale"])[:, None]).to(dt)}


def work(case):
    e = DTYPES[case["dtype"]].itemsize
    i = ITYPES[case["itype"]].itemsize if "itype" in case else 0
    op = case["op"]
    if op == "embed":
        n = case["n"] * case["cols"]
        return {"bytes": 2 * n * e + case["n"] * i, "flops": n}
    if op == "embed_grad":
        n = case["n"] * case["cols"]
        return {"bytes": (n + case["vocab"] * case["cols"]) * e + case["n"] * i, "flops": 2 * n}
    if "wtype" in case:
        rows, cols = case["rows"], case["cols"]
        n, w = rows * cols, cols * DTYPES[case["wtype"]].itemsize
        if op == "norm":
            return {"bytes": 4 * n * e + w + 4 * rows, "flops": 5 * n}
        if op == "norm_q":
            groups = -(-cols // (case["group"] or cols))
            return {"bytes": n * (3 * e + 1) + w + 4 * rows * (1 + groups), "flops": 8 * n}
        return {"bytes": 4 * n * e + w + 4 * cols + 4 * rows, "flops": 11 * n}
    rows, n = case["rows"], case["rows"] * case["cols"]
    if op == "logprob":
        return {"bytes": n * e + rows * (i + 12 + 8 * case["top"]), "flops": 6 * n}
    if op == "logprob_grad":
        return {"bytes": 2 * n * e + rows * (i + 16), "flops": 6 * n}
    return {"bytes": 2 * n * e + rows * (12 + case["teacher"] * (i + e)), "flops": 8 * n}


def exact(case, seed):
    """What ``run`` returns for these inputs, in 64 bits and a block of rows at a time."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        picked = s["table"].double().mul_(s["scale"])
        picked = torch.cat((picked, picked.new_zeros(1, case["cols"])))
        return picked[s["tokens"].long()]  # -1 picks the row of zeros at the end
    if op == "embed_grad":
        dtable = torch.zeros(case["vocab"] + 1, case["cols"], dtype=torch.float64, device="cuda")
        at = s["tokens"].long() % (case["vocab"] + 1)  # positions without a token fall into a last row
        dtable.index_put_((at,), s["dout"].double() * s["scale"], accumulate=True)
        return dtable[:-1]
    parts = []
    rows = (s["dy"] if op == "norm_grad" else s["x"] if "x" in s else s["logits"]).shape[0]
    block = max(1, (1 << 26) // case["cols"])
    for a in range(0, rows, block):
        b = min(rows, a + block)
        part = {k: v[a:b].double() if v.is_floating_point() else v[a:b].long() for k, v in s.items()
                if isinstance(v, torch.Tensor) and k != "weight"}
        parts.append(_exact_rows(case, s, part))
    if op == "logprob_grad":
        return torch.cat([p["dlogits"] for p in parts])
    out = {k: None if v is None else torch.cat([p[k] for p in parts]) for k, v in parts[0].items() if k != "dweight"}
    if op == "norm_grad":
        out["dweight"] = torch.stack([p["dweight"] for p in parts]).sum(0)
    return out


def _exact_rows(case, s, v):
    op, cols = case["op"], case["cols"]
    if op in ("norm", "norm_q"):
        h = v["x"] + v["residual"]
        rstd = 1.0 / torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / cols + EPS)
        y = torch.einsum("rc,r,c->rc", h, rstd, s["weight"].double())
        if op == "norm":
            return {"y": y, "h": h, "rstd": rstd}
        group = case["group"] or cols
        scales = torch.stack([t.abs().max(1).values for t in y.split(group, 1)], 1).clamp(min=AMAX_FLOOR) / E4M3_MAX
        return {"q": y / scales.repeat_interleave(group, 1)[:, :cols], "scales": scales, "h": h, "rstd": rstd}
    if op == "norm_grad":
        w = s["weight"].double()
        inner = torch.einsum("rc,rc,c->r", v["dy"], v["h"], w)
        dx = (torch.einsum("rc,c,r->rc", v["dy"], w, v["rstd"])
              - torch.einsum("rc,r->rc", v["h"], v["rstd"] ** 3 * inner / cols) + v["dh"])
        return {"dx": dx, "dweight": torch.einsum("rc,rc,r->c", v["dy"], v["h"], v["rstd"])}
    row = torch.arange(v["logits"].shape[0], device="cuda")
    if op == "logprob":
        logp = torch.log_softmax(v["logits"], 1)
        at = torch.where(v["tokens"] >= 0, logp[row, v["tokens"]], 0.0)
        entropy = torch.special.entr(logp.exp()).sum(1)
        return {"logp": at, "entropy": entropy, "lse": torch.logsumexp(v["logits"], 1),
                "top_logp": logp.topk(case["top"], 1).values, "top_ids": None}
    if op == "logprob_grad":
        p = torch.exp(v["logits"] - v["lse"][:, None])
        d = torch.zeros_like(p)
        given = v["tokens"] >= 0
        d[row[given], v["tokens"][given]] = v["dlogp"][given]
        d -= p * torch.where(given, v["dlogp"], 0.0)[:, None]
        return {"dlogits": d + v["dentropy"][:, None] * (torch.special.entr(p) - p * v["entropy"][:, None])}
    x = v["logits"] * s["scale"]
    logp = torch.log_softmax(x, 1)
    given = v["ids"] >= 0
    q = torch.nan_to_num(torch.softmax(torch.where(given, v["teacher"] * s["scale"], -math.inf), 1))
    dense = torch.zeros_like(logp).index_put_((row[:, None].expand_as(v["ids"])[given], v["ids"][given]), q[given])
    loss = -torch.special.entr(q).sum(1) - (dense * logp).sum(1)
    d = (logp.exp() * dense.sum(1, keepdim=True) - dense) * (v["dloss"] * s["scale"])[:, None]
    return {"loss": loss, "lse": torch.logsumexp(x, 1), "dlogits": d}
