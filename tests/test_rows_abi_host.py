"""The row operators' C ABI on the host: refusals, sizes and overlap rules.

Every call here is rejected, or has nothing to do, before any CUDA call."""
import os

import pytest

import memory_bound_elementwise_gb300 as ew

pytestmark = pytest.mark.skipif(not os.path.exists(ew.LIB_PATH), reason="libew.so not built")

OK, INVALID, NULLP, DTYPE, OVERLAP = 0, 1, 2, 3, 4
P = 0x10000000  # fake addresses, never dereferenced
MB = 1 << 20
BIG = (1 << 31) - (1 << 16)


def norm(dt=2, x=P, xs=64, r=None, rs=0, wt=2, w=None, eps=1e-6, y=P + MB, ys=64, h=None, hs=0, rstd=None, rows=4,
         cols=64):
    return ew.lib().ew_rmsnorm(dt, x, xs, r, rs, wt, w, eps, y, ys, h, hs, rstd, rows, cols, None)


def quant(dt=2, x=P, xs=64, qt=0, group=32, q=P + MB, qs=64, s=P + 2 * MB, ss=2, rows=4, cols=64, eps=1e-6):
    return ew.lib().ew_rmsnorm_quant(dt, x, xs, None, 0, 2, None, eps, qt, group, q, qs, s, ss, None, 0, None, rows, cols,
                                     None)


def norm_grad(dt=2, dy=P, h=P + MB, rstd=P + 2 * MB, dh=None, dx=P + 3 * MB, dw=P + 4 * MB, rows=4, cols=64,
              work=P + 5 * MB, size=MB, s=64):
    return ew.lib().ew_rmsnorm_grad(dt, dy, s, h, s, 2, None, rstd, dh, s, dx, s, dw, rows, cols, work, size, None)


def test_norm_refusals():
    assert norm(dt=3) == DTYPE and norm(dt=-1) == DTYPE and norm(w=P + 2 * MB, wt=1) == DTYPE
    assert norm(rows=0, x=None, y=None) == OK and ew.last_launch()["launches"] == 0
    assert norm(rows=-1) == INVALID and norm(cols=0) == INVALID and norm(rows=BIG + 1) == INVALID
    assert norm(cols=BIG + 1, xs=BIG + 1, ys=BIG + 1) == INVALID
    assert norm(x=None) == NULLP and norm(y=None) == NULLP
    assert norm(x=P + 1) == INVALID and norm(y=P + MB + 1) == INVALID and norm(rstd=P + 2 * MB + 2) == INVALID
    assert norm(xs=63) == INVALID and norm(ys=10) == INVALID and norm(r=P + 2 * MB, rs=1) == INVALID
    assert norm(xs=1 << 62) == INVALID
    assert norm(eps=-1e-9) == INVALID and norm(eps=float("nan")) == INVALID and norm(eps=float("inf")) == INVALID


def test_norm_overlap():
    row = 64 * 2
    assert norm(y=P + row) == OVERLAP                      # the next row of x
    assert norm(y=P + 2) == OVERLAP
    assert norm(y=P, ys=128) == OVERLAP                    # the same base at another stride
    assert norm(h=P + MB, hs=64) == OVERLAP                # y and h the same
    assert norm(w=P + MB + 8) == OVERLAP
    assert norm(rstd=P + MB) == OVERLAP
    # two matrices side by side in rows of 128 elements share nothing; shifted by one element they do
    assert norm(xs=128, y=P + row - 2, ys=128) == OVERLAP
    assert norm(xs=128, y=P + row + 2, ys=128) == OVERLAP  # y's row ends in x's next row
    assert norm(xs=128, x=P + row, y=P + 2, ys=128) == OVERLAP


def test_quant_refusals():
    assert quant(dt=3) == DTYPE and quant(qt=2) == DTYPE
    assert quant(group=31) == INVALID and quant(group=-32) == INVALID and quant(group=512) == INVALID
    assert quant(s=None) == NULLP and quant(q=None) == NULLP
    assert quant(ss=1) == INVALID and quant(s=P + 2 * MB + 1) == INVALID and quant(qs=63) == INVALID
    assert quant(q=P) == OVERLAP and quant(s=P + MB) == OVERLAP  # no in-place form, scales inside q
    assert quant(rows=0) == OK


def test_norm_grad_refusals():
    assert norm_grad(dt=3) == DTYPE
    assert norm_grad(rows=-1) == INVALID and norm_grad(cols=0) == INVALID
    assert norm_grad(dy=None) == NULLP and norm_grad(h=None) == NULLP and norm_grad(rstd=None) == NULLP
    assert norm_grad(dx=None) == NULLP and norm_grad(work=None) == NULLP
    need = ew.lib().ew_rmsnorm_grad_workspace(4, 64)
    assert need == 4 * 64 * 4 and norm_grad(size=need - 1) == INVALID
    assert norm_grad(work=P + 5 * MB + 128) == INVALID
    assert norm_grad(dx=P + MB) == OVERLAP and norm_grad(dx=P + 2) == OVERLAP and norm_grad(work=P) == OVERLAP
    assert norm_grad(rows=0, dw=None) == OK
    assert ew.lib().ew_rmsnorm_grad_workspace(-1, 64) == -1 and ew.lib().ew_rmsnorm_grad_workspace(4, BIG + 1) == -1
    assert ew.last_launch()["launches"] == 0


def embed(dt=2, it=1, table=P, n=100, ts=64, tokens=P + MB, out=P + 2 * MB, os_=64, rows=4, cols=64):
    return ew.lib().ew_embed(dt, it, table, n, ts, tokens, 1.0, out, os_, rows, cols, None)


def embed_grad(dt=2, it=1, dout=P, ds=64, tokens=P + MB, gt=0, dtable=P + 2 * MB, n=100, ts=64, rows=4, cols=64, acc=0,
               work=P + 8 * MB, size=8 * MB):
    return ew.lib().ew_embed_grad(dt, it, dout, ds, tokens, 1.0, gt, dtable, n, ts, rows, cols, acc, work, size, None)


def test_embed_refusals():
    assert embed(dt=3) == DTYPE and embed(it=2) == DTYPE and embed(it=-1) == DTYPE
    assert embed(rows=0, tokens=None, out=None) == OK
    assert embed(rows=-1) == INVALID and embed(cols=0) == INVALID and embed(n=-1) == INVALID and embed(n=BIG + 1) == INVALID
    assert embed(table=None) == NULLP and embed(tokens=None) == NULLP and embed(out=None) == NULLP
    assert embed(tokens=P + MB + 4) == INVALID and embed(ts=63) == INVALID and embed(out=P + 1) == INVALID
    assert embed(out=P) == OVERLAP and embed(out=P + MB) == OVERLAP


def test_embed_grad_refusals():
    assert embed_grad(dt=3) == DTYPE and embed_grad(gt=1) == DTYPE and embed_grad(it=5) == DTYPE
    assert embed_grad(acc=2) == INVALID and embed_grad(size=100) == INVALID and embed_grad(work=P + 8 * MB + 8) == INVALID
    assert embed_grad(rows=-1) == INVALID and embed_grad(cols=BIG + 1) == INVALID and embed_grad(ds=1) == INVALID
    assert embed_grad(dout=None) == NULLP and embed_grad(tokens=None) == NULLP and embed_grad(dtable=None) == NULLP
    assert embed_grad(work=None) == NULLP
    assert embed_grad(dtable=P) == OVERLAP and embed_grad(work=P) == OVERLAP
    assert embed_grad(n=0) == OK and embed_grad(rows=0, acc=1) == OK
    assert ew.lib().ew_embed_grad_workspace(100, -1, 64) == -1
    assert ew.lib().ew_embed_grad_workspace(0, 0, 1) == 0
    assert ew.last_launch()["launches"] == 0


def logprob(dt=2, it=1, x=P, s=64, tok=P + MB, scale=1.0, top=0, lp=P + 2 * MB, ent=None, lse=None, tl=P + 3 * MB,
            ti=P + 4 * MB, rows=4, cols=64):
    return ew.lib().ew_logprob(dt, it, x, s, tok, scale, top, lp, ent, lse, tl, ti, rows, cols, None)


def logprob_grad(dt=2, it=1, x=P, s=64, tok=P + MB, lse=P + 2 * MB, ent=P + 3 * MB, dlp=P + 4 * MB, dent=P + 5 * MB,
                 scale=1.0, d=P + 6 * MB, ds=64, rows=4, cols=64):
    return ew.lib().ew_logprob_grad(dt, it, x, s, tok, lse, ent, dlp, dent, scale, d, ds, rows, cols, None)


def distill_step(dt=2, it=1, x=P, s=64, ids=P + MB, ids_s=8, tt=2, t=P + 2 * MB, ts=8, k=8, scale=1.0, dloss=P + 3 * MB,
                 loss=P + 4 * MB, lse=P + 5 * MB, d=P + 6 * MB, ds=64, rows=4, cols=64):
    return ew.lib().ew_distill_step(dt, it, x, s, ids, ids_s, tt, t, ts, k, scale, dloss, loss, lse, d, ds, rows, cols,
                                    None)


def test_logprob_refusals():
    assert logprob(dt=3) == DTYPE and logprob(it=2) == DTYPE
    assert logprob(rows=-1) == INVALID and logprob(cols=0) == INVALID and logprob(s=63) == INVALID
    assert logprob(top=-1) == INVALID and logprob(top=65) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** 21):
        assert logprob(scale=scale) == INVALID and logprob_grad(scale=scale) == INVALID
        assert distill_step(scale=scale) == INVALID
    assert logprob(x=None) == NULLP and logprob(tok=None) == NULLP and logprob(top=3, ti=None) == NULLP
    assert logprob(tok=P + MB + 4) == INVALID and logprob(lp=P + 2) == INVALID
    assert logprob(lp=P) == OVERLAP and logprob(ent=P + 2 * MB) == OVERLAP and logprob(top=2, tl=P + 4 * MB) == OVERLAP
    assert logprob(rows=0, x=None) == OK


def test_logprob_grad_refusals():
    assert logprob_grad(dt=-1) == DTYPE and logprob_grad(it=9) == DTYPE
    assert logprob_grad(tok=None) == NULLP and logprob_grad(ent=None) == NULLP and logprob_grad(lse=None) == NULLP
    assert logprob_grad(d=None) == NULLP and logprob_grad(ds=10) == INVALID and logprob_grad(d=P + 1) == INVALID
    assert logprob_grad(d=P + 2) == OVERLAP and logprob_grad(d=P, ds=128) == OVERLAP and logprob_grad(d=P + MB) == OVERLAP
    assert logprob_grad(rows=0) == OK


def test_distill_refusals():
    assert distill_step(dt=3) == DTYPE and distill_step(tt=1) == DTYPE and distill_step(it=-1) == DTYPE
    assert distill_step(k=0) == INVALID and distill_step(k=1025, ids_s=1025, ts=1025) == INVALID
    assert distill_step(ids_s=7) == INVALID and distill_step(ts=7) == INVALID and distill_step(rows=BIG + 1) == INVALID
    for name in ("x", "ids", "t", "dloss", "loss", "lse", "d"):
        assert distill_step(**{name: None}) == NULLP, name
    assert distill_step(d=P + MB) == OVERLAP and distill_step(loss=P) == OVERLAP and distill_step(lse=P + 4 * MB) == OVERLAP
    assert distill_step(rows=0) == OK
    L = ew.lib()
    assert L.ew_distill(2, 1, P, 64, P + MB, 8, 2, P + 2 * MB, 8, 8, 1.0, None, P + 5 * MB, 4, 64, None) == NULLP
    assert L.ew_distill_grad(2, 1, P, 64, P + MB, 8, 2, P + 2 * MB, 8, 8, 1.0, None, P + 3 * MB, P + 6 * MB, 64, 4, 64,
                             None) == NULLP
    assert ew.last_launch()["launches"] == 0


def layernorm(dt=2, x=P, xs=64, r=None, rs=0, wt=2, w=None, b=None, eps=1e-5, y=P + MB, ys=64, h=None, hs=0, mean=None,
              rstd=None, rows=4, cols=64):
    return ew.lib().ew_layernorm(dt, x, xs, r, rs, wt, w, b, eps, y, ys, h, hs, mean, rstd, rows, cols, None)


def layernorm_grad(dt=2, dy=P, h=P + MB, mean=P + 2 * MB, rstd=P + 3 * MB, dh=None, dx=P + 4 * MB, dw=P + 5 * MB,
                   db=P + 6 * MB, rows=4, cols=64, work=P + 7 * MB, size=MB, s=64, wt=2, w=None):
    return ew.lib().ew_layernorm_grad(dt, dy, s, h, s, wt, w, mean, rstd, dh, s, dx, s, dw, db, rows, cols, work, size, None)


def test_layernorm_refusals():
    assert layernorm(dt=3) == DTYPE and layernorm(w=P + 2 * MB, wt=1) == DTYPE and layernorm(b=P + 2 * MB, wt=1) == DTYPE
    assert layernorm(rows=0, x=None, y=None) == OK and ew.last_launch()["launches"] == 0
    assert layernorm(rows=-1) == INVALID and layernorm(cols=0) == INVALID and layernorm(rows=BIG + 1) == INVALID
    assert layernorm(x=None) == NULLP and layernorm(y=None) == NULLP
    assert layernorm(x=P + 1) == INVALID and layernorm(mean=P + 2 * MB + 2) == INVALID and layernorm(b=P + 1) == INVALID
    assert layernorm(xs=63) == INVALID and layernorm(ys=10) == INVALID and layernorm(r=P + 2 * MB, rs=1) == INVALID
    for eps in (-1e-9, float("nan"), float("inf")):
        assert layernorm(eps=eps) == INVALID
    assert layernorm(y=P + 2) == OVERLAP and layernorm(y=P, ys=128) == OVERLAP and layernorm(h=P + MB, hs=64) == OVERLAP
    assert layernorm(b=P + MB + 8) == OVERLAP and layernorm(mean=P + MB) == OVERLAP
    assert layernorm(mean=P + 2 * MB, rstd=P + 2 * MB) == OVERLAP


def test_layernorm_grad_refusals():
    assert layernorm_grad(dt=3) == DTYPE and layernorm_grad(w=P + 8 * MB, wt=1) == DTYPE
    assert layernorm_grad(rows=-1) == INVALID and layernorm_grad(cols=0) == INVALID
    for name in ("dy", "h", "mean", "rstd", "dx", "work"):
        assert layernorm_grad(**{name: None}) == NULLP, name
    need = ew.lib().ew_layernorm_grad_workspace(4, 64)
    assert need == 4 * 64 * 8 and layernorm_grad(size=need - 1) == INVALID and layernorm_grad(work=P + 7 * MB + 128) == INVALID
    assert layernorm_grad(dx=P + MB) == OVERLAP and layernorm_grad(dx=P + 2) == OVERLAP and layernorm_grad(work=P) == OVERLAP
    assert layernorm_grad(db=P + 5 * MB) == OVERLAP and layernorm_grad(db=P + 7 * MB + 64) == OVERLAP
    assert layernorm_grad(rows=0, dw=None, db=None) == OK
    assert ew.lib().ew_layernorm_grad_workspace(-1, 64) == -1 and ew.lib().ew_layernorm_grad_workspace(4, BIG + 1) == -1
    assert ew.last_launch()["launches"] == 0


def expert_sort(it=0, e=P, es=2, n=8, align=1, pos=P + MB, off=P + 2 * MB, cnt=P + 3 * MB, slots=P + 4 * MB, cap=8, rows=4, k=2,
                work=None, size=0):
    return ew.lib().ew_expert_sort(it, e, es, n, align, pos, off, cnt, slots, cap, rows, k, work, size, None)


def dispatch(dt=2, x=P, xs=64, pos=P + MB, slots=P + 2 * MB, out=P + 3 * MB, os_=64, cap=8, rows=4, k=2, cols=64):
    return ew.lib().ew_expert_dispatch(dt, x, xs, pos, slots, out, os_, cap, rows, k, cols, None)


def combine(dt=2, y=P, ys=64, cap=8, pos=P + MB, wt=0, w=P + 2 * MB, r=P + 3 * MB, rs=64, out=P + 4 * MB, os_=64, rows=4, k=2,
            cols=64):
    return ew.lib().ew_expert_combine(dt, y, ys, cap, pos, wt, w, r, rs, out, os_, rows, k, cols, None)


def combine_grad(dt=2, dout=P, ds=64, y=P + MB, ys=64, cap=8, pos=P + 2 * MB, slots=P + 3 * MB, wt=0, w=P + 4 * MB,
                 dy=P + 5 * MB, dys=64, dw=P + 6 * MB, rows=4, k=2, cols=64):
    return ew.lib().ew_expert_combine_grad(dt, dout, ds, y, ys, cap, pos, slots, wt, w, dy, dys, dw, rows, k, cols, None)


def test_expert_capacity():
    cap = ew.lib().ew_expert_capacity
    assert cap(4, 2, 8, 1) == 8 and cap(0, 2, 8, 16) == 0
    assert cap(1, 8, 256, 128) == 8 * 128          # eight experts of one slot each
    assert cap(100, 1, 3, 8) == (100 + 3 * 7) // 8 * 8
    for bad in ((-1, 2, 8, 1), (4, 0, 8, 1), (4, 65, 8, 1), (4, 2, 0, 1), (4, 2, 1025, 1), (4, 2, 8, 0), (4, 2, 8, 65537),
                (BIG // 2 + 1, 2, 8, 1), (BIG // 2, 2, 8, 2), (BIG + 1, 1, 8, 1)):
        assert cap(*bad) == -1, bad
    # whatever the choices are, the rows suffice: the fullest case by brute force
    for rows, n, align in ((5, 3, 4), (7, 2, 3), (2, 6, 5)):
        most = max(sum(-(-c // align) * align for c in split) for split in splits(rows, n))
        assert cap(rows, 1, n, align) >= most and cap(rows, 1, n, align) - most < align


def splits(total, parts):
    if parts == 1:
        yield (total,)
        return
    for first in range(total + 1):
        for rest in splits(total - first, parts - 1):
            yield (first, *rest)


def test_expert_sort_refusals():
    assert expert_sort(it=2) == DTYPE and expert_sort(k=65) == INVALID and expert_sort(n=1025) == INVALID
    assert expert_sort(cap=7) == INVALID and expert_sort(cap=BIG + 1) == INVALID and expert_sort(align=2) == INVALID
    assert expert_sort(es=1) == INVALID and expert_sort(e=P + 2) == INVALID and expert_sort(rows=-1) == INVALID
    for name in ("e", "pos", "off", "cnt", "slots"):
        assert expert_sort(**{name: None}) == NULLP, name
    assert expert_sort(pos=P) == OVERLAP and expert_sort(cnt=P + 2 * MB + 32) == OVERLAP
    need = ew.lib().ew_expert_sort_workspace
    assert need(4, 2, 8) == 0 and need(-1, 2, 8) == -1 and need(4, 2, 1025) == -1
    big = need(100000, 2, 8)
    assert big > 0
    args = dict(rows=100000, cap=200000, n=8, e=P, pos=P + 8 * MB, slots=P + 16 * MB, off=P + 32 * MB, cnt=P + 33 * MB)
    assert expert_sort(**args, size=big - 1, work=P + 40 * MB) == INVALID and expert_sort(**args, size=big) == NULLP
    assert expert_sort(**args, size=big, work=P + 40 * MB + 64) == INVALID and expert_sort(**args, size=big, work=P + 33 * MB) == OVERLAP
    assert ew.last_launch()["launches"] == 0


def test_expert_rows_refusals():
    for call, names in ((dispatch, ("x", "pos", "slots", "out")), (combine, ("y", "pos", "out")),
                        (combine_grad, ("dout", "y", "pos", "slots", "dy"))):
        assert call(dt=3) == DTYPE and call(k=0) == INVALID and call(k=65) == INVALID and call(cols=0) == INVALID
        assert call(rows=-1) == INVALID and call(cap=-1) == INVALID and call(cap=BIG + 1) == INVALID
        for name in names:
            assert call(**{name: None}) == NULLP, (call.__name__, name)
        assert call(pos=P + MB // 2 + 2) == INVALID
    assert dispatch(rows=0, cap=0) == OK and combine(rows=0) == OK and combine_grad(rows=0, cap=0) == OK
    assert combine(wt=1) == DTYPE and combine_grad(wt=1) == DTYPE
    assert dispatch(xs=63) == INVALID and combine(rs=63) == INVALID and combine_grad(dys=63) == INVALID
    assert dispatch(out=P) == OVERLAP and combine(out=P) == OVERLAP and combine(out=P + 3 * MB, os_=128) == OVERLAP
    assert combine_grad(dy=P + MB) == OVERLAP and combine_grad(dy=P) == OVERLAP and combine_grad(dw=P + 4 * MB) == OVERLAP
    assert combine_grad(dw=None, y=None, dy=P) == OVERLAP
    assert ew.last_launch()["launches"] == 0


def policy_step(dt=2, it=1, x=P, s=64, tok=P + MB, adv=P + 2 * MB, old=P + 3 * MB, ref=P + 4 * MB, low=0.2, high=0.2, kl=0.1,
                scale=1.0, dloss=P + 5 * MB, loss=P + 6 * MB, lp=P + 7 * MB, lse=P + 8 * MB, d=P + 9 * MB, ds=64, rows=4, cols=64):
    return ew.lib().ew_policy_step(dt, it, x, s, tok, adv, old, ref, low, high, kl, scale, dloss, loss, lp, lse, d, ds, rows,
                                   cols, None)


def test_policy_refusals():
    assert policy_step(dt=3) == DTYPE and policy_step(it=2) == DTYPE
    assert policy_step(rows=-1) == INVALID and policy_step(cols=0) == INVALID and policy_step(s=63) == INVALID
    nan, inf = float("nan"), float("inf")
    for how in (dict(low=-0.1), dict(low=1.5), dict(low=nan), dict(high=-1e-9), dict(high=nan), dict(kl=-1.0), dict(kl=inf),
                dict(kl=nan), dict(scale=0.0), dict(scale=2.0 ** 21), dict(scale=nan)):
        assert policy_step(**how) == INVALID, how
    for name in ("x", "tok", "adv", "dloss", "loss", "d"):
        assert policy_step(**{name: None}) == NULLP, name
    assert policy_step(tok=P + MB + 4) == INVALID and policy_step(lse=P + 2) == INVALID and policy_step(ds=10) == INVALID
    assert policy_step(d=P + 2) == OVERLAP and policy_step(d=P, ds=128) == OVERLAP and policy_step(loss=P) == OVERLAP
    assert policy_step(lp=P + 8 * MB) == OVERLAP and policy_step(lse=P + 2 * MB) == OVERLAP
    assert policy_step(rows=0, x=None, high=inf) == OK
    L = ew.lib()
    args = (P, 64, P + MB, P + 2 * MB, None, None, 0.2, 0.2, 0.0, 1.0)
    assert L.ew_policy(2, 1, *args, None, None, None, 4, 64, None) == NULLP
    assert L.ew_policy_grad(2, 1, *args, None, P + 3 * MB, P + 4 * MB, P + 5 * MB, 64, 4, 64, None) == NULLP
    assert L.ew_policy_grad(2, 1, *args, P + 3 * MB, None, P + 4 * MB, P + 5 * MB, 64, 4, 64, None) == NULLP
    assert L.ew_policy_grad(2, 1, *args, P + 6 * MB, P + 3 * MB, P + 4 * MB, P + 3 * MB, 64, 4, 64, None) == OVERLAP
    assert ew.last_launch()["launches"] == 0
