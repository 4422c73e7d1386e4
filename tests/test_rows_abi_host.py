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
