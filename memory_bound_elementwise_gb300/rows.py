"""Row operators: torch entry points over the C ABI (include/ew.h, "row operators").

Matrices are CUDA tensors whose last dimension is contiguous.  Two-dimensional
ones may have any row stride; others are contiguous and count as rows of their
last dimension.  Outputs that are not given are allocated; calls are enqueued
on ``stream`` (default: torch's current stream) and do not synchronise.  What is
allocated belongs to that stream.  Arguments that do not fit raise ``ValueError``
or ``TypeError``, and ``EwError`` carries the library's status.

Gradients are calls of their own (``ew_*_grad``, ``ew_distill_step``): autograd does
not see these functions.  Results require no gradient whatever the inputs do, and
writing to a given output leaves its version counter as it is.  To use them in a
graph, wrap forward and backward calls in a ``torch.autograd.Function``.

The checks, allocations and calls are in the compiled binding
(csrc/ew_torch.cpp), built beside libew.so.
"""
import collections
import importlib.machinery
import importlib.util
import os

import torch

from . import LIB_PATH, check, lib


def _load():
    lib()  # says how to build what is missing
    path = os.path.join(os.path.dirname(LIB_PATH), "_ew_torch.so")
    if not os.path.exists(path):
        raise RuntimeError("the torch binding is not built (%s). Build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`." % path)
    loader = importlib.machinery.ExtensionFileLoader("_ew_torch", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_ew_torch", loader))
    loader.exec_module(module)
    module.set_check(check)
    return module


_C = _load()
_QTYPES = {torch.float8_e4m3fn: False, torch.int8: True}


def _on(stream, call, *args):
    """The same call with ``stream`` as torch's current stream: its allocations belong to it."""
    with torch.cuda.stream(stream):
        return call(*args)


# ---------------------------------------------------------------- embedding

def ew_embed(table, tokens, out=None, scale=1.0, stream=None):
    """out[t] = scale * table[tokens[t]]; returns out, of tokens' shape by the table's columns.

    A token outside the table gives a row of zeros."""
    if stream is not None:
        return _on(stream, ew_embed, table, tokens, out, scale)
    return _C.embed(table, tokens, out, scale)


def ew_embed_grad(dout, tokens, table_rows, dtable=None, scale=1.0, accumulate=False, stream=None):
    """Gradient of ew_embed for a table of ``table_rows`` rows; returns dtable.

    dtable has dout's dtype or float32; it is written whole, or with
    ``accumulate`` the gradient is added to what it holds.  The same tokens and
    values give the same bits each time."""
    if stream is not None:
        return _on(stream, ew_embed_grad, dout, tokens, table_rows, dtable, scale, accumulate)
    return _C.embed_grad(dout, tokens, table_rows, dtable, scale, accumulate)


# ---------------------------------------------------------------- norm

def ew_rmsnorm(x, weight, residual=None, eps=1e-6, y=None, h=None, rstd=None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) * weight with h = x + residual; returns (y, h, rstd).

    ``weight`` has x's dtype or float32 (None: ones).  Without a residual h is
    x, or, where y is x, a copy of it.  ``rstd`` (float32, one a row) and ``h`` are
    what ew_rmsnorm_grad takes.  y may be x or residual, h may be x or residual,
    for in place."""
    if stream is not None:
        return _on(stream, ew_rmsnorm, x, weight, residual, eps, y, h, rstd)
    return _C.rmsnorm(x, weight, residual, eps, y, h, rstd)


def ew_rmsnorm_quant(x, weight, residual=None, eps=1e-6, group=0, q=None, scales=None, h=None, rstd=None,
                     dtype=torch.float8_e4m3fn, stream=None):
    """The norm with an 8-bit output: returns (q, scales, h, rstd), q * scale standing for y.

    ``dtype`` is torch.float8_e4m3fn or torch.int8; ``group`` is 32, 64, 128 or
    256 columns a scale, or 0 for one scale a row; scales: float32, rows x groups."""
    if stream is not None:
        return _on(stream, ew_rmsnorm_quant, x, weight, residual, eps, group, q, scales, h, rstd, dtype)
    int8 = _QTYPES.get(dtype if q is None else q.dtype)
    if int8 is None:
        raise TypeError("dtype: float8_e4m3fn or int8, got %s" % (dtype if q is None else q.dtype))
    return _C.rmsnorm_quant(x, weight, residual, eps, group, q, scales, h, rstd, int8)


def ew_rmsnorm_grad(dy, h, weight, rstd, dh=None, dx=None, dweight=None, stream=None):
    """Gradients of ew_rmsnorm: returns (dx, dweight), dx for x and for the residual alike.

    ``h`` and ``rstd`` come from the forward call; ``dh`` is the gradient that
    reaches h by the residual stream.  dweight is float32.  dx may be dy or dh."""
    if stream is not None:
        return _on(stream, ew_rmsnorm_grad, dy, h, weight, rstd, dh, dx, dweight)
    return _C.rmsnorm_grad(dy, h, weight, rstd, dh, dx, dweight)


# ---------------------------------------------------------------- logits

Logprobs = collections.namedtuple("Logprobs", "logp entropy lse top_logp top_ids")


def ew_logprob(logits, tokens, top=0, scale=1.0, stream=None):
    """Log probabilities under softmax(scale * logits), one row a token.

    Returns Logprobs(logp, entropy, lse, top_logp, top_ids): float32, one a row,
    and the ``top`` (at most 64) largest logits' log probabilities and int32
    columns, largest first, equal ones by the lower column.  A token outside
    the row (such as -1) has logp 0.  ``tokens`` may be None: then logp is None."""
    if stream is not None:
        return _on(stream, ew_logprob, logits, tokens, top, scale)
    return Logprobs._make(_C.logprob(logits, tokens, top, scale))


def ew_logprob_grad(logits, tokens, lse, entropy, dlogp, dentropy=None, scale=1.0, dlogits=None, stream=None):
    """Gradient with respect to the logits of ew_logprob's logp (times dlogp) and entropy (times dentropy); returns
    dlogits, which may be logits.  dlogp or dentropy may be None.  Rows whose lse is 4096 or more in size are
    summed again, as float32 does not hold their normalisation."""
    if stream is not None:
        return _on(stream, ew_logprob_grad, logits, tokens, lse, entropy, dlogp, dentropy, scale, dlogits)
    return _C.logprob_grad(logits, tokens, lse, entropy, dlogp, dentropy, scale, dlogits)


def ew_distill(logits, ids, teacher, scale=1.0, stream=None):
    """Distillation from a teacher's top logits: returns (loss, lse), float32, one a row.

    ``ids`` (int32 or int64) and ``teacher`` are rows x k: columns of the logits
    and the teacher's logits there; an id of -1 does not count.  The loss is the
    divergence of softmax(scale * logits) from softmax(scale * teacher) over the
    k entries; scale is 1 / temperature."""
    if stream is not None:
        return _on(stream, ew_distill, logits, ids, teacher, scale)
    return _C.distill(logits, ids, teacher, scale)


def ew_distill_grad(logits, ids, teacher, lse, dloss, scale=1.0, dlogits=None, stream=None):
    """Gradient of ew_distill's loss (times dloss, float32, one a row) with respect to the logits, from its lse;
    returns dlogits, which may be logits."""
    if stream is not None:
        return _on(stream, ew_distill_grad, logits, ids, teacher, lse, dloss, scale, dlogits)
    return _C.distill_grad(logits, ids, teacher, lse, dloss, scale, dlogits)


def ew_distill_step(logits, ids, teacher, dloss, scale=1.0, dlogits=None, stream=None):
    """ew_distill and ew_distill_grad in one call, where dloss is known beforehand; returns (loss, lse, dlogits)."""
    if stream is not None:
        return _on(stream, ew_distill_step, logits, ids, teacher, dloss, scale, dlogits)
    return _C.distill_step(logits, ids, teacher, dloss, scale, dlogits)
