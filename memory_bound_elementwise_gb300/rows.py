"""Row operators: torch entry points over the C ABI (include/ew.h, "row operators").

Matrices are CUDA tensors whose last dimension is contiguous.  Two-dimensional
ones may have any row stride; others are contiguous and count as rows of their
last dimension.  Outputs that are not given are allocated; calls are enqueued
on ``stream`` (default: torch's current stream) and do not synchronise.  What is
allocated belongs to that stream.  Arguments that do not fit raise ``ValueError``
or ``TypeError`` here, or ``EwError`` with the library's status.
"""
import collections
import contextlib

import torch

_F32, _F16, _BF16 = 0, 1, 2
_CODES = {torch.float32: _F32, torch.float16: _F16, torch.bfloat16: _BF16}
_INDEX = {torch.int32: 0, torch.int64: 1}
_QTYPES = {torch.float8_e4m3fn: 0, torch.int8: 1}

_fns = {}


def _call(name, *args):
    fn = _fns.get(name)
    if fn is None:
        from . import lib
        fn = _fns[name] = getattr(lib(), name)
    status = fn(*args)
    if status != 0:
        from . import check
        check(status, name)


def _bytes(name, *args):
    """A workspace function's answer."""
    fn = _fns.get(name)
    if fn is None:
        from . import lib
        fn = _fns[name] = getattr(lib(), name)
    n = fn(*args)
    if n < 0:
        raise ValueError("%s: sizes out of range" % name)
    return n


def _code(t, what):
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError("%s: unsupported dtype %s (float32, float16, bfloat16)" % (what, t.dtype))
    return c


def _matrix(t, what, device):
    """(rows, cols, stride) of a tensor as a matrix of its last dimension."""
    if t.device != device:
        raise ValueError("%s must be on %s" % (what, device))
    shape = t.shape
    if len(shape) == 2:
        rows, cols = shape
        stride, inner = t.stride()
        if rows <= 1 and stride < cols:
            stride = cols  # the stride of a single row says nothing
        if (inner == 1 or cols == 1) and (stride >= cols or rows <= 1):
            return rows, cols, stride
    elif len(shape) >= 1 and t.is_contiguous():
        cols = shape[-1]
        return (t.numel() // cols if cols else 0), cols, cols
    raise ValueError("%s: a matrix needs a contiguous last dimension and rows that do not overlap" % what)


def _like(t, what, rows, cols, dtype, device):
    """The row stride of a tensor that has to be rows x cols of dtype."""
    r, c, stride = _matrix(t, what, device)
    if r != rows or c != cols or t.dtype != dtype:
        raise ValueError("%s: expected %d x %d of %s, got %s of %s" % (what, rows, cols, dtype, tuple(t.shape), t.dtype))
    return stride


def _vector(t, what, n, dtype, device):
    if t.device != device or t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s: expected %d contiguous elements of %s on %s" % (what, n, dtype, device))
    return t.data_ptr()


def _cuda_device(t, what):
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % what)
    device = t.device
    if device.index != torch.cuda.current_device():
        raise ValueError("%s must be on the current device" % what)
    return device


def _raw_stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


_here = contextlib.nullcontext()


def _allocating(stream):
    """Allocations inside belong to the stream that the call runs on."""
    return _here if stream is None else torch.cuda.stream(stream)


def _tokens(t, what, n, device):
    """(type code, pointer) of n token ids."""
    code = _INDEX.get(t.dtype)
    if code is None:
        raise TypeError("%s: int32 or int64, got %s" % (what, t.dtype))
    return code, _vector(t, what, n, t.dtype, device)


def ew_embed(table, tokens, out=None, scale=1.0, stream=None):
    """out[t] = scale * table[tokens[t]]; returns out, of tokens' shape by the table's columns.

    A token outside the table gives a row of zeros."""
    device = _cuda_device(table, "table")
    code = _code(table, "table")
    table_rows, cols, stride = _matrix(table, "table", device)
    rows = tokens.numel()
    icode, iptr = _tokens(tokens, "tokens", rows, device)
    if out is None:
        with _allocating(stream):
            out = torch.empty((*tokens.shape, cols), dtype=table.dtype, device=device)
        out_stride = cols
    else:
        out_stride = _like(out, "out", rows, cols, table.dtype, device)
    _call("ew_embed", code, icode, table.data_ptr(), table_rows, stride, iptr, scale, out.data_ptr(), out_stride, rows,
          cols, _raw_stream(stream, device))
    return out


def ew_embed_grad(dout, tokens, table_rows, dtable=None, scale=1.0, accumulate=False, stream=None):
    """Gradient of ew_embed for a table of ``table_rows`` rows; returns dtable.

    dtable has dout's dtype or float32; it is written whole, or with
    ``accumulate`` the gradient is added to what it holds.  The same tokens and
    values give the same bits each time."""
    device = _cuda_device(dout, "dout")
    code = _code(dout, "dout")
    rows, cols, stride = _matrix(dout, "dout", device)
    icode, iptr = _tokens(tokens, "tokens", rows, device)
    if dtable is None and accumulate:
        raise ValueError("accumulate needs a dtable to add to")
    if dtable is not None and dtable.dtype != dout.dtype and dtable.dtype != torch.float32:
        raise TypeError("dtable: %s or float32, got %s" % (dout.dtype, dtable.dtype))
    with _allocating(stream):
        if dtable is None:
            dtable = torch.empty((table_rows, cols), dtype=dout.dtype, device=device)
            table_stride = cols
        else:
            table_stride = _like(dtable, "dtable", table_rows, cols, dtable.dtype, device)
        need = _bytes("ew_embed_grad_workspace", table_rows, rows, cols)
        work = torch.empty(need, dtype=torch.uint8, device=device)
    _call("ew_embed_grad", code, icode, dout.data_ptr(), stride, iptr, scale, _CODES[dtable.dtype], dtable.data_ptr(),
          table_rows, table_stride, rows, cols, 1 if accumulate else 0, work.data_ptr(), need,
          _raw_stream(stream, device))
    return dtable


def _weight(weight, cols, dtype, code, device):
    """(type code, pointer) of a norm's weight."""
    if weight is None:
        return code, None
    if weight.dtype != dtype and weight.dtype != torch.float32:
        raise TypeError("weight: %s or float32, got %s" % (dtype, weight.dtype))
    return _CODES[weight.dtype], _vector(weight, "weight", cols, weight.dtype, device)


def _norm_inputs(x, weight, residual, h, rstd):
    """What both norm calls take: checked and with the outputs h and rstd allocated."""
    device = _cuda_device(x, "x")
    code = _code(x, "x")
    dtype = x.dtype
    rows, cols, x_stride = _matrix(x, "x", device)
    wcode, wptr = _weight(weight, cols, dtype, code, device)
    r_ptr, r_stride, h_ptr, h_stride = None, 0, None, 0
    if residual is not None:
        r_ptr, r_stride = residual.data_ptr(), _like(residual, "residual", rows, cols, dtype, device)
        if h is None:
            h = torch.empty(x.shape, dtype=dtype, device=device)
            h_ptr, h_stride = h.data_ptr(), cols
    if h is None:
        h = x  # without a residual h is x: nothing to write
    elif h_ptr is None:
        h_ptr, h_stride = h.data_ptr(), _like(h, "h", rows, cols, dtype, device)
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=device)
        rstd_ptr = rstd.data_ptr()
    else:
        rstd_ptr = _vector(rstd, "rstd", rows, torch.float32, device)
    head = (code, x.data_ptr(), x_stride, r_ptr, r_stride, wcode, wptr)
    return device, dtype, rows, cols, h, rstd, head, (h_ptr, h_stride, rstd_ptr, rows, cols)


def ew_rmsnorm(x, weight, residual=None, eps=1e-6, y=None, h=None, rstd=None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) * weight with h = x + residual; returns (y, h, rstd).

    ``weight`` has x's dtype or float32 (None: ones).  Without a residual h is
    x.  ``rstd`` (float32, one a row) and ``h`` are what ew_rmsnorm_grad takes.
    y may be x or residual, h may be x or residual, for in place."""
    with _allocating(stream):
        device, dtype, rows, cols, h, rstd, head, tail = _norm_inputs(x, weight, residual, h, rstd)
        if y is None:
            y = torch.empty(x.shape, dtype=dtype, device=device)
            y_stride = cols
        else:
            y_stride = _like(y, "y", rows, cols, dtype, device)
    _call("ew_rmsnorm", *head, eps, y.data_ptr(), y_stride, *tail, _raw_stream(stream, device))
    return y, h, rstd


def ew_rmsnorm_quant(x, weight, residual=None, eps=1e-6, group=0, q=None, scales=None, h=None, rstd=None,
                     dtype=torch.float8_e4m3fn, stream=None):
    """The norm with an 8-bit output: returns (q, scales, h, rstd), q * scale standing for y.

    ``dtype`` is torch.float8_e4m3fn or torch.int8; ``group`` is 32, 64, 128 or
    256 columns a scale, or 0 for one scale a row; scales: float32, rows x groups."""
    if q is not None:
        dtype = q.dtype
    if dtype not in _QTYPES:
        raise TypeError("dtype: float8_e4m3fn or int8, got %s" % dtype)
    with _allocating(stream):
        device, _, rows, cols, h, rstd, head, tail = _norm_inputs(x, weight, residual, h, rstd)
        groups = -(-cols // group) if group > 0 else 1
        if q is None:
            q = torch.empty(x.shape, dtype=dtype, device=device)
            q_stride = cols
        else:
            q_stride = _like(q, "q", rows, cols, dtype, device)
        if scales is None:
            scales = torch.empty((rows, groups), dtype=torch.float32, device=device)
            s_stride = groups
        else:
            s_stride = _like(scales, "scales", rows, groups, torch.float32, device)
    _call("ew_rmsnorm_quant", *head, eps, _QTYPES[dtype], group, q.data_ptr(), q_stride, scales.data_ptr(), s_stride,
          *tail, _raw_stream(stream, device))
    return q, scales, h, rstd


def ew_rmsnorm_grad(dy, h, weight, rstd, dh=None, dx=None, dweight=None, stream=None):
    """Gradients of ew_rmsnorm: returns (dx, dweight), dx for x and for the residual alike.

    ``h`` and ``rstd`` come from the forward call; ``dh`` is the gradient that
    reaches h by the residual stream.  dweight is float32.  dx may be dy or dh."""
    device = _cuda_device(dy, "dy")
    code, dtype = _code(dy, "dy"), dy.dtype
    rows, cols, dy_stride = _matrix(dy, "dy", device)
    h_stride = _like(h, "h", rows, cols, dtype, device)
    wcode, wptr = _weight(weight, cols, dtype, code, device)
    r_ptr = _vector(rstd, "rstd", rows, torch.float32, device)
    dh_ptr, dh_stride = (None, 0) if dh is None else (dh.data_ptr(), _like(dh, "dh", rows, cols, dtype, device))
    with _allocating(stream):
        if dx is None:
            dx = torch.empty(dy.shape, dtype=dtype, device=device)
            dx_stride = cols
        else:
            dx_stride = _like(dx, "dx", rows, cols, dtype, device)
        if dweight is None:
            dweight = torch.empty(cols, dtype=torch.float32, device=device)
            dw_ptr = dweight.data_ptr()
        else:
            dw_ptr = _vector(dweight, "dweight", cols, torch.float32, device)
        need = _bytes("ew_rmsnorm_grad_workspace", rows, cols)
        work = torch.empty(need, dtype=torch.uint8, device=device)
    _call("ew_rmsnorm_grad", code, dy.data_ptr(), dy_stride, h.data_ptr(), h_stride, wcode, wptr, r_ptr, dh_ptr,
          dh_stride, dx.data_ptr(), dx_stride, dw_ptr, rows, cols, work.data_ptr(), need, _raw_stream(stream, device))
    return dx, dweight


Logprobs = collections.namedtuple("Logprobs", "logp entropy lse top_logp top_ids")


def ew_logprob(logits, tokens, top=0, scale=1.0, stream=None):
    """Log probabilities under softmax(scale * logits), one row a token.

    Returns Logprobs(logp, entropy, lse, top_logp, top_ids): float32, one a row,
    and the ``top`` (at most 64) largest logits' log probabilities and int32
    columns, largest first, equal ones by the lower column.  A token outside
    the row (such as -1) has logp 0.  ``tokens`` may be None: then logp is None."""
    device = _cuda_device(logits, "logits")
    code = _code(logits, "logits")
    rows, cols, stride = _matrix(logits, "logits", device)
    icode, iptr = (0, None) if tokens is None else _tokens(tokens, "tokens", rows, device)
    with _allocating(stream):
        each = torch.empty((3, rows), dtype=torch.float32, device=device)
        top_logp = torch.empty((rows, top), dtype=torch.float32, device=device)
        top_ids = torch.empty((rows, top), dtype=torch.int32, device=device)
    at, step = each.data_ptr(), 4 * rows
    _call("ew_logprob", code, icode, logits.data_ptr(), stride, iptr, scale, top, at if iptr else None, at + step,
          at + 2 * step, top_logp.data_ptr(), top_ids.data_ptr(), rows, cols, _raw_stream(stream, device))
    logp, entropy, lse = each.unbind(0)
    return Logprobs(None if tokens is None else logp, entropy, lse, top_logp, top_ids)


def ew_logprob_grad(logits, tokens, lse, entropy, dlogp, dentropy=None, scale=1.0, dlogits=None, stream=None):
    """Gradient with respect to the logits of ew_logprob's logp (times dlogp) and entropy (times dentropy); returns
    dlogits, which may be logits.  dlogp or dentropy may be None."""
    device = _cuda_device(logits, "logits")
    code, dtype = _code(logits, "logits"), logits.dtype
    rows, cols, stride = _matrix(logits, "logits", device)
    icode, iptr, dlogp_ptr = 0, None, None
    if dlogp is not None:
        icode, iptr = _tokens(tokens, "tokens", rows, device)
        dlogp_ptr = _vector(dlogp, "dlogp", rows, torch.float32, device)
    lse_ptr = _vector(lse, "lse", rows, torch.float32, device)
    ent_ptr, dent_ptr = None, None
    if dentropy is not None:
        ent_ptr = _vector(entropy, "entropy", rows, torch.float32, device)
        dent_ptr = _vector(dentropy, "dentropy", rows, torch.float32, device)
    dlogits, dstride = _gradient_of(logits, dlogits, rows, cols, dtype, device, stream)
    _call("ew_logprob_grad", code, icode, logits.data_ptr(), stride, iptr, lse_ptr, ent_ptr, dlogp_ptr, dent_ptr, scale,
          dlogits.data_ptr(), dstride, rows, cols, _raw_stream(stream, device))
    return dlogits


def _gradient_of(logits, dlogits, rows, cols, dtype, device, stream):
    if dlogits is not None:
        return dlogits, _like(dlogits, "dlogits", rows, cols, dtype, device)
    with _allocating(stream):
        return torch.empty(logits.shape, dtype=dtype, device=device), cols


def _distill_inputs(logits, ids, teacher):
    device = _cuda_device(logits, "logits")
    code = _code(logits, "logits")
    rows, cols, stride = _matrix(logits, "logits", device)
    icode = _INDEX.get(ids.dtype)
    if icode is None:
        raise TypeError("ids: int32 or int64, got %s" % ids.dtype)
    if teacher.dtype != logits.dtype and teacher.dtype != torch.float32:
        raise TypeError("teacher: %s or float32, got %s" % (logits.dtype, teacher.dtype))
    n, k, ids_stride = _matrix(ids, "ids", device)
    if n != rows:
        raise ValueError("ids: expected %d rows, got %d" % (rows, n))
    teacher_stride = _like(teacher, "teacher", rows, k, teacher.dtype, device)
    head = (code, icode, logits.data_ptr(), stride, ids.data_ptr(), ids_stride, _CODES[teacher.dtype],
            teacher.data_ptr(), teacher_stride, k)
    return device, rows, cols, head


def ew_distill(logits, ids, teacher, scale=1.0, stream=None):
    """Distillation from a teacher's top logits: returns (loss, lse), float32, one a row.

    ``ids`` (int32 or int64) and ``teacher`` are rows x k: columns of the logits
    and the teacher's logits there; an id of -1 does not count.  The loss is the
    divergence of softmax(scale * logits) from softmax(scale * teacher) over the
    k entries; scale is 1 / temperature."""
    device, rows, cols, head = _distill_inputs(logits, ids, teacher)
    with _allocating(stream):
        each = torch.empty((2, rows), dtype=torch.float32, device=device)
    at = each.data_ptr()
    _call("ew_distill", *head, scale, at, at + 4 * rows, rows, cols, _raw_stream(stream, device))
    return each.unbind(0)


def ew_distill_grad(logits, ids, teacher, lse, dloss, scale=1.0, dlogits=None, stream=None):
    """Gradient of ew_distill's loss (times dloss, float32, one a row) with respect to the logits, from its lse;
    returns dlogits, which may be logits."""
    device, rows, cols, head = _distill_inputs(logits, ids, teacher)
    lse_ptr = _vector(lse, "lse", rows, torch.float32, device)
    dloss_ptr = _vector(dloss, "dloss", rows, torch.float32, device)
    dlogits, dstride = _gradient_of(logits, dlogits, rows, cols, logits.dtype, device, stream)
    _call("ew_distill_grad", *head, scale, lse_ptr, dloss_ptr, dlogits.data_ptr(), dstride, rows, cols,
          _raw_stream(stream, device))
    return dlogits


def ew_distill_step(logits, ids, teacher, dloss, scale=1.0, dlogits=None, stream=None):
    """ew_distill and ew_distill_grad in one call, where dloss is known beforehand; returns (loss, lse, dlogits)."""
    device, rows, cols, head = _distill_inputs(logits, ids, teacher)
    dloss_ptr = _vector(dloss, "dloss", rows, torch.float32, device)
    dlogits, dstride = _gradient_of(logits, dlogits, rows, cols, logits.dtype, device, stream)
    with _allocating(stream):
        each = torch.empty((2, rows), dtype=torch.float32, device=device)
    at = each.data_ptr()
    _call("ew_distill_step", *head, scale, dloss_ptr, at, at + 4 * rows, dlogits.data_ptr(), dstride, rows, cols,
          _raw_stream(stream, device))
    loss, lse = each.unbind(0)
    return loss, lse, dlogits
