"""Helpers for the row operators' tests: matrices with strides and offsets
inside guarded buffers, and error bounds.

Bounds follow from the arithmetic: one rounding to a type of p significand
bits is off by at most 2^-p relatively (and half the smallest subnormal), and a
binary32 sum of m terms by at most m * 2^-24 times the sum of their sizes.
"""
import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}    # one rounding, relative
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # and absolute
EPS32 = 2.0 ** -24
GUARD = 512


class Guarded:
    """A rows x cols matrix of row stride cols + pad, ``offset`` elements past a
    256-byte boundary, all other elements of its buffer holding a sentinel byte."""

    def __init__(self, rows, cols, dtype, pad=0, offset=0, fill=None, device="cuda"):
        size = torch.empty(0, dtype=dtype).element_size()
        self.stride, self.rows, self.cols = cols + pad, rows, cols
        n = (rows - 1) * self.stride + cols if rows else 0
        self.lo = GUARD + offset * size
        self.raw = torch.full((self.lo + n * size + GUARD,), 0x5A, dtype=torch.uint8, device=device)
        body = self.raw[self.lo:self.lo + n * size]
        if dtype in (torch.float8_e4m3fn, torch.int8):
            flat = body.view(torch.int8).view(dtype)
        else:
            flat = body.view(dtype) if offset == 0 else _view(self.raw, self.lo, n, dtype)
        self.t = torch.as_strided(flat, (rows, cols), (self.stride, 1)) if rows else flat.new_empty(0, cols)
        self.before = None
        if fill is not None:
            self.t.copy_(fill)
        self.before = self._outside()

    def _outside(self):
        keep = self.raw.clone()
        mask = torch.ones_like(keep, dtype=torch.bool)
        size = self.t.element_size()
        if self.rows:
            at = torch.arange(self.rows, device=keep.device)[:, None] * self.stride * size + self.lo
            mask[(at + torch.arange(self.cols * size, device=keep.device)).reshape(-1)] = False
        return keep[mask]

    def intact(self):
        """No byte outside the matrix has changed."""
        return torch.equal(self._outside(), self.before)


def _view(raw, lo, n, dtype):
    size = torch.empty(0, dtype=dtype).element_size()
    store = raw.untyped_storage()
    return torch.empty(0, dtype=dtype, device=raw.device).set_(store, (raw.storage_offset() + lo) // size, (n,))


def assert_within(got, want, bound, what=""):
    """|got - want| <= bound elementwise; NaN and infinities have to match."""
    got, want = got.double(), want.double()
    bound = torch.as_tensor(bound, dtype=torch.float64, device=want.device).expand_as(want)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what + ": infinities differ"
    off = torch.where(fine, (got - want).abs() - bound, torch.full_like(want, -1.0))
    worst = int(off.argmax()) if off.numel() else 0
    assert not off.numel() or float(off.max()) <= 0, "%s: at %d got %r want %r bound %r" % (
        what, worst, float(got.reshape(-1)[worst]), float(want.reshape(-1)[worst]),
        float(bound.reshape(-1)[worst]))


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, seed, dtype=torch.float32, spread=1.0):
    return (torch.randn(shape, generator=generator(seed), device="cuda") * spread).to(dtype)
