"""Shared pieces of the 8-bit operators' GPU tests: matrices inside larger buffers of sentinel bytes, and
comparisons with the 64-bit oracle whose bounds follow from the number of fp32 roundings."""

import numpy as np
import torch

from oracle import q8

U16 = 2.0 ** -8             # bf16: half a unit in the last place, relative
U32 = 2.0 ** -24            # fp32
SENTINEL = 0xA5


class Q8Matrix:
    """An 8-bit matrix at an offset of larger sentinel-filled buffers: writes outside it show."""

    def __init__(self, rows, cols, pad_cols=16, lead=32, pad_scales=3):
        ld = (cols + 15) // 16 * 16 + pad_cols
        nb = (cols + 127) // 128
        self.rows, self.cols, self.nb = rows, cols, nb
        self.codes_buf = torch.full((lead + max(rows, 1) * ld + 64,), SENTINEL, dtype=torch.uint8, device="cuda")
        self.scales_buf = torch.full((5 + max(rows, 1) * (nb + pad_scales) + 64,), SENTINEL, dtype=torch.uint8, device="cuda")
        self.codes = torch.as_strided(self.codes_buf, (rows, cols), (ld, 1), lead)
        self.scales = torch.as_strided(self.scales_buf, (rows, nb), (nb + pad_scales, 1), 5)

    @property
    def pair(self):
        return self.codes.view(torch.float8_e4m3fn), self.scales.view(torch.float8_e8m0fnu)

    def fill(self, codes, scales):
        self.codes.copy_(torch.from_numpy(codes))
        self.scales.copy_(torch.from_numpy(scales))
        return self

    def numpy(self):
        return self.codes.cpu().numpy(), self.scales.cpu().numpy()

    def assert_untouched_outside(self):
        for buf, view in ((self.codes_buf, self.codes), (self.scales_buf, self.scales)):
            copy = buf.clone()
            torch.as_strided(copy, view.shape, view.stride(), view.storage_offset()).fill_(SENTINEL)
            assert bool((copy == SENTINEL).all()), "bytes outside the matrix were written"


def encoded(rng, rows, cols, sigma=1.0, **kw):
    """A random 8-bit matrix and its values."""
    codes, scales = q8.encode(rng.standard_normal((rows, cols)) * sigma)
    return Q8Matrix(rows, cols, **kw).fill(codes, scales), q8.decode(codes, scales)


class Bf16Matrix:
    """A bf16 matrix at an odd or even element of a sentinel-filled buffer, rows `ld` elements apart."""

    def __init__(self, rows, cols, lead=0, pad=0):
        ld = cols + pad
        self.buf = torch.full((lead + max(rows, 1) * ld + 33,), -3.0, dtype=torch.bfloat16, device="cuda")
        self.t = torch.as_strided(self.buf, (rows, cols), (ld, 1), lead)

    def fill(self, values):
        self.t.copy_(torch.from_numpy(np.asarray(values, np.float32)).to(torch.bfloat16))
        return self.t.float().cpu().numpy().astype(np.float64)

    def assert_untouched_outside(self):
        copy = self.buf.clone()
        torch.as_strided(copy, self.t.shape, self.t.stride(), self.t.storage_offset()).fill_(-3.0)
        assert bool((copy == -3.0).all()), "elements outside the matrix were written"


def to64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check_encoded(got, want, rel):
    """Codes and scales against unrounded 64-bit values computed with relative error up to `rel` of
    `want` (an array of absolute errors, or a number times |want|) before the encoding."""
    codes, scales = got
    err = rel if isinstance(rel, np.ndarray) else rel * np.abs(want)
    tops = q8.block_tops(want)
    slack = q8.block_tops(err)
    lo = np.vectorize(q8.block_exponent, otypes=[np.int64])(np.maximum(tops - slack, 0))
    hi = np.vectorize(q8.block_exponent, otypes=[np.int64])(tops + slack)
    e = scales.astype(np.int64) - 127
    assert np.all((e >= lo) & (e <= hi)), "a block's scale is not the smallest that holds it"
    wide = np.repeat(np.ldexp(1.0, e), q8.BLOCK, axis=1)[:, :want.shape[1]]
    value = q8.VALUES[codes] * wide
    with np.errstate(divide="ignore"):
        step = np.ldexp(wide, (np.maximum(np.floor(np.log2(np.abs(want) / wide + 1e-300)), -6) - 3).astype(np.int64))
    off = np.abs(value - want)
    assert np.all(off <= step * 0.5 + err), "a code is not the nearest: %g" % np.max(off / (step * 0.5 + err))


def check_close(got, want, bound, what):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%s: %d of %d values off, worst %.3g of the bound" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / bound))
