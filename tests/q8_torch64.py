"""The 8-bit format in 64 bits with torch operations, on the GPU for matrices that the numpy oracle takes too long for,
and comparisons of whole matrices with it."""

import torch

from oracle import q8

BLOCK = q8.BLOCK


def _values(like):
    return torch.from_numpy(q8.VALUES).to(like.device)


def _blocks(x):
    rows, cols = x.shape
    pad = -cols % BLOCK
    return torch.nn.functional.pad(x, (0, pad)).view(rows, -1, BLOCK) if pad else x.reshape(rows, -1, BLOCK)


def two_to(e):
    """2^e for integers, exactly (a device's exp2 and pow may be off in the last place)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def steps(t):
    """Distance between the codes' values around t: three bits of mantissa from 2^-6 up."""
    return two_to(torch.frexp(t.abs().clamp(min=2.0 ** -6)).exponent - 4)


def wide(scales, cols):
    """2^e of every value's block, from the scales' bytes."""
    return two_to(scales.long() - 127).repeat_interleave(BLOCK, dim=1)[:, :cols]


def decode(codes, scales):
    return _values(codes)[codes.long()] * wide(scales, codes.shape[1])


def exponents(tops):
    """Smallest integers e >= -127 with tops <= 448 * 2^e."""
    mant, ex = torch.frexp(tops)                                 # tops = mant * 2^ex, 448 = 0.875 * 2^9
    e = torch.where(mant > 0.875, ex - 8, ex - 9).long()
    return torch.where(tops == 0, torch.full_like(e, -127), e).clamp(min=-127)


def encode(x):
    """(codes, scales) as bytes, of finite float64 values."""
    rows, cols = x.shape
    e = exponents(_blocks(x).abs().amax(2))
    scales = (e + 127).to(torch.uint8)
    t = x / wide(scales, cols)
    step = steps(t)
    magnitude = torch.round(t.abs() / step) * step               # ties to even
    code = torch.searchsorted(_values(x)[:127].contiguous(), magnitude).to(torch.uint8)
    return torch.where(torch.signbit(x), code | 0x80, code), scales


def same(got, want):
    """Whether codes and scales are equal, byte for byte."""
    return all(torch.equal(g.view(torch.uint8), w) for g, w in zip(got, want))


def check_encoded(got, want, err):
    """Codes and scales against 64-bit values known to within `err` before the encoding: each scale is the smallest that
    holds its block, each code one of the nearest to some value within err."""
    codes, scales = (x.view(torch.uint8) for x in got)
    tops, slack = _blocks(want).abs().amax(2), _blocks(err).amax(2)
    e = scales.long() - 127
    assert bool(((e >= exponents((tops - slack).clamp(min=0))) & (e <= exponents(tops + slack))).all()), "a block's scale"
    w = wide(scales, want.shape[1])
    step = steps(want / w) * w
    off = (_values(codes)[codes.long()] * w - want).abs()
    worst = (off / (0.5 * step + err)).max().item()
    assert worst <= 1.0, "a code is not the nearest: %g" % worst


def check_close(got, want, bound):
    worst = ((got.double() - want).abs() / bound).max().item()
    assert worst <= 1.0, "worst %.3g of the bound" % worst
