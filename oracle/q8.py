"""The 8-bit training operators in 64-bit floating point: the format, the norm, the gated activation, the
product, and their gradients, straight from their definitions (include/zs.h, "8-bit training operators").

Matrices are numpy arrays of float64; an 8-bit matrix is (codes, scales), two uint8 arrays.  Nothing here
rounds to fewer bits than float64 except the 8-bit encoding itself.
"""

import numpy as np

BLOCK = 128
MAX_CODE = 448.0


def code_values():
    """The 256 e4m3 values: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = -1.0 if c >> 7 else 1.0, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = np.nan
        else:
            out[c] = sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return out


VALUES = code_values()


def nearest_code(x):
    """Codes of finite values with |x| <= 448, to nearest, ties to the even mantissa; NaN -> 0x7f."""
    x = np.asarray(x, np.float64)
    mag = VALUES[:127]                                       # codes 0 .. 126 are the magnitudes, increasing
    a = np.abs(x)
    hi = np.clip(np.searchsorted(mag, a), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    middle = (mag[lo] + mag[hi]) / 2
    up = (a > middle) | ((a == middle) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isnan(x), 0x7f, code).astype(np.uint8)


def block_exponent(top):
    """Smallest integer e >= -127 with top <= 448 * 2^e."""
    e = -127
    if top > 0:
        e = max(-127, int(np.ceil(np.log2(top / MAX_CODE))) - 2)
        while top > MAX_CODE * 2.0 ** e:
            e += 1
    return e


def block_tops(x):
    """Largest finite magnitude of each row's blocks of 128 columns."""
    rows, cols = x.shape
    nb = (cols + BLOCK - 1) // BLOCK
    tops = np.zeros((rows, nb))
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    for b in range(nb):
        part = a[:, b * BLOCK:(b + 1) * BLOCK]
        if part.shape[1]:
            tops[:, b] = part.max(axis=1) if rows else 0.0
    return tops


def encode(x):
    """(codes, scales) of a float64 matrix."""
    x = np.asarray(x, np.float64)
    tops = block_tops(x)
    exps = np.vectorize(block_exponent, otypes=[np.int64])(tops) if tops.size else tops.astype(np.int64)
    wide = np.repeat(exps, BLOCK, axis=1)[:, :x.shape[1]]
    clean = np.where(np.isfinite(x), x, np.nan)
    return nearest_code(np.ldexp(clean, -wide)), (exps + 127).astype(np.uint8)


def scale_values(scales):
    out = np.ldexp(1.0, scales.astype(np.int64) - 127)
    return np.where(scales == 255, np.nan, out)


def decode(codes, scales):
    return VALUES[codes] * np.repeat(scale_values(scales), BLOCK, axis=1)[:, :codes.shape[1]]


# ------------------------------------------------------------------ operators

def norm(x, residual, weight, eps):
    """(y, s, r): the normalised rows, the sums, the reciprocal norms."""
    t = x if residual is None else x + residual
    r = 1.0 / np.sqrt((t * t).mean(axis=1) + eps)
    return t * r[:, None] * weight, t, r


def norm_backward(dy, s, weight, rstd, ds=None):
    """(dx, dw)."""
    xh = s * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    return dx if ds is None else dx + ds, (dy * xh).sum(axis=0)


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def gate(g, u):
    return g * sigmoid(g) * u


def gate_backward(dh, g, u):
    """(dgate, dup)."""
    p = sigmoid(g)
    return dh * u * p * (1.0 + g * (1.0 - p)), dh * g * p


def product(a, b):
    return a @ b.T
