"""AdamW states in 8 bits in 64-bit floating point, from their definition (include/zs.h, "many tensors at once")."""

import math

import numpy as np

from .q8 import VALUES

BLOCK = 256
MAGNITUDES = VALUES[:127]


def mix(x):
    """The finalizer of murmur3's 32-bit hash, on Python integers."""
    m = 0xffffffff
    x = ((x ^ (x >> 16)) * 0x85ebca6b) & m
    x = ((x ^ (x >> 13)) * 0xc2b2ae35) & m
    return x ^ (x >> 16)


def random_bits(seed, tensor, n):
    """The 32 random bits of elements 0 .. n - 1 (n < 2^32) of a tensor."""
    key = mix(mix((seed + 0x9e3779b9 * (tensor + 1)) & 0xffffffff))
    x = np.arange(n, dtype=np.uint64) ^ np.uint64(key)
    m = np.uint64(0xffffffff)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x85ebca6b)) & m
    x = ((x ^ (x >> np.uint64(13))) * np.uint64(0xc2b2ae35)) & m
    return (x ^ (x >> np.uint64(16))).astype(np.int64)


def block_tops(x):
    """Largest finite magnitude of each block, 0 where it is below 2^-100."""
    a = np.zeros(-(-len(x) // BLOCK) * BLOCK)
    a[:len(x)] = np.where(np.isfinite(x), np.abs(x), 0.0)
    top = a.reshape(-1, BLOCK).max(axis=1)
    return np.where(top >= 2.0 ** -100, top, 0.0)


def codes(t, random, positive):
    """Codes of the scaled values |t| <= 448 (a little more is the largest code): up with the distance from the lower
    code against `random` of 2^16."""
    a = np.abs(np.asarray(t, np.float64))
    lower = np.clip(np.searchsorted(MAGNITUDES, a, side="right") - 1, 0, 126)
    upper = np.minimum(lower + 1, 126)
    gap = np.where(upper > lower, MAGNITUDES[upper] - MAGNITUDES[lower], 1.0)
    share = np.where(upper > lower, (a - MAGNITUDES[lower]) / gap, 0.0)
    c = np.where(share + random / 65536.0 >= 1.0, upper, lower)
    if positive:
        c = np.where((a > 0) & (c == 0), 1, c)
    c = np.where(np.isfinite(t), c, 0x7f).astype(np.uint8)
    return c if positive else np.where(np.signbit(t) & np.isfinite(t), c | 0x80, c).astype(np.uint8)


def encode(x, random, positive):
    """(codes, scales) of a state's values."""
    top = block_tops(x)
    wide = np.repeat(top, BLOCK)[:len(x)]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(wide > 0, x * (448.0 / wide), np.where(np.isfinite(x), 0.0, x))
    return codes(t, random, positive), top / 448.0


def decode(code, scales):
    return VALUES[code] * np.repeat(scales, BLOCK)[:len(code)]


def scalars(hp, step):
    """beta1, beta2, eps, decay, c1, c2, step_size, sqrt_bc2 as the fp32 values that the update uses."""
    lr, b1, b2, eps, wd = (float(np.float32(hp[k])) for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
    every = (b1, b2, eps, 1 - lr * wd, 1 - b1, 1 - b2, lr / (1 - b1 ** step), math.sqrt(1 - b2 ** step))
    return tuple(float(np.float32(x)) for x in every)


def adamw(g, p, m, v, hp, step, factor=1.0):
    """(p, m, v) after a step."""
    b1, b2, eps, decay, c1, c2, size, root = scalars(hp, step)
    g = g * factor
    m = b1 * m + c1 * g
    v = b2 * v + c2 * g * g
    return p * decay - size * m / (np.sqrt(v) / root + eps), m, v


def grad_norm(grads, max_norm):
    norm = math.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6))
