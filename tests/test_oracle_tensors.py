"""Pins of the oracle of states in 8 bits: the hash, the rounding's mean, the formula (no GPU)."""

import numpy as np

import synth
from oracle import q8, steps, tensors


def test_random_bits_are_the_hash_of_every_element():
    for seed, t, n in ((0, 0, 300), (12345, 7, 70), (0xffffffff, 400, 33)):
        key = tensors.mix(tensors.mix((seed + 0x9e3779b9 * (t + 1)) % 2 ** 32))
        assert [tensors.mix(i ^ key) for i in range(n)] == tensors.random_bits(seed, t, n).tolist()
    assert tensors.mix(0) == 0 and tensors.mix(1) == 0x514e28b7          # murmur3's finalizer
    h = tensors.random_bits(3, 1, 1 << 16)
    for half in (h & 0xffff, h >> 16):                                  # a uniform 16-bit number: mean 32767.5, deviation 74
        assert abs(half.mean() - 32767.5) < 5 * 74


def test_codes_round_up_as_often_as_the_distance_says():
    every = np.arange(65536)
    for t in (0.3, 1.0, 1.06, 447.0, 2.0 ** -9 * 0.25, 2.0 ** -8 * 1.4, 300.0):
        mean = q8.VALUES[tensors.codes(np.full(65536, t), every, False)].mean()
        assert abs(mean - t) <= t * 2.0 ** -16 + 2.0 ** -25
        assert np.array_equal(tensors.codes(np.full(65536, -t), every, False), tensors.codes(np.full(65536, t), every, False) | 0x80)
    assert tensors.codes(np.array([448.0, 448.0001, 0.0]), np.array([65535] * 3), False).tolist() == [126, 126, 0]


def test_a_positive_root_keeps_a_code():
    assert tensors.codes(np.array([1e-9, 0.0, 1.0]), np.zeros(3), True).tolist() == [1, 0, 0x38]
    assert tensors.codes(np.array([1e-9]), np.zeros(1), False).tolist() == [0]


def test_encode_and_decode():
    rng = np.random.default_rng(0)
    x = rng.standard_normal(700) * np.exp(rng.uniform(-3, 3, 700))
    x[600:] = 0.0
    code, scale = tensors.encode(x, rng.integers(0, 65536, 700), False)
    assert scale.shape == (3,)
    back = tensors.decode(code, scale)
    wide = np.repeat(scale, 256)[:700]
    assert np.all(np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -3, wide * 2.0 ** -9))
    code, scale = tensors.encode(np.array([np.nan, np.inf, 1.0, -2.0]), np.zeros(4), False)
    assert code[:2].tolist() == [0x7f, 0x7f] and scale.tolist() == [2.0 / 448] and code[3] == 0xfe
    code, scale = tensors.encode(np.array([2.0 ** -101, -1e-40]), np.zeros(2), False)
    assert scale.tolist() == [0.0] and (code & 0x7f).tolist() == [0, 0]


def test_step_is_the_flat_step():
    rng = np.random.default_rng(4)
    n, hp = 500, synth.HPARAMS
    p, m, v = rng.standard_normal(n).astype(np.float32), np.zeros(n, np.float32), np.zeros(n, np.float32)
    bits = ((rng.standard_normal(n) * 1e-3).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    g = (bits.astype(np.uint32) << 16).view(np.float32)
    want = steps.adamw(p, m, v, bits, hp, 3)
    got = tensors.adamw(g.astype(np.float64), p.astype(np.float64), m.astype(np.float64), v.astype(np.float64), hp, 3)
    for a, b in zip(got, want[:3]):
        assert np.allclose(a, b.astype(np.float64), rtol=1e-6, atol=1e-12)
    assert [float(x) for x in steps.adamw_scalars(hp, 3).values()] == list(tensors.scalars(hp, 3))
