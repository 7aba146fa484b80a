"""Pins of the 64-bit oracle of the 8-bit training operators: the e4m3 table and rounding against torch's
conversion, the scale rule by enumeration, and the gradients against central differences."""

import numpy as np
import pytest
import torch

from oracle import q8


def test_code_table_equals_torch():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(q8.VALUES))
    ok = ~np.isnan(t)
    assert np.array_equal(t[ok], q8.VALUES[ok])


def test_rounding_equals_torch_on_every_bf16_value_in_range():
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(q8.nearest_code(x.double().numpy()), want)


def test_ties_go_to_the_even_mantissa():
    mag = q8.VALUES[:127]
    for k in range(126):
        code = int(q8.nearest_code(np.array([(mag[k] + mag[k + 1]) / 2]))[0])
        assert code == (k if k % 2 == 0 else k + 1)


@pytest.mark.parametrize("top,e", [(0.0, -127), (448.0, 0), (np.nextafter(448.0, 1e9), 1), (224.0, -1), (1.0, -8),
                                   (1.75, -8), (1.76, -7), (3.3895313892515355e38, 120), (1e-40, -127),
                                   (448 * 2.0 ** -127, -127), (449 * 2.0 ** -127, -126)])
def test_block_exponent(top, e):
    assert q8.block_exponent(top) == e
    assert top <= 448 * 2.0 ** e and (e == -127 or top > 448 * 2.0 ** (e - 1))


def test_encode_keeps_non_finite_values_out_of_the_scale():
    x = np.ones((1, 130))
    x[0, 3], x[0, 5], x[0, 129] = np.inf, np.nan, -np.inf
    codes, scales = q8.encode(x)
    assert scales.tolist() == [[127 - 8, 127 - 8]]
    assert (codes[0, [3, 5, 129]] & 0x7f == 0x7f).all()
    assert (q8.decode(codes, scales)[0, 6:128] == 1.0).all()


def test_encoding_again_along_the_other_direction_loses_nothing_but_small_values():
    rng = np.random.default_rng(3)
    v = q8.decode(*q8.encode(rng.standard_normal((200, 300))))
    codes, scales = q8.encode(v.T)
    again = q8.decode(codes, scales).T
    small = np.repeat(q8.scale_values(scales), q8.BLOCK, axis=1)[:, :200].T * 2.0 ** -6
    assert np.array_equal(again[np.abs(v) >= small], v[np.abs(v) >= small])
    assert np.all(np.abs(again - v) <= small * 2.0 ** -4)


def _slope(f, x, at, h):
    a, b = x.copy(), x.copy()
    a[at] += h
    b[at] -= h
    return (f(a) - f(b)) / (2 * h)


def test_norm_gradient_equals_differences():
    rng = np.random.default_rng(1)
    x, w, up = rng.standard_normal((3, 17)), rng.standard_normal(17), rng.standard_normal((3, 17))
    ds = rng.standard_normal((3, 17))
    eps = 1e-5

    def loss(x, w):
        y, s, _ = q8.norm(x, None, w, eps)
        return (y * up).sum() + (s * ds).sum()

    _, s, r = q8.norm(x, None, w, eps)
    dx, dw = q8.norm_backward(up, s, w, r, ds)
    for at in np.ndindex(x.shape):
        assert abs(_slope(lambda v: loss(v, w), x, at, 1e-5) - dx[at]) <= 1e-8 * (1 + abs(dx[at]))
    for at in np.ndindex(w.shape):
        assert abs(_slope(lambda v: loss(x, v), w, at, 1e-5) - dw[at]) <= 1e-8 * (1 + abs(dw[at]))


def test_gate_gradient_equals_differences():
    rng = np.random.default_rng(2)
    g, u, up = (rng.standard_normal((4, 9)) * 2 for _ in range(3))
    dg, du = q8.gate_backward(up, g, u)
    for at in np.ndindex(g.shape):
        assert abs(_slope(lambda v: (q8.gate(v, u) * up).sum(), g, at, 1e-5) - dg[at]) <= 1e-8 * (1 + abs(dg[at]))
        assert abs(_slope(lambda v: (q8.gate(g, v) * up).sum(), u, at, 1e-5) - du[at]) <= 1e-8 * (1 + abs(du[at]))


def test_product_gradients_are_products():
    """The input and weight gradients are products of the same kind: what the transposed operands are for."""
    rng = np.random.default_rng(4)
    x, w, dy = rng.standard_normal((5, 7)), rng.standard_normal((6, 7)), rng.standard_normal((5, 6))
    dx, dw = q8.product(dy, w.T), q8.product(dy.T, x.T)
    assert np.allclose(dx, dy @ w) and np.allclose(dw, dy.T @ x)
    for at in np.ndindex(w.shape):
        assert abs(_slope(lambda v: (q8.product(x, v) * dy).sum(), w, at, 1e-4) - dw[at]) <= 1e-8
