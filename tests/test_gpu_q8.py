"""The 8-bit training operators against the 64-bit oracle: encoding both ways, norm, gated activation and
product, forward and backward, at the sizes, strides and values where they can go wrong."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
from oracle import q8
from q8_helpers import U16, U32, Bf16Matrix, Q8Matrix, check_close, check_encoded, encoded, to64

pytestmark = pytest.mark.gpu

SIZES = [(1, 1), (1, 128), (3, 129), (17, 16), (127, 255), (128, 128), (130, 384), (257, 77), (300, 520)]
LAYOUTS = [dict(lead=0, pad=0), dict(lead=8, pad=8), dict(lead=1, pad=0), dict(lead=3, pad=5)]


@pytest.fixture(autouse=True)
def _status_stays_clear():
    yield
    torch.cuda.synchronize()
    assert zs.zs_device_status(clear=True) == zs.ZS_DEVERR_NONE


# ------------------------------------------------------------------ encode, decode, transpose

@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_encode_both_ways_is_exact(rows, cols, layout):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = Bf16Matrix(rows, cols, **layout)
    v = x.fill(rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-20, 20, (rows, 1))))
    q, qt = Q8Matrix(rows, cols), Q8Matrix(cols, rows)
    zs.zs_q8_encode(x.t, q.pair, qt.pair)
    for got, want in ((q, q8.encode(v)), (qt, q8.encode(v.T))):
        codes, scales = got.numpy()
        assert np.array_equal(scales, want[1])
        assert np.array_equal(codes, want[0])
        got.assert_untouched_outside()
    one, other = Q8Matrix(rows, cols), Q8Matrix(cols, rows)       # each direction by itself
    zs.zs_q8_encode(x.t, one.pair)
    zs.zs_q8_encode(x.t, None, other.pair)
    assert torch.equal(one.codes, q.codes) and torch.equal(other.codes, qt.codes)
    assert torch.equal(one.scales, q.scales) and torch.equal(other.scales, qt.scales)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("layout", [LAYOUTS[0], LAYOUTS[3]])
def test_decode_and_transpose_are_exact(rows, cols, layout):
    rng = np.random.default_rng(rows * 1000 + cols + 7)
    q, v = encoded(rng, rows, cols)
    y = Bf16Matrix(rows, cols, **layout)
    zs.zs_q8_decode(q.pair, y.t)
    assert np.array_equal(to64(y.t), v)
    y.assert_untouched_outside()
    qt = Q8Matrix(cols, rows)
    zs.zs_q8_transpose(q.pair, qt.pair)
    want = q8.encode(v.T)
    assert np.array_equal(qt.numpy()[0], want[0]) and np.array_equal(qt.numpy()[1], want[1])
    qt.assert_untouched_outside()


@pytest.mark.parametrize("spread", [0, 3, 15, 16, 40, 120])
@pytest.mark.parametrize("rows,cols", [(128, 64), (300, 200), (77, 130)])
def test_transpose_of_rows_with_far_scales(spread, rows, cols):
    """Scales of neighbouring rows up to 2^120 apart, columns of every size, rows and columns of zeros, NaN codes
    and NaN scales: the transpose is exact whichever way a tile takes."""
    rng = np.random.default_rng(spread * 100 + rows)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-spread, spread + 1, (rows, 1)))
    x *= np.exp2(rng.integers(-spread // 2, 1, (1, cols)))
    x[rng.integers(0, rows, 5)] = 0.0
    x[:, rng.integers(0, cols, 5)] = 0.0
    x[rows // 2:rows // 2 + 20, :] *= np.exp2(-spread)                  # warps of rows far below the others
    codes, scales = q8.encode(x)
    codes[rows // 3, cols // 2] = 0x7f
    codes[0, :3] = 0x80                                                # negative zeros
    if spread == 40:
        scales[rows // 4, 0] = 255
    q = Q8Matrix(rows, cols).fill(codes, scales)
    qt = Q8Matrix(cols, rows)
    zs.zs_q8_transpose(q.pair, qt.pair)
    want = q8.encode(q8.decode(codes, scales).T)
    got = qt.numpy()
    assert np.array_equal(got[1], want[1])
    a, b = q8.VALUES[got[0]], q8.VALUES[want[0]]
    assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)])
    qt.assert_untouched_outside()


def test_transpose_near_the_ends_of_the_scales():
    """Scale bytes 0 to 254: values down to 2^-136 and up to 448 * 2^119 (beyond, fp32 would overflow)."""
    for low, high in ((0, 12), (0, 40), (100, 140), (230, 246), (236, 247)):
        rng = np.random.default_rng(low + high)
        codes = rng.integers(0, 127, (130, 70)).astype(np.uint8) | (rng.integers(0, 2, (130, 70)) << 7).astype(np.uint8)
        scales = rng.integers(low, high, (130, 1)).astype(np.uint8)
        q, qt = Q8Matrix(130, 70).fill(codes, scales), Q8Matrix(70, 130)
        zs.zs_q8_transpose(q.pair, qt.pair)
        want = q8.encode(q8.decode(codes, scales).T)
        assert np.array_equal(qt.numpy()[1], want[1])
        assert np.array_equal(q8.VALUES[qt.numpy()[0]], q8.VALUES[want[0]])


def test_encode_values_at_the_edges():
    """Zeros, the smallest and largest bf16 values, ties, infinities and NaN, each in a block of its own."""
    rows = np.zeros((10, 256))
    rows[1, :] = 2.0 ** -133                       # bf16's smallest subnormal
    rows[2, :] = 3.3895313892515355e38             # its largest value
    rows[3, 0], rows[3, 1:] = 448.0, 1.0625        # a tie between 1 and 1.125
    rows[4, 0], rows[4, 1:] = 450.0, 17.0
    rows[5, 5] = np.inf
    rows[6, 7], rows[6, 9] = np.nan, 1.0
    rows[7, :128] = -np.inf                        # a block with nothing finite
    rows[8, :] = -(2.0 ** -120)
    rows[9, 0], rows[9, 1:] = 1e30, 1e-30
    x = Bf16Matrix(10, 256)
    v = x.fill(rows)
    q, qt = Q8Matrix(10, 256), Q8Matrix(256, 10)
    zs.zs_q8_encode(x.t, q.pair, qt.pair)
    for got, want in ((q, q8.encode(v)), (qt, q8.encode(v.T))):
        assert np.array_equal(got.numpy()[1], want[1])
        a, b = q8.VALUES[got.numpy()[0]], q8.VALUES[want[0]]
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)])


def test_decode_reads_every_code_and_scale_byte():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 2, axis=1)
    q = Q8Matrix(256, 256).fill(codes, scales)
    y = torch.empty(256, 256, dtype=torch.bfloat16, device="cuda")
    zs.zs_q8_decode(q.pair, y)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(q8.decode(codes, scales).astype(np.float32)).to(torch.bfloat16).float().numpy()
    got = y.float().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_rows_past_four_gigabytes():
    """Rows 2^31 bytes apart: the last row's codes start past 2^32."""
    ld = 1 << 31
    buf = torch.zeros(2 * ld + 4096, dtype=torch.uint8, device="cuda")
    codes = torch.as_strided(buf, (3, 300), (ld, 1))
    scales = torch.zeros(3, 3, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((3, 300)).astype(np.float32)).to(torch.bfloat16).cuda()
    zs.zs_q8_encode(x, (codes, scales))
    want = q8.encode(to64(x))
    assert np.array_equal(codes.cpu().numpy(), want[0])
    y = torch.empty_like(x)
    zs.zs_q8_decode((codes, scales), y)
    assert np.array_equal(to64(y), q8.decode(*want))
    b, bv = encoded(rng, 5, 300)
    out = torch.empty(3, 5, dtype=torch.bfloat16, device="cuda")
    zs.zs_q8_matmul((codes, scales), b.pair, out)
    v = q8.decode(*want)
    check_close(to64(out), v @ bv.T, U16 * np.abs(v @ bv.T) + 64 * U32 * (np.abs(v) @ np.abs(bv.T)), "product")


# ------------------------------------------------------------------ norm

# the row statistics' fp32 sums are chains of at most 64 terms, then a few roundings per value
NORM_REL = 80 * U32


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (5, 100), (3, 129), (7, 1000), (4, 4096), (2, 9000),
                                       (3, 20011), (2, 40000)])
@pytest.mark.parametrize("layout", [LAYOUTS[0], LAYOUTS[3]])
@pytest.mark.parametrize("full", [True, False])
def test_norm(rows, cols, layout, full):
    rng = np.random.default_rng(rows + cols)
    x, res, w = Bf16Matrix(rows, cols, **layout), Bf16Matrix(rows, cols, **layout), Bf16Matrix(1, cols, lead=layout["lead"])
    xv, rv, wv = (m.fill(rng.standard_normal((m.t.shape[0], cols)) * s) for m, s in ((x, 0.3), (res, 1.0), (w, 1.0)))
    y, sq = Q8Matrix(rows, cols), Q8Matrix(rows, cols)
    s, rstd = Bf16Matrix(rows, cols, **layout), torch.full((rows,), -1.0, device="cuda")
    if full:
        zs.zs_rmsnorm_q8(x.t, res.t, w.t[0], 1e-5, y.pair, s=s.t, rstd=rstd, s_q8=sq.pair)
    else:
        zs.zs_rmsnorm_q8(x.t, None, w.t[0], 1e-5, y.pair)
    yv, t, r = q8.norm(xv, rv if full else None, wv[0], 1e-5)
    check_encoded(y.numpy(), yv, NORM_REL)
    y.assert_untouched_outside()
    if full:
        check_encoded(sq.numpy(), t, U32 * 2)
        check_close(to64(s.t), t, (U16 + 2 * U32) * np.abs(t), "s")
        check_close(rstd.cpu().numpy(), r, NORM_REL * r, "rstd")
        sq.assert_untouched_outside()
        s.assert_untouched_outside()


def test_norm_in_place_and_rows_of_zeros_and_non_finite_rows():
    x = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")
    res = torch.zeros_like(x)
    x[1], res[1], x[2, 3], x[3, 4] = 1.5, 0.5, float("inf"), float("nan")
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    y, rstd = zs.q8_empty(4, 512), torch.empty(4, device="cuda")
    zs.zs_rmsnorm_q8(x, res, w, 0.25, y, s=res, rstd=rstd)
    v = y[0].float() * y[1].float().repeat_interleave(128, 1)
    assert bool((v[0] == 0).all()) and rstd[0].item() == 2.0          # 1 / sqrt(0 + 0.25)
    assert bool((res[1] == 2.0).all()) and bool((v[1] == v[1, 0]).all())
    assert abs(v[1, 0].item() - 2.0 / 4.25 ** 0.5) <= 0.07
    assert bool(torch.isnan(v[3]).all()) and bool(torch.isnan(v[2, 3]))
    # a row of zeros with eps = 0: 0 * infinity
    zs.zs_rmsnorm_q8(torch.zeros_like(x), None, w, 0.0, y)
    assert bool(torch.isnan(y[0].float()).all())


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (5, 100), (33, 129), (700, 1000), (40, 4096), (9, 9000),
                                       (3, 20011), (5, 40000)])
@pytest.mark.parametrize("layout", [LAYOUTS[0], LAYOUTS[3]])
@pytest.mark.parametrize("kept", ["bf16", "q8"])
def test_norm_backward(rows, cols, layout, kept):
    rng = np.random.default_rng(rows + cols + 1)
    dy, ds, w = Bf16Matrix(rows, cols, **layout), Bf16Matrix(rows, cols, **layout), Bf16Matrix(1, cols, lead=layout["lead"])
    dyv, dsv = (m.fill(rng.standard_normal((rows, cols)) * 1e-3) for m in (dy, ds))
    wv = w.fill(1 + 0.1 * rng.standard_normal((1, cols)))[0]
    if kept == "q8":
        sm, sv = encoded(rng, rows, cols)
        s = sm.pair
    else:
        sm = Bf16Matrix(rows, cols, **layout)
        sv = sm.fill(rng.standard_normal((rows, cols)))
        s = sm.t
    rstd = torch.from_numpy((1 / np.sqrt((sv ** 2).mean(1) + 1e-5)).astype(np.float32)).cuda()
    r = rstd.cpu().numpy().astype(np.float64)
    dx, dw = Bf16Matrix(rows, cols, **layout), Bf16Matrix(1, cols, lead=layout["lead"])
    dw0 = dw.fill(rng.standard_normal((1, cols)))[0]
    parts = torch.full((min(rows, 37), cols), float("nan"), device="cuda")
    want_dx, want_dw = q8.norm_backward(dyv, sv, wv, r, dsv)
    xh = np.abs(sv * r[:, None])
    g = np.abs(dyv * wv)
    mean = (g * xh).mean(axis=1, keepdims=True)
    dx_bound = U16 * np.abs(want_dx) + 100 * U32 * (r[:, None] * (g + xh * mean) + np.abs(dsv))
    dw_sum = (np.abs(dyv) * xh).sum(axis=0)
    zs.zs_rmsnorm_backward(dy.t, s, w.t[0], rstd, dx.t, dw.t[0], parts, ds=ds.t, scale=0.25, first=False)
    check_close(to64(dx.t), want_dx, dx_bound, "dx")
    check_close(to64(dw.t)[0], dw0 + 0.25 * want_dw, U16 * np.abs(dw0 + 0.25 * want_dw) + (rows + 8) * U32 * dw_sum
                + U32 * np.abs(dw0) * 4, "dw added")
    dx.assert_untouched_outside()
    dw.assert_untouched_outside()
    # first: dw is only written; without ds; other numbers of partials; in place over dy
    dw.t.fill_(float("nan"))
    many = torch.full((700, cols), float("nan"), device="cuda")
    zs.zs_rmsnorm_backward(dy.t, s, w.t[0], rstd, dy.t, dw.t[0], many)
    check_close(to64(dw.t)[0], want_dw, U16 * np.abs(want_dw) + (rows + 8) * U32 * dw_sum, "dw")
    check_close(to64(dy.t), want_dx - dsv, U16 * np.abs(want_dx - dsv) + dx_bound - U16 * np.abs(want_dx), "dx in place")


@pytest.mark.parametrize("rows,cols", [(650, 4096), (999, 6160), (6001, 4080)])
@pytest.mark.parametrize("layout", [LAYOUTS[0], dict(lead=16, pad=16)])
@pytest.mark.parametrize("kept", ["bf16", "q8"])
def test_norm_backward_of_many_rows_per_part(rows, cols, layout, kept):
    test_norm_backward(rows, cols, layout, kept)


@pytest.mark.parametrize("rows,cols", [(305, 4096), (2000, 4090), (400, 8192), (1300, 528)])
@pytest.mark.parametrize("layout", [LAYOUTS[0], LAYOUTS[3]])
def test_norm_of_more_rows_than_are_resident(rows, cols, layout):
    test_norm(rows, cols, layout, True)


def test_norm_backward_without_rows_writes_the_empty_sum():
    cols = 100
    z = torch.empty(0, cols, dtype=torch.bfloat16, device="cuda")
    w, dw = (torch.full((cols,), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    parts = torch.full((4, cols), float("nan"), device="cuda")
    zs.zs_rmsnorm_backward(z, z, w, torch.empty(0, device="cuda"), z, dw, parts, first=False)
    assert bool((dw == 3).all())
    zs.zs_rmsnorm_backward(z, z, w, torch.empty(0, device="cuda"), z, dw, parts)
    assert bool((dw == 0).all())


# ------------------------------------------------------------------ gated activation

# the fast exponential and quotient are within 2^-18 for |gate| <= 20 here, the rest a few roundings
GATE_REL = 2.0 ** -17


@pytest.mark.parametrize("rows,cols", SIZES + [(2, 1500), (1, 11008)])
@pytest.mark.parametrize("layout", [LAYOUTS[0], LAYOUTS[3]])
def test_gate(rows, cols, layout):
    rng = np.random.default_rng(rows + cols + 2)
    both = Bf16Matrix(rows, 2 * cols, **layout)
    v = both.fill(rng.standard_normal((rows, 2 * cols)) * 4)
    g, u = both.t[:, :cols], both.t[:, cols:]
    h, gq, uq = (Q8Matrix(rows, cols) for _ in range(3))
    zs.zs_swiglu_q8(g, u, h.pair, gq.pair, uq.pair)
    check_encoded(h.numpy(), q8.gate(v[:, :cols], v[:, cols:]), GATE_REL)
    for m, x in ((gq, v[:, :cols]), (uq, v[:, cols:])):
        want = q8.encode(x)
        assert np.array_equal(m.numpy()[0], want[0]) and np.array_equal(m.numpy()[1], want[1])
        m.assert_untouched_outside()
    h.assert_untouched_outside()
    only = Q8Matrix(rows, cols)
    zs.zs_swiglu_q8(g, u, only.pair)
    assert torch.equal(only.codes, h.codes)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("layout", [LAYOUTS[0], LAYOUTS[3]])
def test_gate_backward(rows, cols, layout):
    rng = np.random.default_rng(rows + cols + 3)
    gq, g = encoded(rng, rows, cols, 4.0)
    uq, u = encoded(rng, rows, cols, 2.0)
    dh = Bf16Matrix(rows, cols, **layout)
    d = dh.fill(rng.standard_normal((rows, cols)) * 1e-3)
    outs = [Q8Matrix(rows, cols), Q8Matrix(rows, cols), Q8Matrix(cols, rows), Q8Matrix(cols, rows), Q8Matrix(cols, rows)]
    zs.zs_swiglu_backward_q8(dh.t, gq.pair, uq.pair, *(o.pair for o in outs))
    dg, du = q8.gate_backward(d, g, u)
    # 1 + gate * (1 - p) cancels for negative gates: its roundings are relative to 1 + |gate| * (1 - p)
    p = q8.sigmoid(g)
    dg_err = GATE_REL * np.abs(d * u * p) * (1 + np.abs(g) * (1 - p))
    h, h_err = q8.gate(g, u), GATE_REL * np.abs(q8.gate(g, u))
    for o, want, err in zip(outs, (dg, du, dg.T, du.T, h.T), (dg_err, GATE_REL * np.abs(du), dg_err.T,
                                                             GATE_REL * np.abs(du.T), h_err.T)):
        check_encoded(o.numpy(), want, np.ascontiguousarray(err))
        o.assert_untouched_outside()
    for k in range(5):                                             # each output by itself
        alone = Q8Matrix(outs[k].rows, outs[k].cols)
        zs.zs_swiglu_backward_q8(dh.t, gq.pair, uq.pair, *(alone.pair if i == k else None for i in range(5)))
        assert torch.equal(alone.codes, outs[k].codes) and torch.equal(alone.scales, outs[k].scales)


def test_gate_far_values():
    """Gates whose exponential leaves fp32's range: sigmoid is 0 or 1, and nothing turns into NaN."""
    g = torch.tensor([[-3e38, -200.0, -100.0, -88.0, 0.0, 88.0, 200.0, 3e38]], device="cuda").to(torch.bfloat16)
    u = torch.ones_like(g)
    h, gq, uq = zs.q8_empty(1, 8), zs.q8_empty(1, 8), zs.q8_empty(1, 8)
    zs.zs_swiglu_q8(g, u, h, gq, uq)
    v = (h[0].float() * h[1].float())[0]
    assert bool(torch.isfinite(v).all()) and bool((v[:5] == 0).all()) and v[7].item() > 2e38
    small = torch.tensor([[-200.0, -100.0, 0.0, 100.0, 200.0]], device="cuda").to(torch.bfloat16)
    one = torch.ones_like(small)
    gq, uq = zs.q8_empty(1, 5), zs.q8_empty(1, 5)
    zs.zs_swiglu_q8(small, one, zs.q8_empty(1, 5), gq, uq)
    dg, du = zs.q8_empty(1, 5), zs.q8_empty(1, 5)
    zs.zs_swiglu_backward_q8(one, gq, uq, dg, du)
    a, b = ((m[0].float() * m[1].float())[0].tolist() for m in (dg, du))
    assert a[0] == 0 and a[2] == 0.5 and a[4] == 1 and b[0] == 0 and b[2] == 0 and abs(b[4] - 200) <= 8


# ------------------------------------------------------------------ product

def _product_bound(av, bv, want, k):
    # one rounding to bf16; the sum: products exact, one addition per 32 columns kept to 2^-23 or better,
    # and the additions inside them
    return U16 * np.abs(want) + (k / 8 + 16) * 2 * U32 * (np.abs(av) @ np.abs(bv).T)


PRODUCTS = [(1, 1, 1), (1, 8, 16), (2, 300, 100), (16, 64, 128), (33, 129, 129), (64, 200, 640), (65, 130, 513),
            (100, 40, 1000), (128, 128, 128), (128, 256, 2048), (129, 257, 385), (200, 1000, 3000), (300, 24, 4100),
            (513, 520, 200), (1, 1000, 5000), (5, 2000, 1111), (700, 900, 1)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k):
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    a, av = encoded(rng, m, k)
    b, bv = encoded(rng, n, k, 0.02)
    want = av @ bv.T
    for layout in (LAYOUTS[0], LAYOUTS[3]):
        out = Bf16Matrix(m, n, **layout)
        out.t.fill_(float("nan"))
        zs.zs_q8_matmul(a.pair, b.pair, out.t)
        check_close(to64(out.t), want, _product_bound(av, bv, want, k), "out")
        out.assert_untouched_outside()
        before = out.fill(rng.standard_normal((m, n)) * np.abs(want).max())
        zs.zs_q8_matmul(a.pair, b.pair, out.t, scale=-0.25, first=False)
        both = before - 0.25 * want
        check_close(to64(out.t), both, _product_bound(av, bv, want, k) + U16 * np.abs(both) + 2 * U32 * np.abs(before),
                    "out added")
        out.assert_untouched_outside()


def test_product_scales_differ_between_blocks():
    """Every block with its own scale on both sides: a scale taken from a neighbouring row or block shows."""
    rng = np.random.default_rng(11)
    m, n, k = 150, 280, 1700
    nb = (k + 127) // 128

    def operand(rows):
        codes = q8.nearest_code(rng.choice([-1.0, 1.0, 2.0, -3.0], (rows, k)))
        scales = rng.integers(117, 138, (rows, nb)).astype(np.uint8)
        return Q8Matrix(rows, k).fill(codes, scales), q8.decode(codes, scales)

    a, av = operand(m)
    b, bv = operand(n)
    want = av @ bv.T
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    zs.zs_q8_matmul(a.pair, b.pair, out)
    check_close(to64(out), want, _product_bound(av, bv, want, k), "out")
    few = torch.empty(9, n, dtype=torch.bfloat16, device="cuda")
    zs.zs_q8_matmul((a.pair[0][:9], a.pair[1][:9]), b.pair, few)
    check_close(to64(few), want[:9], _product_bound(av[:9], bv, want[:9], k), "few rows")


@pytest.mark.parametrize("m,n,k", [(200, 7, 5000), (70, 16, 11000), (513, 33, 3000), (9000, 20, 700), (6400, 50, 130)])
def test_product_of_few_rows_of_b(m, n, k):
    test_product(m, n, k)


@pytest.mark.parametrize("m,n,k", [(2600, 1500, 1100), (2561, 1537, 77), (5000, 700, 1300), (3001, 2045, 500), (2600, 1500, 1024)])
def test_product_of_large_tiles(m, n, k):
    # odd counts of 256-row tiles, the last one nearly empty; rows of codes that cross 128-byte lines and not
    test_product(m, n, k)


@pytest.mark.parametrize("k", [100, 300, 640, 1100])
def test_product_of_many_tiles_with_scales_of_their_own(k):
    # tiles of one group of scales and of a few, every block with its own: each tile's products read their own scales
    rng = np.random.default_rng(k)
    m, n, nb = 3500, 2900, -(-k // 128)

    def operand(rows):
        codes = rng.integers(0, 0x50, (rows, k)).astype(np.uint8)
        scales = rng.integers(117, 138, (rows, nb)).astype(np.uint8)
        return Q8Matrix(rows, k).fill(codes, scales), q8.decode(codes, scales)

    a, av = operand(m)
    b, bv = operand(n)
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        zs.zs_q8_matmul(a.pair, b.pair, out)
    want = av @ bv.T
    check_close(to64(out), want, _product_bound(av, bv, want, k), "out")


def test_product_reads_nothing_outside_its_matrices():
    """NaN codes and NaN scales around the operands do not reach the result."""
    rng = np.random.default_rng(12)
    for m, n, k in ((5, 70, 200), (130, 140, 333)):
        a, av = encoded(rng, m, k)
        b, bv = encoded(rng, n, k)
        for q in (a, b):
            codes, scales = q.numpy()
            q.codes_buf.fill_(0x7f)
            q.scales_buf.fill_(0xff)
            q.fill(codes, scales)
        out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        zs.zs_q8_matmul(a.pair, b.pair, out)
        check_close(to64(out), av @ bv.T, _product_bound(av, bv, av @ bv.T, k), "out")


def test_product_nan_and_far_scales():
    a, b = (Q8Matrix(4, 256).fill(np.full((4, 256), 0x38, np.uint8), np.full((4, 2), 127, np.uint8)) for _ in range(2))
    a.codes[1, 200] = 0x7f                       # a NaN code
    a.scales[2, 0] = 0xff                        # a NaN scale
    a.scales[3, :] = 0                           # 2^-127
    out = torch.empty(4, 4, dtype=torch.bfloat16, device="cuda")
    zs.zs_q8_matmul(a.pair, b.pair, out)
    v = out.float()
    assert bool((v[0] == 256).all()) and bool(torch.isnan(v[1:3]).all())
    b.scales.fill_(254)                          # 2^127: together 1
    zs.zs_q8_matmul(a.pair, b.pair, out)
    assert bool((out[3].float() == 256).all())


def test_product_of_nothing():
    a, b = zs.q8_empty(3, 0), zs.q8_empty(4, 0)
    out = torch.full((3, 4), 5.0, dtype=torch.bfloat16, device="cuda")
    zs.zs_q8_matmul(a, b, out, first=False)
    assert bool((out == 5).all())
    zs.zs_q8_matmul(a, b, out)
    assert bool((out == 0).all())
    zs.zs_q8_matmul(zs.q8_empty(0, 9), zs.q8_empty(4, 9), out[:0])


# ------------------------------------------------------------------ streams, graphs, repeats

def _unit(m, c, f):
    """One MLP unit forward and backward; every buffer it writes."""
    g = torch.Generator(device="cuda").manual_seed(m + c + f)
    rand = lambda r, k, s: (torch.randn(r, k, generator=g, device="cuda") * s).to(torch.bfloat16)  # noqa: E731
    x, res, w = rand(m, c, 0.3), rand(m, c, 1.0), rand(1, c, 1.0)[0]
    w_in, w_out = rand(2 * f, c, 0.02), rand(c, f, 0.02)
    q = lambda r, k: zs.q8_empty(r, k)  # noqa: E731
    t = {"wi": q(2 * f, c), "wi_t": q(c, 2 * f), "wo": q(c, f), "wo_t": q(f, c), "y": q(m, c), "sq": q(m, c), "y_t": q(c, m),
         "gate": q(m, f), "up": q(m, f), "h": q(m, f), "dy": q(m, c), "dy_t": q(c, m), "d": q(m, 2 * f), "d_t": q(2 * f, m),
         "h_t": q(f, m)}
    b = lambda r, k: torch.empty(r, k, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o = {"s": b(m, c), "rstd": torch.empty(m, device="cuda"), "gu": b(m, 2 * f), "out": b(m, c), "dh": b(m, f), "dn": b(m, c),
         "dx": b(m, c), "dwi": b(2 * f, c), "dwo": b(c, f), "dw": b(1, c), "parts": torch.empty(64, c, device="cuda")}
    dout = rand(m, c, 1e-3)

    def step():
        zs.zs_q8_encode(w_in, t["wi"], t["wi_t"])
        zs.zs_q8_encode(w_out, t["wo"], t["wo_t"])
        zs.zs_rmsnorm_q8(x, res, w, 1e-5, t["y"], s=o["s"], rstd=o["rstd"], s_q8=t["sq"])
        zs.zs_q8_matmul(t["y"], t["wi"], o["gu"])
        zs.zs_swiglu_q8(o["gu"][:, :f], o["gu"][:, f:], t["h"], t["gate"], t["up"])
        zs.zs_q8_matmul(t["h"], t["wo"], o["out"])
        zs.zs_q8_encode(dout, t["dy"], t["dy_t"])
        zs.zs_q8_matmul(t["dy"], t["wo_t"], o["dh"])
        nb = f // 128
        zs.zs_swiglu_backward_q8(o["dh"], t["gate"], t["up"], (t["d"][0][:, :f], t["d"][1][:, :nb]),
                                 (t["d"][0][:, f:], t["d"][1][:, nb:]), (t["d_t"][0][:f], t["d_t"][1][:f]),
                                 (t["d_t"][0][f:], t["d_t"][1][f:]), t["h_t"])
        zs.zs_q8_matmul(t["dy_t"], t["h_t"], o["dwo"])
        zs.zs_q8_matmul(t["d"], t["wi_t"], o["dn"])
        zs.zs_q8_transpose(t["y"], t["y_t"])
        zs.zs_q8_matmul(t["d_t"], t["y_t"], o["dwi"])
        zs.zs_rmsnorm_backward(o["dn"], t["sq"], w, o["rstd"], o["dx"], o["dw"][0], o["parts"], ds=dout)

    bufs = [v for k, v in o.items() if k != "parts"] + [x.view(torch.uint8) for p in t.values() for x in p]
    return step, bufs


def _snapshot(bufs):
    torch.cuda.synchronize()
    return [b.clone() for b in bufs]


def test_repeats_streams_and_graphs_give_the_same_bits():
    step, bufs = _unit(270, 384, 256)
    step()
    want = _snapshot(bufs)
    side = torch.cuda.Stream()
    for how in ("again", "stream", "graph"):
        for b in bufs:
            b.zero_()
        torch.cuda.synchronize()
        if how == "again":
            step()
        elif how == "stream":
            with torch.cuda.stream(side):
                step()
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for b in bufs:
                b.zero_()
            graph.replay()
        got = _snapshot(bufs)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want)), how


def test_unit_gradients_follow_the_formulas():
    """The whole unit's gradients against the same unit in 64 bits without any 8-bit rounding: the
    direction of each gradient is right (cosine) and its length too."""
    m, c, f = 256, 384, 256
    step, bufs = _unit(m, c, f)
    step()
    torch.cuda.synchronize()
    g = torch.Generator(device="cuda").manual_seed(m + c + f)
    rand = lambda r, k, s: (torch.randn(r, k, generator=g, device="cuda") * s).to(torch.bfloat16)  # noqa: E731
    x, res, w = rand(m, c, 0.3), rand(m, c, 1.0), rand(1, c, 1.0)[0]
    w_in, w_out = rand(2 * f, c, 0.02), rand(c, f, 0.02)
    dout = rand(m, c, 1e-3)
    xv, rv, wv, wi, wo, dv = (v.double().cpu().numpy() for v in (x, res, w, w_in, w_out, dout))
    y, t, r = q8.norm(xv, rv, wv, 1e-5)
    gu = y @ wi.T
    gate, up = gu[:, :f], gu[:, f:]
    dh = dv @ wo
    dg, du = q8.gate_backward(dh, gate, up)
    d = np.concatenate([dg, du], axis=1)
    dx, dw = q8.norm_backward(d @ wi, t, wv, r, dv)
    got = {"dx": bufs[6], "dwi": bufs[7], "dwo": bufs[8], "dw": bufs[9][0]}
    # an e4m3 rounding is 2^-4 at most, about 2.6 % in the mean square; a gradient here passes through
    # fewer than ten of them, independent of each other: below 10 % of its length
    for name, want in (("dx", dx), ("dwi", d.T @ y), ("dwo", dv.T @ q8.gate(gate, up)), ("dw", dw)):
        have = to64(got[name])
        assert np.linalg.norm(have - want) <= 0.1 * np.linalg.norm(want), name
