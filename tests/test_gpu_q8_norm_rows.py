"""The norm and its backward pass over many rows per CTA whose addresses fit no wide access: rows read ahead through
shared memory, in place as well."""

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
import q8_torch64 as q64
from q8_helpers import U16, U32, Bf16Matrix, Q8Matrix

pytestmark = pytest.mark.gpu

SIZES = [(9001, 514), (6001, 2047), (3001, 4097), (1501, 7001), (701, 17001)]
LAYOUTS = [dict(lead=1, pad=0), dict(lead=6, pad=3)]


@pytest.fixture(autouse=True)
def _status_stays_clear():
    yield
    torch.cuda.synchronize()
    assert zs.zs_device_status(clear=True) == zs.ZS_DEVERR_NONE


def _matrix(rows, cols, layout, seed, sigma, mean=0.0):
    m = Bf16Matrix(rows, cols, **layout)
    g = torch.Generator(device="cuda").manual_seed(seed)
    m.t.copy_(mean + sigma * torch.randn(rows, cols, generator=g, device="cuda"))
    return m


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_norm(rows, cols, layout):
    x, res = _matrix(rows, cols, layout, 1, 0.3), _matrix(rows, cols, layout, 2, 1.0)
    w = _matrix(1, cols, layout, 3, 0.1, 1.0)
    y, kept, s, rstd = Q8Matrix(rows, cols), Q8Matrix(rows, cols), Bf16Matrix(rows, cols, **layout), torch.empty(rows, device="cuda")
    zs.zs_rmsnorm_q8(x.t, res.t, w.t[0], 1e-5, y.pair, s=s.t, rstd=rstd, s_q8=kept.pair)
    total = x.t.double() + res.t.double()
    r = (total.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    want = total * r * w.t.double()
    # the rows' sums of squares: chains of at most 100 fp32 additions; then a few roundings per value
    rel = 110 * U32
    q64.check_encoded((y.codes, y.scales), want, rel * want.abs())
    q64.check_encoded((kept.codes, kept.scales), total, 2 * U32 * total.abs())
    q64.check_close(s.t, total, (U16 + 2 * U32) * total.abs() + 1e-40)
    q64.check_close(rstd, r[:, 0], rel * r[:, 0])
    for m in (y, kept, s):
        m.assert_untouched_outside()
    again = Q8Matrix(rows, cols)
    zs.zs_rmsnorm_q8(x.t, res.t, w.t[0], 1e-5, again.pair, s=res.t)              # the sum over the residual
    assert torch.equal(again.codes, y.codes) and torch.equal(again.scales, y.scales) and torch.equal(res.t, s.t)
    res.assert_untouched_outside()


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kept8", [False, True])
def test_norm_backward(rows, cols, layout, kept8):
    dy, ds = _matrix(rows, cols, layout, 4, 1e-3), _matrix(rows, cols, layout, 5, 1e-3)
    w, sm = _matrix(1, cols, layout, 6, 0.1, 1.0), _matrix(rows, cols, layout, 7, 1.0)
    s, sv = sm.t, sm.t.double()
    if kept8:
        q = Q8Matrix(rows, cols)
        for to, of in zip((q.codes, q.scales), q64.encode(sv)):
            to.copy_(of)
        s, sv = q.pair, q64.decode(q.codes, q.scales)
    rstd = (sv.square().mean(1) + 1e-5).rsqrt().float()
    r, dyv = rstd.double()[:, None], dy.t.double()
    xh, g = sv * r, dyv * w.t.double()
    want = r * (g - xh * (g * xh).mean(1, keepdim=True)) + ds.t.double()
    bound = U16 * want.abs() + 150 * U32 * (r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) + ds.t.double().abs())
    want_dw, size_dw = (dyv * xh).sum(0), (dyv * xh).abs().sum(0)
    dx, dw = Bf16Matrix(rows, cols, **layout), Bf16Matrix(1, cols, lead=layout["lead"])
    partials = torch.full((304, cols), float("nan"), device="cuda")
    zs.zs_rmsnorm_backward(dy.t, s, w.t[0], rstd, dx.t, dw.t[0], partials, ds=ds.t)
    q64.check_close(dx.t, want, bound)
    # a part's rows one after another, then the parts: fewer than rows additions
    q64.check_close(dw.t[0], want_dw, U16 * want_dw.abs() + (rows + 8) * U32 * size_dw)
    dx.assert_untouched_outside()
    dw.assert_untouched_outside()
    for over in (dy, ds):                                                        # in place
        was, dw2 = over.t.clone(), torch.empty_like(dw.t[0])
        zs.zs_rmsnorm_backward(dy.t, s, w.t[0], rstd, over.t, dw2, partials, ds=ds.t)
        assert torch.equal(over.t, dx.t) and torch.equal(dw2, dw.t[0])
        over.assert_untouched_outside()
        over.t.copy_(was)
