"""The 8-bit kernels' waits run out: the call reports it, leaves nothing under way, and the next call is right."""

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _limits_and_status_as_they_were():
    zs.zs_device_status(clear=True)
    yield
    zs.zs_set_q8_wait_limit()
    torch.cuda.synchronize()
    assert zs.zs_device_status(clear=True) == zs.ZS_DEVERR_NONE


def _filled(rows, cols, seed, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * sigma).to(torch.bfloat16)
    q = zs.q8_empty(rows, cols)
    zs.zs_q8_encode(x, q)
    return x, q


def _bits(outs):
    torch.cuda.synchronize()
    return [x.contiguous().view(torch.uint8).clone() for x in outs]


def _runs_out(call, outs, code, surely=True):
    """call() as ever, then with waits that look once, then with very short ones, and as ever again."""
    call()
    want = _bits(outs)
    assert zs.zs_device_status() == zs.ZS_DEVERR_NONE
    for _ in range(10):
        zs.zs_set_q8_wait_limit(0)
        call()
        torch.cuda.synchronize()
        assert zs.zs_device_status(clear=True) in ((code,) if surely else (zs.ZS_DEVERR_NONE, code))
        zs.zs_set_q8_wait_limit()
        call()                                   # over what the call before left, if anything
        assert all(torch.equal(a, b) for a, b in zip(_bits(outs), want))
        assert zs.zs_device_status() == zs.ZS_DEVERR_NONE
    for limit in (1, 300, 3000):                 # most of these waits end in time
        zs.zs_set_q8_wait_limit(limit)
        call()
        torch.cuda.synchronize()
        assert zs.zs_device_status(clear=True) in (zs.ZS_DEVERR_NONE, code)
    zs.zs_set_q8_wait_limit()
    call()
    assert all(torch.equal(a, b) for a, b in zip(_bits(outs), want))


# CTA pairs in several widths, many tiles each and one; whole sums and sums split over clusters, few rows of either operand
@pytest.mark.parametrize("m,n,k", [(2600, 1500, 1100), (5000, 4000, 300), (2561, 1537, 77), (1, 22016, 512), (5, 3000, 2000),
                                   (200, 100, 5000), (513, 33, 3000), (300, 300, 300)])
def test_product(m, n, k):
    a, b = _filled(m, k, 1)[1], _filled(n, k, 2, 0.02)[1]
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    _runs_out(lambda: zs.zs_q8_matmul(a, b, out), [out], zs.ZS_DEVERR_MATMUL_WAIT)


# one tile and several per CTA
@pytest.mark.parametrize("rows,cols", [(300, 520), (9000, 2048)])
def test_encode(rows, cols):
    x, q = _filled(rows, cols, 3)
    q_t = zs.q8_empty(cols, rows)
    _runs_out(lambda: zs.zs_q8_encode(x, q, q_t), [*q, *q_t], zs.ZS_DEVERR_TILE_WAIT)


@pytest.mark.parametrize("rows,cols", [(300, 520), (9000, 2048)])
def test_transpose(rows, cols):
    q, q_t = _filled(rows, cols, 4)[1], zs.q8_empty(cols, rows)
    _runs_out(lambda: zs.zs_q8_transpose(q, q_t), list(q_t), zs.ZS_DEVERR_TILE_WAIT)


@pytest.mark.parametrize("rows,cols", [(300, 520), (9000, 2048)])
@pytest.mark.parametrize("start", [0, 1])
def test_gate_backward(rows, cols, start):
    # from an odd start the threads copy dh themselves, and wait for that before they look: the codes may be there by then
    gate, up = _filled(rows, cols, 5)[1], _filled(rows, cols, 6)[1]
    dh = _filled(rows, cols + 8, 7, 1e-3)[0][:, start:start + cols]
    outs = [zs.q8_empty(rows, cols) for _ in range(2)] + [zs.q8_empty(cols, rows) for _ in range(3)]
    _runs_out(lambda: zs.zs_swiglu_backward_q8(dh, gate, up, *outs), [x for q in outs for x in q], zs.ZS_DEVERR_TILE_WAIT,
              surely=start == 0)


@pytest.mark.parametrize("kept8", [False, True])
def test_norm_backward(kept8):
    # rows through the ring: many per CTA, of 256 threads and more
    rows, cols = 6001, 4096
    dy, ds = _filled(rows, cols, 8)[0], _filled(rows, cols, 9)[0]
    s = _filled(rows, cols, 10)[1 if kept8 else 0]
    weight, rstd = _filled(1, cols, 11)[0][0], torch.ones(rows, device="cuda")
    dx, dw = torch.empty_like(dy), torch.empty_like(weight)
    partials = torch.zeros(304, cols, device="cuda")
    _runs_out(lambda: zs.zs_rmsnorm_backward(dy, s, weight, rstd, dx, dw, partials, ds=ds), [dx, dw], zs.ZS_DEVERR_TILE_WAIT)
