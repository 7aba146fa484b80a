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


def _runs_out(call, outs, code):
    """call() as ever, then with waits that look once, then with very short ones, and as ever again."""
    call()
    want = _bits(outs)
    assert zs.zs_device_status() == zs.ZS_DEVERR_NONE
    for _ in range(10):
        zs.zs_set_q8_wait_limit(0)
        call()
        torch.cuda.synchronize()
        assert zs.zs_device_status(clear=True) == code
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
