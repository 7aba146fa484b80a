"""The experts' products in every tile width, over several tiles per pair of CTAs, against the 64-bit oracle: uneven groups,
columns that the tiles share unevenly, tables that do not fit beside the widest tile."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
from oracle import experts, q8
from q8_helpers import U16, U32, Bf16Matrix, Q8Matrix, check_close, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_stays_clear():
    yield
    torch.cuda.synchronize()
    assert zs.zs_device_status(clear=True) == zs.ZS_DEVERR_NONE


def _width(tp, columns, blocks, widest=256):
    """The host's choice of a tile width, for operands whose rows are not a multiple of 128 bytes apart."""
    room = torch.cuda.get_device_properties(0).multi_processor_count // 2
    best, least = 128, 1e300
    for bn in (256, 224, 192, 160, 128):
        rounds = -(-tp * -(-columns // bn) // room)
        cost = rounds * blocks * (200 + 0.765 * bn) + 2500.0 * (rounds if bn == 256 else 1)
        if bn <= widest and cost < least:
            best, least = bn, cost
    return best


def _sizes(rng, groups, mean, unit=1):
    """Groups of `mean` units on average, one empty where there are several."""
    share = rng.uniform(0.3, 1.7, groups)
    if groups > 2:
        share[1] = 0
    at = np.round(np.concatenate([[0], np.cumsum(share / share.sum())]) * groups * mean).astype(int)
    return np.diff(at) * unit


def _operand(rng, rows, cols):
    """Codes of both signs below 32, and scales of their own for every block."""
    codes = (rng.integers(0, 0x60, (rows, cols)) | rng.integers(0, 2, (rows, cols)) << 7).astype(np.uint8)
    scales = rng.integers(117, 138, (rows, -(-cols // 128))).astype(np.uint8)
    return Q8Matrix(rows, cols).fill(codes, scales), q8.decode(codes, scales)


def _bound(size, want, k):
    # one rounding to bf16, products exact, an addition per 32 columns and those inside
    return U16 * np.abs(want) + (k / 8 + 16) * 2 * U32 * size


@pytest.mark.parametrize("width,groups,mean,n,k", [
    (160, 9, 1100, 700, 200), (192, 6, 600, 2050, 200), (224, 9, 600, 1700, 200), (224, 6, 1100, 1500, 384), (256, 3, 600, 1800, 1280),
    (256, 8, 600, 1536, 2304), (224, 740, 98, 400, 130), (192, 1024, 97, 520, 130)])
def test_rows(width, groups, mean, n, k):
    rng = np.random.default_rng(n + k)
    sizes = _sizes(rng, groups, mean)
    m = sum(sizes)
    assert _width(groups * (-(-(m // groups) // 256)), n, -(-k // 128), 256 if groups <= 735 else 224) == width
    a, av = _operand(rng, m, k)
    b, bv = _operand(rng, groups * n, k)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    host = starts.tolist()
    want, size = experts.product(av, bv, host), experts.product(np.abs(av), np.abs(bv), host)
    for layout in (dict(lead=0, pad=-n % 16), dict(lead=3, pad=5)):
        out = Bf16Matrix(m, n, **layout)
        out.t.fill_(float("nan"))
        zs.zs_q8_matmul_experts(a.pair, b.pair, starts, out.t)
        check_close(to64(out.t), want, _bound(size, want, k), "out")
        out.assert_untouched_outside()


@pytest.mark.parametrize("width,groups,m,n,blocks", [
    (160, 9, 900, 900, 9), (192, 9, 300, 2050, 9), (224, 9, 700, 1700, 9), (224, 9, 900, 1300, 20), (256, 8, 300, 1024, 20),
    (256, 8, 300, 2048, 120), (256, 8, 1200, 700, 120)])
def test_sums(width, groups, m, n, blocks):
    rng = np.random.default_rng(m + n)
    sizes = _sizes(rng, groups, blocks, 128)
    k = sum(sizes)
    assert _width(groups * -(-m // 256), n, k / 128 / groups) == width
    a, av = _operand(rng, m, k)
    b, bv = _operand(rng, n, k)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    host = starts.tolist()
    want, size = experts.product_grad(av, bv, host), experts.product_grad(np.abs(av), np.abs(bv), host)
    for layout in (dict(lead=0, pad=-n % 16), dict(lead=3, pad=5)):
        out = Bf16Matrix(groups * m, n, **layout)
        out.t.fill_(float("nan"))
        zs.zs_q8_matmul_experts_grad(a.pair, b.pair, starts, out.t)
        check_close(to64(out.t), want, _bound(size, want, max(sizes)) + 1e-38, "out")
        out.assert_untouched_outside()
