"""The large product in every tile width, over sums longer than its rings of stages and of scales and over several tiles
per pair of CTAs, with rows of codes that begin at 128-byte lines and that do not."""

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
import q8_torch64 as q64
from q8_helpers import U16, U32, Bf16Matrix, Q8Matrix

pytestmark = pytest.mark.gpu

# width: on 76 pairs of CTAs.  Sums of 7 blocks go round the ring of six stages, of 17 take two batches of scales and
# one block of a third group's; the last tiles are ragged in both directions.
SIZES = [("128, two tiles per pair", 3105, 1292, 2147), ("128, two tiles per pair", 3097, 1302, 869),
         ("160, four", 8249, 1345, 2176), ("160, three", 6463, 1125, 896),
         ("192, three", 6412, 1292, 2100), ("192, four", 1554, 7210, 890),
         ("224, three", 8221, 1162, 2176), ("224, four", 1538, 8491, 2160), ("224, four", 1556, 8262, 881),
         ("256, three", 2063, 6355, 2176), ("256, one", 1545, 2262, 896)]


@pytest.fixture(autouse=True)
def _status_stays_clear():
    yield
    torch.cuda.synchronize()
    assert zs.zs_device_status(clear=True) == zs.ZS_DEVERR_NONE


def _operand(rows, k, lines, seed):
    """Every block with a scale of its own, so that one taken from a neighbouring row, block or group shows."""
    ld = -(-k // 128) * 128 + 128 if lines else -(-k // 16) * 16 + 16
    if not lines and ld % 128 == 0:
        ld += 16
    m = Q8Matrix(rows, k, pad_cols=ld - -(-k // 16) * 16, lead=128)
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 0x50, (rows, k), generator=g, device="cuda") | torch.randint(0, 2, (rows, k), generator=g, device="cuda") << 7
    m.codes.copy_(codes.to(torch.uint8))
    m.scales.copy_(torch.randint(117, 138, m.scales.shape, generator=g, device="cuda").to(torch.uint8))
    assert m.codes.stride(0) == ld and (ld % 128 == 0) == lines
    return m


@pytest.mark.parametrize("lines", [True, False])
@pytest.mark.parametrize("width,m,n,k", SIZES)
def test_product(width, m, n, k, lines):
    a, b = _operand(m, k, lines, 1), _operand(n, k, lines, 2)
    av, bv = q64.decode(a.codes, a.scales), q64.decode(b.codes, b.scales)
    want = av @ bv.t()
    # one rounding to bf16; the sum: one addition per 32 columns kept to 2^-23 or better and the additions inside them
    bound = U16 * want.abs() + (k / 8 + 16) * 2 * U32 * (av.abs() @ bv.abs().t())
    for layout in (dict(lead=0, pad=-n % 16), dict(lead=8, pad=8 - n % 8), dict(lead=1, pad=(n + 1) % 2)):
        out = Bf16Matrix(m, n, **layout)
        out.t.fill_(float("nan"))
        zs.zs_q8_matmul(a.pair, b.pair, out.t)
        q64.check_close(out.t, want, bound)
        out.assert_untouched_outside()
        first = out.t.clone()
        before = (torch.randn(m, n, device="cuda") * float(want.abs().max())).to(torch.bfloat16)
        out.t.copy_(before)
        zs.zs_q8_matmul(a.pair, b.pair, out.t, scale=-0.25, first=False)
        both = before.double() - 0.25 * want
        q64.check_close(out.t, both, bound + U16 * both.abs() + 2 * U32 * before.double().abs())
        out.assert_untouched_outside()
        for _ in range(3):                       # the same bits again
            zs.zs_q8_matmul(a.pair, b.pair, out.t)
            assert torch.equal(out.t, first)
