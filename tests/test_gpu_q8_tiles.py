"""The persistent kernels with several tiles per CTA: encode, transpose and the gate's backward pass, with more and with
fewer tiles across than CTAs, ragged at both edges."""

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
import q8_torch64 as q64
from q8_helpers import Q8Matrix, U32

pytestmark = pytest.mark.gpu

# 1188 and 1224 tiles of 128 columns (two CTAs to an SM: about 304 at a time), 33 and 408 across; 2840 and 3260 of the
# transpose's 64 (four CTAs to an SM), 40 and 815 across
SIZES = [(4501, 4200), (300, 52111)]
TURNS = [(9001, 2500), (401, 52111)]


@pytest.fixture(autouse=True)
def _status_stays_clear():
    yield
    torch.cuda.synchronize()
    assert zs.zs_device_status(clear=True) == zs.ZS_DEVERR_NONE


def _bf16(rows, cols, start, seed, sigma=1.0):
    """Values whose rows and columns differ in size, from element `start` of a buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.zeros(start + rows * cols + 16, dtype=torch.bfloat16, device="cuda")
    x = buf[start:start + rows * cols].view(rows, cols)
    f = torch.randn(rows, cols, generator=g, device="cuda") * sigma
    f *= torch.exp2(torch.randint(-9, 10, (rows, 1), generator=g, device="cuda"))
    f *= torch.exp2(torch.randint(-4, 1, (1, cols), generator=g, device="cuda"))
    x.copy_(f)
    return x


def _coded(rows, cols, seed, sigma):
    """A matrix in 8 bits with blocks of every size, inside sentinel bytes."""
    m = Q8Matrix(rows, cols)
    codes, scales = q64.encode(_bf16(rows, cols, 0, seed, sigma).double())
    m.codes.copy_(codes)
    m.scales.copy_(scales)
    return m


# cols of 4200 and 52111: rows 16-byte aligned (tiled copies) and not; start 1: never
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("start", [0, 1])
def test_encode_both_ways(rows, cols, start):
    x = _bf16(rows, cols, start, rows + start)
    want, want_t = q64.encode(x.double()), q64.encode(x.double().t().contiguous())
    q, q_t = Q8Matrix(rows, cols), Q8Matrix(cols, rows)
    zs.zs_q8_encode(x, q.pair, q_t.pair)
    assert q64.same((q.codes, q.scales), want) and q64.same((q_t.codes, q_t.scales), want_t)
    one, other = Q8Matrix(rows, cols), Q8Matrix(cols, rows)
    zs.zs_q8_encode(x, one.pair)
    zs.zs_q8_encode(x, None, other.pair)
    assert q64.same((one.codes, one.scales), want) and q64.same((other.codes, other.scales), want_t)
    for m in (q, q_t, one, other):
        m.assert_untouched_outside()


@pytest.mark.parametrize("rows,cols", [(4501, 4200), (300, 52112)])
def test_encode_of_aligned_rows(rows, cols):
    x = _bf16(rows, cols, 0, rows)
    q, q_t = Q8Matrix(rows, cols), Q8Matrix(cols, rows)
    zs.zs_q8_encode(x, q.pair, q_t.pair)
    assert q64.same((q.codes, q.scales), q64.encode(x.double()))
    assert q64.same((q_t.codes, q_t.scales), q64.encode(x.double().t().contiguous()))


@pytest.mark.parametrize("rows,cols", TURNS)
def test_transpose(rows, cols):
    q, q_t = _coded(rows, cols, rows, 1.0), Q8Matrix(cols, rows)
    zs.zs_q8_transpose(q.pair, q_t.pair)
    assert q64.same((q_t.codes, q_t.scales), q64.encode(q64.decode(q.codes, q.scales).t().contiguous()))
    q_t.assert_untouched_outside()


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("start", [0, 1])
def test_gate_backward(rows, cols, start):
    gate, up = _coded(rows, cols, 1, 0.015), _coded(rows, cols, 2, 1.0)
    dh = _bf16(rows, cols, start, 3, 1e-3)
    outs = [Q8Matrix(rows, cols) for _ in range(2)] + [Q8Matrix(cols, rows) for _ in range(3)]
    zs.zs_swiglu_backward_q8(dh, gate.pair, up.pair, *(o.pair for o in outs))
    g, u, d = q64.decode(gate.codes, gate.scales), q64.decode(up.codes, up.scales), dh.double()
    p = torch.sigmoid(g)
    dg, du, h = d * u * p * (1 + g * (1 - p)), d * g * p, g * p * u
    # the sigmoid: the exponent's two roundings (2^-24 and 2^-25 of |gate| log2 e, gates below 52) times ln 2, the
    # hardware's power of two and reciprocal (2^-22 each); a few products and sums of 2^-24; 1 + gate (1 - p) cancels for
    # negative gates, so its roundings, the sigmoid's among them, are relative to 1 + |gate|
    rel = 80 * U32 + 2 * 2.0 ** -22 + 8 * U32
    errs = (rel * (d * u * p).abs() * (1 + g.abs()), rel * du.abs(), rel * h.abs())
    assert float(g.abs().max()) < 52
    for o, want, err in zip(outs, (dg, du, dg.t(), du.t(), h.t()), (errs[0], errs[1], errs[0].t(), errs[1].t(), errs[2].t())):
        q64.check_encoded((o.codes, o.scales), want.contiguous(), err.contiguous() + 2.0 ** -140)
        o.assert_untouched_outside()
    for k in range(5):                                             # each output by itself
        alone = Q8Matrix(outs[k].rows, outs[k].cols)
        zs.zs_swiglu_backward_q8(dh, gate.pair, up.pair, *(alone.pair if i == k else None for i in range(5)))
        assert torch.equal(alone.codes, outs[k].codes) and torch.equal(alone.scales, outs[k].scales)
