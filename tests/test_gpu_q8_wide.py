"""Rows of the gated activation longer than one launch's grid has room for."""

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs

pytestmark = pytest.mark.gpu


def _part(q, lo, hi):
    return q[0][:, lo:hi], q[1][:, lo // 128:-(-hi // 128)]


@pytest.mark.parametrize("start", [0, 1])
def test_gate_of_very_long_rows(start):
    """Against the same columns in three calls; the last few reach past the second launch's first piece."""
    rows, cols = 1, 2 ** 27 + 2 ** 25 + 77
    g = torch.Generator(device="cuda").manual_seed(5)
    both = torch.empty(2, cols + 16, dtype=torch.bfloat16, device="cuda")
    for row in both:
        row.copy_(torch.randn(cols + 16, generator=g, device="cuda"))
    gate, up = (x[None, start:start + cols] for x in both)
    outs = [zs.q8_empty(rows, cols) for _ in range(3)]
    for q in outs:
        q[0].view(torch.uint8).fill_(0x11)
        q[1].view(torch.uint8).fill_(0x11)
    zs.zs_swiglu_q8(gate, up, *outs)
    for lo, hi in ((0, 2 ** 26), (2 ** 26, 2 ** 27), (2 ** 27, cols)):
        want = [zs.q8_empty(rows, hi - lo) for _ in range(3)]
        zs.zs_swiglu_q8(gate[:, lo:hi], up[:, lo:hi], *want)
        for q, w in zip(outs, want):
            for x, y in zip(_part(q, lo, hi), w):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (lo, hi)
