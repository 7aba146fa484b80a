"""Refusals of the experts' operators: bad arguments are found before anything is enqueued (no GPU)."""

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
from test_abi_q8 import A, BAD_Q, BIG, _q


def _call(name, args):
    return getattr(zs._lib, name)(*args.values())


PLACES = dict(starts=A, counts=A, n_experts=3)
SORT = dict(ids=A, id_bytes=8, tokens=4, choices=2, n_experts=3, align=128, row_of=A, starts=A, counts=A, stream=None)
DISPATCH = dict(x=A, ldx=200, tokens=4, cols=200, row_of=A, choices=2, **PLACES, rows=9, y=_q(), y_bf16=A, ldy=200, stream=None)
COMBINE = dict(y=A, ldy=200, rows=9, cols=200, row_of=A, weights=A, tokens=4, choices=2, residual=A, ldr=200, out=A, ldo=200, stream=None)
BACK = dict(dout=A, lddout=200, y=A, ldy=200, rows=9, cols=200, row_of=A, weights=A, tokens=4, choices=2, **PLACES, dy=_q(), dy_bf16=A,
            lddy=200, dweights=A, stream=None)
ROWS = dict(a=_q(), b=_q(), starts=A, n_experts=3, m=4, n=5, k=200, scale=1.0, first=1, out=A, ldo=5, stream=None)
ROUTES = [dict(tokens=-1), dict(tokens=BIG), dict(choices=0), dict(choices=33), dict(row_of=None), dict(row_of=A + 2)]
EXPERTS = [dict(n_experts=0), dict(n_experts=1025), dict(starts=None), dict(starts=A + 1), dict(counts=None), dict(counts=A + 2)]
PLANES = [dict(rows=-1), dict(rows=BIG), dict(cols=0), dict(cols=BIG)]

CASES = [("zs_expert_sort", SORT, c) for c in ROUTES + EXPERTS + [
    dict(ids=None), dict(ids=A + 4), dict(id_bytes=2), dict(id_bytes=4, ids=A + 2), dict(align=0), dict(align=65537), dict(tokens=BIG // 2),
    dict(tokens=(BIG - 256 - 3 * 127) // 2 + 1)]]
CASES += [("zs_expert_dispatch", DISPATCH, c) for c in ROUTES + EXPERTS + PLANES + [
    dict(x=None), dict(x=A + 1), dict(ldx=199), dict(y=None, y_bf16=None), dict(y_bf16=A + 1), dict(ldy=199)] + [dict(y=q) for q in BAD_Q]]
CASES += [("zs_expert_combine", COMBINE, c) for c in ROUTES + PLANES + [
    dict(y=None), dict(y=A + 1), dict(ldy=1), dict(weights=A + 2), dict(residual=A + 1), dict(ldr=199), dict(out=None), dict(out=A + 1), dict(ldo=3)]]
CASES += [("zs_expert_combine_backward", BACK, c) for c in ROUTES + EXPERTS + PLANES + [
    dict(dout=None), dict(lddout=3), dict(y=None), dict(ldy=199), dict(weights=A + 1), dict(dweights=A + 2), dict(dy_bf16=A + 1), dict(lddy=2),
    dict(dy=None, dy_bf16=None, dweights=None)] + [dict(dy=q) for q in BAD_Q]]
for name in ("zs_q8_matmul_experts", "zs_q8_matmul_experts_grad"):
    CASES += [(name, ROWS, c) for c in [
        dict(a=None), dict(b=None), dict(starts=None), dict(starts=A + 2), dict(n_experts=0), dict(n_experts=1025), dict(m=-1), dict(n=-1),
        dict(k=-1), dict(k=BIG), dict(m=BIG), dict(n=BIG), dict(out=None), dict(out=A + 1), dict(ldo=4), dict(scale=float("nan")),
        dict(scale=float("inf"))] + [dict(a=q) for q in BAD_Q] + [dict(b=q) for q in BAD_Q]]
CASES += [("zs_q8_matmul_experts", ROWS, dict(k=0)), ("zs_q8_matmul_experts", ROWS, dict(n=BIG // 3, ldo=BIG)),
          ("zs_q8_matmul_experts_grad", ROWS, dict(m=BIG // 3))]


@pytest.mark.parametrize("name,args,change", CASES, ids=lambda v: str(v) if isinstance(v, str) else "")
def test_refused_with_a_message(name, args, change):
    assert _call(name, dict(args, **change)) == zs.ZS_ERR_INVALID
    text = zs.zs_last_error()
    assert text.startswith(name + ": ") and len(text) > len(name) + 8


@pytest.mark.parametrize("name,args,empty", [("zs_expert_dispatch", DISPATCH, "tokens"), ("zs_expert_dispatch", DISPATCH, "rows"),
                                             ("zs_expert_combine", COMBINE, "tokens"), ("zs_expert_combine_backward", BACK, "tokens"),
                                             ("zs_q8_matmul_experts", ROWS, "m"), ("zs_q8_matmul_experts", ROWS, "n"),
                                             ("zs_q8_matmul_experts_grad", ROWS, "m"), ("zs_q8_matmul_experts_grad", ROWS, "n")])
def test_nothing_to_do_enqueues_nothing(name, args, empty):
    assert _call(name, dict(args, **{empty: 0})) == zs.ZS_OK


def test_the_binding_refuses_tensors_that_do_not_fit():
    i = torch.zeros(4, 2, dtype=torch.int32)
    x = torch.zeros(4, 200, dtype=torch.bfloat16)
    starts, counts = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_expert_sort(i, 128, i, starts, counts)
    with pytest.raises(ValueError, match="matrix"):
        zs.zs_expert_sort(i[0], 128, i, starts, counts)
    with pytest.raises(ValueError, match="neither"):
        zs.zs_expert_dispatch(x, i, starts, counts)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_expert_combine(x, i, None, x)
    with pytest.raises(ValueError, match="out must be 12 x 5"):
        zs.zs_q8_matmul_experts_grad(zs.q8_empty(4, 200, device="cpu"), None, starts, torch.zeros(4, 5, dtype=torch.bfloat16))


def test_rows_that_are_always_enough():
    assert zs.expert_rows(0, 4, 8, 128) == 0 and zs.expert_rows(5, 2, 3) == 10
    assert zs.expert_rows(1, 8, 64, 128) == 8 * 128 and zs.expert_rows(1000, 2, 8, 128) % 128 == 0
    assert zs.expert_rows(1000, 2, 8, 128) >= 2000 + 8 * 127
