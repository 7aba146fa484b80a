"""Refusals of the 8-bit operators: bad arguments are found before anything is enqueued (no GPU)."""

import ctypes

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs

LIB = ctypes.CDLL(zs.LIB_PATH)
A = 1 << 20                    # an aligned address that nothing may read


def _q(codes=A, scales=A, ld=256, ld_scales=2):
    return ctypes.byref(zs.zs_q8(codes, scales, ld, ld_scales))


def _call(name, *args):
    out = []
    for x in args:
        out.append(ctypes.c_float(x) if isinstance(x, float) else ctypes.c_int64(x) if isinstance(x, int) else x)
    return getattr(LIB, name)(*out)


ENCODE = dict(x=A, ldx=256, rows=4, cols=200, q=_q(), q_t=_q(ld=16, ld_scales=1), stream=None)
DECODE = dict(q=_q(), rows=4, cols=200, y=A, ldy=200, stream=None)
TRANSPOSE = dict(q=_q(), rows=4, cols=200, q_t=_q(ld=16, ld_scales=1), stream=None)
MATMUL = dict(a=_q(), b=_q(), m=4, n=5, k=200, scale=1.0, first=1, out=A, ldo=5, stream=None)
NORM = dict(x=A, ldx=200, residual=A, ldr=200, weight=A, eps=1e-5, rows=4, cols=200, y=_q(), s=A, lds=200, s_q8=_q(),
            rstd=A, stream=None)
BACK = dict(dy=A, lddy=200, s=None, lds=0, s_q8=_q(), weight=A, rstd=A, ds=A, ldds=200, rows=4, cols=200, dx=A, lddx=200,
            dw=A, scale=1.0, first=1, partials=A, n_partials=4, stream=None)
GATE = dict(gate=A, ldg=200, up=A, ldu=200, rows=4, cols=200, h=_q(), gate_q=_q(), up_q=_q(), stream=None)
GATE_BACK = dict(dh=A, lddh=200, gate_q=_q(), up_q=_q(), rows=4, cols=200, dgate=_q(), dup=_q(),
                 dgate_t=_q(ld=16, ld_scales=1), dup_t=None, h_t=None, stream=None)
BIG = 1 << 31
BAD_Q = [_q(codes=A + 8), _q(scales=None), _q(codes=None), _q(ld=192), _q(ld=250), _q(ld_scales=1), _q(ld=1 << 39)]

CASES = [("zs_q8_encode", ENCODE, c) for c in (
    [dict(x=None), dict(x=A + 1), dict(ldx=199), dict(rows=-1), dict(rows=BIG), dict(cols=0), dict(cols=BIG),
     dict(q=None, q_t=None), dict(q_t=_q(ld=0, ld_scales=1)), dict(q_t=_q(ld=16, ld_scales=0))] + [dict(q=q) for q in BAD_Q])]
CASES += [("zs_q8_decode", DECODE, c) for c in (
    [dict(y=None), dict(y=A + 1), dict(ldy=100), dict(q=None), dict(cols=0), dict(rows=-2)] + [dict(q=q) for q in BAD_Q])]
CASES += [("zs_q8_transpose", TRANSPOSE, c) for c in (
    [dict(q=None), dict(q_t=None), dict(rows=-1), dict(cols=0)] + [dict(q=q) for q in BAD_Q])]
CASES += [("zs_q8_matmul", MATMUL, c) for c in (
    [dict(a=None), dict(b=None), dict(m=-1), dict(n=-1), dict(k=-1), dict(m=BIG), dict(k=BIG), dict(out=None), dict(out=A + 1),
     dict(ldo=4), dict(scale=float("nan")), dict(scale=float("inf"))] + [dict(a=q) for q in BAD_Q] + [dict(b=q) for q in BAD_Q])]
CASES += [("zs_rmsnorm_q8", NORM, c) for c in (
    [dict(x=None), dict(weight=None), dict(weight=A + 1), dict(residual=A + 1), dict(ldx=10), dict(ldr=10), dict(lds=10),
     dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(y=None), dict(rstd=A + 2), dict(rows=-1), dict(cols=0)]
    + [dict(y=q) for q in BAD_Q] + [dict(s_q8=q) for q in BAD_Q])]
CASES += [("zs_rmsnorm_backward", BACK, c) for c in (
    [dict(dy=None), dict(s_q8=None), dict(s=A, lds=200), dict(weight=None), dict(rstd=None), dict(rstd=A + 2), dict(ldds=1),
     dict(dx=None), dict(dw=None), dict(dw=A + 1), dict(scale=float("nan")), dict(partials=None), dict(partials=A + 4),
     dict(n_partials=0), dict(lddx=199), dict(rows=-1), dict(cols=0)] + [dict(s_q8=q) for q in BAD_Q])]
CASES += [("zs_swiglu_q8", GATE, c) for c in (
    [dict(gate=None), dict(up=A + 1), dict(ldg=3), dict(ldu=3), dict(h=None), dict(rows=-1), dict(cols=0)]
    + [dict(h=q) for q in BAD_Q] + [dict(up_q=q) for q in BAD_Q])]
CASES += [("zs_swiglu_backward_q8", GATE_BACK, c) for c in (
    [dict(dh=None), dict(lddh=3), dict(gate_q=None), dict(up_q=None), dict(dgate=None, dup=None, dgate_t=None), dict(rows=-1),
     dict(cols=0), dict(dgate_t=_q(ld=0, ld_scales=1))] + [dict(dup=q) for q in BAD_Q])]


@pytest.mark.parametrize("name,args,change", CASES, ids=lambda v: str(v) if isinstance(v, str) else "")
def test_refused_with_a_message(name, args, change):
    assert _call(name, *dict(args, **change).values()) == zs.ZS_ERR_INVALID
    text = zs.zs_last_error()
    assert text.startswith(name + ": ") and len(text) > len(name) + 8


@pytest.mark.parametrize("name,args,empty", [("zs_q8_encode", ENCODE, "rows"), ("zs_q8_decode", DECODE, "rows"),
                                             ("zs_q8_transpose", TRANSPOSE, "rows"), ("zs_q8_matmul", MATMUL, "m"),
                                             ("zs_q8_matmul", MATMUL, "n"), ("zs_rmsnorm_q8", NORM, "rows"),
                                             ("zs_swiglu_q8", GATE, "rows"), ("zs_swiglu_backward_q8", GATE_BACK, "rows")])
def test_empty_matrices_enqueue_nothing(name, args, empty):
    assert _call(name, *dict(args, **{empty: 0}).values()) == zs.ZS_OK


def test_the_binding_refuses_tensors_that_do_not_fit():
    x = torch.zeros(4, 200, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_q8_encode(x, zs.q8_empty(4, 200, device="cpu"))
    with pytest.raises(ValueError, match="bfloat16"):
        zs.zs_q8_encode(x.float())
    with pytest.raises(ValueError, match="matrix"):
        zs.zs_q8_decode(None, x[0])
    with pytest.raises(ValueError, match="matrix"):
        zs.zs_rmsnorm_q8(x[0], None, x[0], 1e-5, None)


def test_an_empty_matrix_has_padded_rows():
    codes, scales = zs.q8_empty(3, 130, device="cpu")
    assert codes.shape == (3, 130) and codes.stride() == (144, 1) and scales.shape == (3, 2)
