"""Refusals of the step over many tensors and of the gradients' norm (no GPU)."""

import ctypes

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
from test_q8_binding import _Placed

A = 1 << 20
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
NAN, INF = float("nan"), float("inf")


def _list(**change):
    ts = (zs.zs_tensor * 2)()
    for t in ts:
        t.n, t.grad, t.master, t.param, t.m, t.v, t.m_scale, t.v_scale = 300, A, A, A, A, A, A, A
    for k, v in change.items():
        setattr(ts[1], k, v)
    return ts


def _step(ts=None, count=2, grad_bytes=2, bits=8, hp=HP, step=1, factor=A):
    return zs._lib.zs_adamw_tensors(_list() if ts is None else ts, count, grad_bytes, bits,
                                    None if hp is None else ctypes.byref(zs._hp(hp)), step, factor, 0, None)


def _norm(ts=None, count=2, grad_bytes=2, max_norm=1.0, partials=A, n_partials=5, out=A):
    return zs._lib.zs_grad_norm(_list() if ts is None else ts, count, grad_bytes, max_norm, partials, n_partials, out, None)


def _refused(rc, name, says):
    assert rc == zs.ZS_ERR_INVALID
    assert zs.zs_last_error().startswith(name + ": ") and says in zs.zs_last_error()


@pytest.mark.parametrize("change,says", [
    (dict(n=-1), "n of tensor 1"), (dict(n=(1 << 40) + 1), "n of tensor 1"), (dict(grad=None), "grad of tensor 1"), (dict(grad=A + 1), "grad of tensor 1"),
    (dict(master=None), "master"), (dict(m=None), "master, m or v"), (dict(v=None), "master, m or v"), (dict(master=A + 2), "aligned"),
    (dict(param=A + 1), "param of tensor 1"), (dict(m_scale=None), "m_scale"), (dict(v_scale=A + 2), "v_scale")])
def test_step_refuses_a_tensor(change, says):
    _refused(_step(_list(**change)), "zs_adamw_tensors", says)


@pytest.mark.parametrize("change,says", [
    (dict(count=-1), "n_tensors"), (dict(grad_bytes=8), "grad_bytes"), (dict(bits=16), "state_bits"), (dict(hp=None), "hparams"),
    (dict(step=0), "step"), (dict(factor=A + 2), "factor"), (dict(hp=dict(HP, lr=NAN)), "finite"), (dict(hp=dict(HP, weight_decay=INF)), "finite"),
    (dict(hp=dict(HP, beta1=1.0)), "betas"), (dict(hp=dict(HP, beta2=-0.1)), "betas"), (dict(ts=_list(m=A + 2), bits=32), "aligned"),
    (dict(ts=_list(grad=A + 2), grad_bytes=4), "grad of tensor 1")])
def test_step_refuses_a_call(change, says):
    _refused(_step(**change), "zs_adamw_tensors", says)


def test_step_refuses_a_missing_list():
    assert zs._lib.zs_adamw_tensors(None, 1, 2, 8, ctypes.byref(zs._hp(HP)), 1, None, 0, None) == zs.ZS_ERR_INVALID
    assert zs._lib.zs_grad_norm(None, 1, 2, 1.0, A, 5, A, None) == zs.ZS_ERR_INVALID


@pytest.mark.parametrize("change,says", [
    (dict(count=-1), "n_tensors"), (dict(grad_bytes=1), "grad_bytes"), (dict(max_norm=0.0), "max_norm"), (dict(max_norm=-1.0), "max_norm"),
    (dict(max_norm=NAN), "max_norm"), (dict(max_norm=INF), "max_norm"), (dict(partials=None), "partials"), (dict(partials=A + 1), "partials"),
    (dict(n_partials=0), "n_partials"), (dict(n_partials=1), "n_partials"), (dict(out=None), "out"), (dict(out=A + 2), "out"), (dict(ts=_list(grad=None)), "grad of tensor 1")])
def test_norm_refuses_a_call(change, says):
    _refused(_norm(**change), "zs_grad_norm", says)


def test_empty_lists_enqueue_nothing():
    assert _step(count=0) == zs.ZS_OK
    empty = _list(n=0, grad=None, master=None, m=None, v=None)
    empty[0].n = 0
    assert _step(empty) == zs.ZS_OK


def test_the_structure_is_the_headers():
    assert ctypes.sizeof(zs.zs_tensor) == 72 and zs.zs_tensor.no_decay.offset == 64


class _At(_Placed):
    """A tensor on GPU 0 with an address of its own."""

    def data_ptr(self):
        return id(self) * 64


def _arrays(**change):
    P = lambda n, dtype, **kw: _At(n, dtype=dtype, **kw)  # noqa: E731
    a = dict(grads=[P(300, BF16), P(5, BF16)], master=[P(300, F32), P(5, F32)], m=[P(300, U8), P(5, U8)], v=[P(300, U8), P(5, U8)],
             params=[P(300, BF16), None], m_scales=[P(2, F32), P(1, F32)], v_scales=[P(2, F32), P(1, F32)])
    return dict(a, **change)


def test_a_list_of_tensors_that_fit():
    ts = zs.TensorList(**_arrays(no_decay=[False, True]))
    assert len(ts) == 2 and ts.state_bits == 8 and ts.grad_bytes == 2 and ts.device == 0
    assert ts._array[0].n == 300 and ts._array[1].no_decay == 1 and not ts._array[1].param
    with pytest.raises(ValueError, match="current device"):
        zs.zs_adamw_tensors(ts, HP, 1)
    with pytest.raises(ValueError, match="current device"):
        zs.zs_grad_norm(ts, 1.0, None, None)


@pytest.mark.parametrize("change,says", [
    (dict(master=[_Placed(300, dtype=F32)]), "master holds 1"), (dict(m_scales=None), "belong together"),
    (dict(master=[_Placed(300, dtype=BF16), _Placed(5, dtype=F32)]), r"master\[0\]"), (dict(m=[_Placed(300, dtype=F32), _Placed(5, dtype=U8)]), r"m\[0\]"),
    (dict(v=[_Placed(300, dtype=U8), _Placed(6, dtype=U8)]), r"v\[1\] must hold 5"), (dict(v_scales=[_Placed(1, dtype=F32)] * 2), r"v_scales\[0\] must hold 2"),
    (dict(grads=[_Placed(300, dtype=BF16), _Placed(5, dtype=F32)]), r"grads\[1\]"), (dict(grads=[_Placed(300, dtype=torch.float16), _Placed(5, dtype=torch.float16)]), "grads"),
    (dict(params=[_Placed(300, dtype=F32), None]), r"params\[0\]"), (dict(params=[None, _Placed(5, dtype=BF16, device=1)]), "cuda:1"),
    (dict(m=[torch.zeros(300, dtype=U8), _Placed(5, dtype=U8)]), "CUDA")])
def test_a_list_refuses_tensors_that_do_not_fit(change, says):
    with pytest.raises(ValueError, match=says):
        zs.TensorList(**_arrays(**change))


def test_other_gradients_have_to_fit_too():
    ts = zs.TensorList(**_arrays())
    ts.set_grads([_Placed(300, dtype=F32), _Placed(5, dtype=F32)])
    assert ts.grad_bytes == 4
    with pytest.raises(ValueError, match="grads holds 1"):
        ts.set_grads([_Placed(300, dtype=F32)])
    with pytest.raises(ValueError, match="must hold 300"):
        ts.set_grads([_Placed(301, dtype=F32), _Placed(5, dtype=F32)])


def test_a_list_refuses_an_array_twice():
    a = _arrays()
    a["m"][1] = a["v"][1]
    with pytest.raises(ValueError, match="twice"):
        zs.TensorList(**a)
    a = _arrays(grads=[_At(300, dtype=BF16)] * 2, master=[_At(300, dtype=F32)] * 2, m=[_At(300, dtype=U8) for _ in "ab"],
                v=[_At(300, dtype=U8) for _ in "ab"], params=None, m_scales=[_At(2, dtype=F32) for _ in "ab"], v_scales=[_At(2, dtype=F32) for _ in "ab"])
    with pytest.raises(ValueError, match="twice"):
        zs.TensorList(**a)
    a["master"] = [_At(300, dtype=F32) for _ in "ab"]
    assert len(zs.TensorList(**a)) == 2                        # gradients are only read


def test_the_seed_is_the_steps_number_where_none_is_given(monkeypatch):
    class Library:
        def zs_adamw_tensors(self, *args):
            seen.append((args[5], args[7]))
            return 0
    seen = []
    ts = zs.TensorList(**_arrays())
    monkeypatch.setattr(zs, "_lib", Library())
    monkeypatch.setattr(zs, "_device", lambda: 0)
    monkeypatch.setattr(zs, "_here", lambda stream, dev: 7)
    for step, kw in ((1, {}), (2, {}), ((1 << 32) + 3, {}), (4, dict(seed=0)), (5, dict(seed=9)), (6, dict(seed=(1 << 32) + 5))):
        zs.zs_adamw_tensors(ts, HP, step, **kw)
    assert seen == [(1, 1), (2, 2), ((1 << 32) + 3, 3), (4, 0), (5, 9), (6, 5)]
