"""The 8-bit operators' Python calls take tensors of the current device only (no GPU: tensors that only say where
they are)."""

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class _Placed:
    """What the binding asks of a tensor, said for a tensor on GPU 0; there is no memory behind it."""

    def __init__(self, *shape, dtype=BF16, device=0):
        self.like = torch.empty(shape, dtype=dtype, device="meta")
        self.device = device
        self.dtype, self.shape, self.is_cuda = dtype, self.like.shape, True

    def get_device(self):
        return self.device

    def data_ptr(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.like, name)


class _NoLibrary:
    """A library whose calls must not be made."""

    def __getattr__(self, name):
        return lambda *args: pytest.fail(name + " was called")


def _q8(rows, cols):
    return _Placed(rows, -(-cols // 16) * 16, dtype=U8), _Placed(rows, -(-cols // 128), dtype=U8)


def _calls():
    M, C = 32, 256
    m, q, q_t, vec = lambda: _Placed(M, C), lambda: _q8(M, C), lambda: _q8(C, M), lambda: _Placed(C)  # noqa: E731
    return [
        (zs.zs_q8_encode, dict(x=m(), q=q(), q_t=q_t())),
        (zs.zs_q8_decode, dict(q=q(), y=m())),
        (zs.zs_q8_transpose, dict(q=q(), q_t=q_t())),
        (zs.zs_q8_matmul, dict(a=q(), b=_q8(64, C), out=_Placed(M, 64))),
        (zs.zs_rmsnorm_q8, dict(x=m(), residual=m(), weight=vec(), eps=1e-5, y=q(), s=m(), rstd=_Placed(M, dtype=F32), s_q8=q())),
        (zs.zs_rmsnorm_backward, dict(dy=m(), s=q(), weight=vec(), rstd=_Placed(M, dtype=F32), dx=m(), dw=vec(),
                                      partials=_Placed(8, C, dtype=F32), ds=m())),
        (zs.zs_rmsnorm_backward, dict(dy=m(), s=m(), weight=vec(), rstd=_Placed(M, dtype=F32), dx=m(), dw=vec(),
                                      partials=_Placed(8, C, dtype=F32))),
        (zs.zs_swiglu_q8, dict(gate=m(), up=m(), h=q(), gate_q=q(), up_q=q())),
        (zs.zs_swiglu_backward_q8, dict(dh=m(), gate_q=q(), up_q=q(), dgate=q(), dup=q(), dgate_t=q_t(), dup_t=q_t(), h_t=q_t())),
    ]


CASES = [(i, name, part) for i, (_, args) in enumerate(_calls()) for name, v in args.items()
         for part in ((0, 1) if isinstance(v, tuple) else (None,) if isinstance(v, _Placed) else ())]


@pytest.mark.parametrize("i,name,part", CASES)
def test_a_tensor_of_another_device_is_refused(monkeypatch, i, name, part):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(zs, "_lib", _NoLibrary())
    call, args = _calls()[i]
    (args[name] if part is None else args[name][part]).device = 1
    with pytest.raises(ValueError, match=r"^%s.* is on cuda:1 and the current device is cuda:0$" % name):
        call(**args)


@pytest.mark.parametrize("i", range(len(_calls())))
def test_nothing_is_enqueued_on_a_device_that_holds_none_of_the_tensors(monkeypatch, i):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(zs, "_lib", _NoLibrary())
    call, args = _calls()[i]
    with pytest.raises(ValueError, match="is on cuda:0 and the current device is cuda:1"):
        call(**args)


def test_a_star_import_has_what_the_calls_take():
    names = {}
    exec("from fsdp_sharded_optimizer_flatparameter_gb300 import *", names)
    assert {"q8_empty", "zs_q8", "ZS_Q8_BLOCK", "ZS_Q8_MAX_PARTIALS", "ZS_DEVERR_TILE_WAIT"} <= set(names)
    assert {n for n in zs.EXPORTED if hasattr(zs, n)} <= set(names) and "Plan" in names
