"""The experts' Python calls take tensors of the current device only (no GPU: tensors that only say where they are)."""

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
from test_q8_binding import _NoLibrary, _Placed, _q8

I32, F32 = torch.int32, torch.float32


def _calls():
    T, K, E, C, R, N = 8, 2, 4, 256, 512, 128
    i = lambda *shape: _Placed(*shape, dtype=I32)  # noqa: E731
    places = lambda: dict(row_of=i(T, K), starts=i(E + 1), counts=i(E))  # noqa: E731
    return [
        (zs.zs_expert_sort, dict(ids=i(T, K), align=128, **places())),
        (zs.zs_expert_dispatch, dict(x=_Placed(T, C), **places(), y=_q8(R, C), y_bf16=_Placed(R, C))),
        (zs.zs_expert_combine, dict(y=_Placed(R, C), row_of=i(T, K), weights=_Placed(T, K, dtype=F32), out=_Placed(T, C), residual=_Placed(T, C))),
        (zs.zs_expert_combine_backward, dict(dout=_Placed(T, C), y=_Placed(R, C), **places(), weights=_Placed(T, K, dtype=F32),
                                             dweights=_Placed(T, K, dtype=F32), dy=_q8(R, C), dy_bf16=_Placed(R, C))),
        (zs.zs_q8_matmul_experts, dict(a=_q8(R, C), b=_q8(E * N, C), starts=i(E + 1), out=_Placed(R, N))),
        (zs.zs_q8_matmul_experts_grad, dict(a=_q8(N, R), b=_q8(C, R), starts=i(E + 1), out=_Placed(E * N, C))),
    ]


CASES = [(n, name, part) for n, (_, args) in enumerate(_calls()) for name, v in args.items()
         for part in ((0, 1) if isinstance(v, tuple) else (None,) if isinstance(v, _Placed) else ())]


@pytest.mark.parametrize("n,name,part", CASES, ids=lambda v: str(v))
def test_a_tensor_elsewhere_is_refused(monkeypatch, n, name, part):
    monkeypatch.setattr(zs, "_lib", _NoLibrary())
    monkeypatch.setattr(zs, "_device", lambda: 0)
    call, args = _calls()[n]
    (args[name] if part is None else args[name][part]).device = 1
    with pytest.raises(ValueError, match=r"(%s).*cuda:1" % name):
        call(**args)


@pytest.mark.parametrize("n,name,part", CASES, ids=lambda v: str(v))
def test_a_tensor_of_another_shape_or_type_is_refused(monkeypatch, n, name, part):
    monkeypatch.setattr(zs, "_lib", _NoLibrary())
    monkeypatch.setattr(zs, "_device", lambda: 0)
    call, args = _calls()[n]
    x = args[name] if part is None else args[name][part]
    for other in (_Placed(*[s + 1 for s in x.shape], dtype=x.dtype), _Placed(*x.shape, dtype=torch.float64)):
        if part is None:
            args[name] = other
        else:
            args[name] = tuple(other if p == part else q for p, q in enumerate(args[name]))
        with pytest.raises(ValueError):
            call(**args)


@pytest.mark.parametrize("n", range(len(_calls())))
def test_what_fits_reaches_the_library(monkeypatch, n):
    class Library:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, args)) or 0
    seen = []
    monkeypatch.setattr(zs, "_lib", Library())
    monkeypatch.setattr(zs, "_device", lambda: 0)
    monkeypatch.setattr(zs, "_here", lambda stream, dev: 7)
    call, args = _calls()[n]
    call(**args)
    assert seen[0][0] == call.__name__ and seen[0][1][-1] == 7
