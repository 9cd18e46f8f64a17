"""The binding of the operators around the experts' products hands only the current GPU's
memory to the library: calls with a tensor in host memory, or on another GPU, are refused
before the library is called. (A tensor class that says where it is stands for GPU tensors.)"""
import types

import pytest
import torch

from mxfp4_microscaling_quantization_amd import mxq
from tests.test_mm_devices_cpu import OnGpu0, OnGpu1


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, and a current device 0."""
    made = []
    stub = types.SimpleNamespace(mxq_act_grad_workspace=lambda *a: 64, mxq_expert_sort_workspace=lambda *a: 64)
    for name in ("mxq_route", "mxq_route_grad", "mxq_expert_sort", "mxq_dispatch", "mxq_combine", "mxq_combine_grad",
                 "mxq_fp8_quantize", "mxq_fp8_act_grad"):
        setattr(stub, name, lambda *a, name=name: made.append(name) or mxq.MXQ_OK)
    monkeypatch.setattr(mxq, "lib", lambda: stub)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return made


def f32(*shape):
    return torch.zeros(shape)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


CALLS = {
    "route": (lambda t: mxq.mxq_route(t[0], 2, out=(t[1], t[2])), [f32(4, 8), f32(4, 2), i32(4, 2)]),
    "route_grad": (lambda t: mxq.mxq_route_grad(t[0], t[1], t[2], t[3], out=t[4]),
                   [f32(4, 2), f32(4, 2), i32(4, 2), f32(4, 8), f32(4, 8)]),
    "expert_sort": (lambda t: mxq.mxq_expert_sort(t[0], 8, mxq.ExpertRows(t[1], t[2], t[3]), t[4]),
                    [i32(4, 2), torch.zeros(9, dtype=torch.int64), i32(4, 2), i32(8), u8(64)]),
    "dispatch": (lambda t: mxq.mxq_dispatch(t[0], t[1], out=t[2]), [f32(4, 32), i32(4, 2), f32(8, 32)]),
    "dispatch_fp8": (lambda t: mxq.mxq_dispatch(t[0], t[1], fmt="fp8", out=(t[2], t[3])),
                     [f32(4, 128), i32(4, 2), u8(8, 128), f32(8, 1)]),
    "combine": (lambda t: mxq.mxq_combine(t[0], t[1], t[2], t[3], out=t[4]),
                [f32(8, 32), i32(4, 2), f32(4, 2), f32(4, 32), f32(4, 32)]),
    "combine_grad": (lambda t: mxq.mxq_combine_grad(t[0], t[1], t[2], t[3], out=t[4], dw=t[5]),
                     [f32(4, 32), f32(8, 32), i32(4, 2), f32(4, 2), f32(8, 32), f32(4, 2)]),
    "fp8_quantize": (lambda t: mxq.mxq_fp8_quantize(t[0], out=(t[1], t[2])), [f32(4, 200), u8(4, 200), f32(4, 2)]),
    "fp8_act_grad": (lambda t: mxq.mxq_fp8_act_grad(t[0], (t[1], t[2]), "gelu", t[3], True, True, t[4], t[5], t[6], t[7]),
                     [f32(4, 8), u8(4, 8), f32(4, 1), torch.tensor([0, 1, 4]), f32(4, 8), f32(2, 8), f32(4, 8), u8(64)]),
}
# outputs that the call makes itself
MADE = {
    "route": (lambda t: mxq.mxq_route(t[0], 2), [f32(4, 8)]),
    "route_grad": (lambda t: mxq.mxq_route_grad(*t), [f32(4, 2), f32(4, 2), i32(4, 2), f32(4, 8)]),
    "expert_sort": (lambda t: mxq.mxq_expert_sort(t[0], 8), [i32(4, 2)]),
    "dispatch": (lambda t: mxq.mxq_dispatch(*t), [f32(4, 32), i32(4, 2)]),
    "dispatch_mxfp4": (lambda t: mxq.mxq_dispatch(*t, fmt="mxfp4"), [f32(4, 32), i32(4, 2)]),
    "combine": (lambda t: mxq.mxq_combine(t[0], t[1], t[2], t[3], torch.float32),
                [f32(8, 32), i32(4, 2), f32(4, 2), f32(4, 32)]),
    "combine_grad": (lambda t: mxq.mxq_combine_grad(*t), [f32(4, 32), f32(8, 32), i32(4, 2), f32(4, 2)]),
    "fp8_quantize": (lambda t: mxq.mxq_fp8_quantize(*t), [f32(4, 200)]),
    "fp8_act_grad": (lambda t: mxq.mxq_fp8_act_grad(t[0], (t[1], t[2]), "gelu", t[3], True, True),
                     [f32(4, 8), u8(4, 8), f32(4, 1), torch.tensor([0, 1, 4])]),
}
ALL = [(n, c) for table in (CALLS, MADE) for n, c in table.items()]


@pytest.mark.parametrize("call", [c for _, c in ALL], ids=[n for n, _ in ALL])
def test_all_on_the_current_gpu(calls, call):
    call[0]([t.as_subclass(OnGpu0) for t in call[1]])
    assert len(calls) == 1


@pytest.mark.parametrize("call,which", [(c, i) for _, c in ALL for i in range(len(c[1]))],
                         ids=[f"{n}-{i}" for n, c in ALL for i in range(len(c[1]))])
def test_one_elsewhere(calls, call, which):
    fn, tensors = call
    on = [t.as_subclass(OnGpu0) for t in tensors]
    for other in (tensors[which], tensors[which].as_subclass(OnGpu1)):
        with pytest.raises(ValueError, match="current GPU"):
            fn(on[:which] + [other] + on[which + 1:])
    assert not calls
