"""A call's tensors lie on one device.  Tensors of another one are made without a GPU as fake tensors, which have
shapes and devices and no memory: the refusal has to come before anything is allocated or launched."""
import contextlib
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import chunked_gated_delta_04_gb300 as gdr

# a machine with a GPU makes its fake tensors' devices real ones, and need not have a second
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake devices")
F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32
# name: (shape, dtype) of the calls' tensors, the first being the one that the others have to join
CONV = dict(x=((1, 6, 8), BF), weight=((8, 4), F32), bias=((8,), F32))
SSM = dict(x=((1, 6, 8), BF), dt=((1, 6, 8), BF), A=((8, 4), F32), Bm=((1, 6, 1, 4), BF), Cm=((1, 6, 1, 4), BF))
NORM = dict(x=((6, 8), BF), post_weight=((8,), F32), gate=((6, 8), BF), scale=((8,), F32))
CALLS = {
    "conv_forward": dict(CONV, initial_state=((2, 3, 8), BF), cu_seqlens=((3,), I32)),
    "conv_backward": dict(CONV, dy=((1, 6, 8), BF), initial_state=((2, 3, 8), BF), dfinal_state=((2, 3, 8), BF), cu_seqlens=((3,), I32)),
    "conv_step": dict(x=((2, 8), BF), state=((3, 3, 8), BF), weight=((8, 4), F32), bias=((8,), F32), slots=((2,), I32)),
    "ssm_forward": dict(SSM, D=((8,), F32), dt_bias=((8,), F32), S0=((2, 8, 4), F32), cu_seqlens=((3,), I32)),
    "ssm_backward": dict(SSM, h_saved=((4 * 8 * 4,), F32), dy=((1, 6, 8), BF), D=((8,), F32), dt_bias=((8,), F32), dS_T=((2, 8, 4), F32),
                         cu_seqlens=((3,), I32)),
    "ssm_step": dict(x=((2, 8), BF), dt=((2, 8), BF), A=((8, 4), F32), Bm=((2, 1, 4), BF), Cm=((2, 1, 4), BF), state=((3, 8, 4), F32),
                     D=((8,), F32), dt_bias=((8,), F32), slots=((2,), I32)),
    "norm_forward": dict(NORM, residual=((6, 8), F32), pre_weight=((8,), F32)),
    "norm_backward": dict(NORM, r=((6, 8), F32), pre_weight=((8,), F32), dr=((6, 8), F32), dy=((6, 8), BF)),
    "step": dict(q=((2, 1, 16), BF), k=((2, 1, 16), BF), v=((2, 2, 16), BF), g=((2, 2), F32), beta=((2, 2), BF), state=((3, 2, 16, 16), F32),
                 slots=((2,), I32)),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, args in CALLS.items() for n in list(args)[1:]])
def test_a_tensor_on_another_device_is_refused(call, name):
    with FakeTensorMode():
        args = {n: torch.empty(shape, dtype=dtype, device="cuda:1" if n == name else "cuda:0") for n, (shape, dtype) in CALLS[call].items()}
        with pytest.raises(ValueError, match=f"^{name}: on cuda:1, the call's first tensor on cuda:0"):
            getattr(gdr, call)(**args)


@pytest.mark.parametrize("call", list(CALLS))
def test_a_stream_is_one_of_the_tensors_device(monkeypatch, call):
    """A handle is taken as a stream of the tensors' device, not of the current one; another device's stream is
    refused: the call would run on a stream that nobody named."""
    made = []

    def external(handle, device=None):
        made.append((handle, device))
        return types.SimpleNamespace(device=device)

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    wrong = list(CALLS[call])[1]  # so that the call ends before it allocates
    with FakeTensorMode():
        args = {n: torch.empty(shape, dtype=dtype, device="cpu" if n == wrong else "cuda:1") for n, (shape, dtype) in CALLS[call].items()}
        with pytest.raises(ValueError, match=wrong):
            getattr(gdr, call)(**args, stream=1 << 20)
        assert made == [(1 << 20, torch.device("cuda:1"))]
        with pytest.raises(ValueError, match="stream: of cuda:0, the call's first tensor on cuda:1"):
            getattr(gdr, call)(**args, stream=types.SimpleNamespace(device=torch.device("cuda:0")))
