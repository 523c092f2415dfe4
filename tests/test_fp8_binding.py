"""Types and devices of the fp8 calls' tensors in the Python binding.  No GPU: the calls are refused, or have no tokens,
and tensors of a device are stand-ins."""
import types

import pytest
import torch

from int4_routed_expert_gemv_b200 import binding as B

F32, BF16, F16, U8 = torch.float32, torch.bfloat16, torch.float16, torch.uint8
STREAM = types.SimpleNamespace(cuda_stream=0, device_index=3)


def tensor(dtype, device=3):
    if dtype is None:
        return None
    return types.SimpleNamespace(dtype=dtype, device=f"cuda:{device}", get_device=lambda: device, data_ptr=lambda: 1 << 16,
                                 numel=lambda: 1 << 30)


def norm(x, residual=None, sum_=None, device=3, stream=STREAM):
    return B.coli_rmsnorm_fp8(64, 0, tensor(x, device), tensor(residual), None, 1e-5, tensor(sum_), None, tensor(U8),
                              tensor(F32), stream=stream)


def matmul(y, residual=None, device=3, stream=STREAM):
    u, s = tensor(U8), tensor(F32)
    return B.coli_fp8_matmul(0, 8, 16, u, s, u, s, tensor(residual), tensor(y, device), u, stream=stream)


def experts(which, device=3, stream=STREAM):
    d, w = B.make_dims(64, 64, 4, 2, 0), B.Weights(None, None, 1 << 16, None, 1 << 20)
    u, s, i, to = tensor(U8), tensor(F32), tensor(torch.int32), tensor(F32, device)
    if which == "gate_up":
        return B.coli_moe_gate_up_fp8(d, w, u, s, 0, i, i, i, i, to, s, u, stream=stream)
    f = B.coli_moe_down_fp8 if which == "down" else B.coli_moe_forward_fp8
    return f(d, w, u, s, 0, s, i, i, i, i, None, to, u, stream=stream)


CALLS = [lambda **k: norm(F32, **k), lambda **k: matmul(BF16, **k)]
CALLS += [lambda w=w, **k: experts(w, **k) for w in ("gate_up", "down", "forward")]


def test_one_type_for_the_stream(colimoe):
    for a, b in [(F32, BF16), (BF16, F32), (F32, F16)]:
        for args in [(a, b, None), (a, None, b), (a, a, b), (a, b, b)]:
            with pytest.raises(TypeError):
                norm(*args)
        with pytest.raises(TypeError):
            matmul(a, b)
    for a in (F32, BF16):
        assert norm(a, a, a) == norm(a, None, None) == norm(a, a, None) == B.COLI_OK
        assert matmul(a, a) == matmul(a, None) == B.COLI_OK
    with pytest.raises(TypeError):
        matmul(F16, None)


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_another_device(colimoe, monkeypatch, call):
    assert call() == B.COLI_OK
    with pytest.raises(ValueError):
        call(device=2)               # another device than the stream's
    with pytest.raises(ValueError):
        call(device=-1)              # no device
    # without a stream, the current device's counts
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    assert call(stream=None) == B.COLI_OK
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError):
        call(stream=None)


def test_tensors_of_the_cpu(colimoe):
    x, q, s = torch.zeros(1, 64), torch.zeros(1, 64, dtype=U8), torch.zeros(1, 1)
    with pytest.raises(ValueError):
        B.coli_rmsnorm_fp8(64, 1, x, None, None, 1e-5, None, None, q, s)
