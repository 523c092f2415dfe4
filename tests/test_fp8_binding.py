"""Types of the fp8 calls' tensors in the Python binding (no GPU: the calls are refused, or have no tokens)."""
import types

import pytest
import torch

from int4_routed_expert_gemv_b200 import binding as B

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NO_STREAM = types.SimpleNamespace(cuda_stream=0)


def norm(x, residual, sum_):
    t = lambda d: None if d is None else torch.zeros(0, 64, dtype=d)      # noqa: E731
    return B.coli_rmsnorm_fp8(64, 0, t(x), t(residual), None, 1e-5, t(sum_), None, torch.zeros(0, 64, dtype=torch.uint8),
                              torch.zeros(0, 1), stream=NO_STREAM)


def matmul(y, residual):
    t = lambda d: None if d is None else torch.zeros(0, 8, dtype=d)       # noqa: E731
    u = torch.zeros(16, 16, dtype=torch.uint8)
    return B.coli_fp8_matmul(0, 8, 16, u, t(F32), u, t(F32), t(residual), t(y), u,
                             stream=NO_STREAM)


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
