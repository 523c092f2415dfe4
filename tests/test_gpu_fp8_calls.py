"""The fp8 calls on the GPU where one kernel's launch, its tiles and its neighbours meet: launches that take
seconds, tiles split between workers, lists that name wrong things, values that are not finite.

References are in 64 bits and the bounds those of fp8ref.py."""
import pytest
import torch

import fp8ref as R
from int4_routed_expert_gemv_b200 import binding as B

pytestmark = pytest.mark.gpu


def dense_ws(T, N, K):
    ws = torch.zeros(B.coli_fp8_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    B.check(B.coli_moe_workspace_init(ws))
    return ws


def test_matmul_of_several_seconds(colimoe):
    # 4.5 million K steps a pair and more than the 4e9 cycles after which a wait gives up; outputs of some rows and columns
    n = 147456
    g = torch.Generator("cuda").manual_seed(1)
    codes = torch.randint(0, 0x7F, (n, n), dtype=torch.uint8, device="cuda", generator=g)      # positive, finite
    xs = 0.5 + torch.rand(n, n // 128, device="cuda", generator=g)
    s = 2.0 ** -20 * (0.5 + torch.rand(n // 128, n // 128, device="cuda", generator=g))
    y = torch.empty(n, n, dtype=torch.bfloat16, device="cuda")
    ws = dense_ws(n, n, n)
    B.check(B.coli_fp8_matmul(n, n, n, codes, xs, codes, s, None, y, ws))
    assert B.coli_moe_read_status(ws) == (B.COLI_OK, 0)
    rows = torch.tensor([0, 255, 256, 70001, n - 1], device="cuda")
    cols = torch.tensor([0, 127, 128, 90003, n - 1], device="cuda")
    x = R.dequant(codes[rows].view(R.E4M3).cpu(), xs[rows].cpu())
    w = R.dequant(codes[cols].view(R.E4M3).cpu(), s[cols // 128].cpu())
    ref = x @ w.T
    bound = ref * R.product_bound(n // 128)      # all terms are positive
    bound = bound + (ref + bound) * 2.0 ** -8
    got = y[rows][:, cols].cpu().double()
    assert ((got - ref).abs() <= bound).all()
