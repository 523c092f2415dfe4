"""The fp8 calls without a GPU: sizes, refusals before anything is enqueued, and the host quantiser."""
import ctypes

import numpy as np
import pytest
import torch

from int4_routed_expert_gemv_b200 import binding as B
from int4_routed_expert_gemv_b200 import quantize as Q

P = ctypes.c_void_p
FAKE, MIS, BIG = P(0x10000), P(0x10004), 1 << 40     # never dereferenced on these paths


def test_sizes(colimoe):
    assert B.coli_moe_blob_bytes_fp8(6144, 2048) == 3 * 6144 * 2048 + 3 * 4 * 48 * 16
    assert B.coli_moe_blob_bytes_fp8(192, 320) == 3 * 192 * 320 + 3 * 4 * 2 * 3
    for bad in [(0, 64), (64, 0), (100, 64), (64, 32), (-64, 64)]:
        assert B.coli_moe_blob_bytes_fp8(*bad) == 0
    d = B.make_dims(6144, 2048, 256, 8, 1)
    assert 0 < B.coli_moe_workspace_bytes_fp8(d, 1) < B.coli_moe_workspace_bytes_fp8(d, 100)
    assert B.coli_moe_workspace_bytes_fp8(d, 0) > 0 and B.coli_moe_workspace_bytes_fp8(d, -1) == 0
    # a workspace for T_max tokens does for every smaller batch, on both sides of every kernel's range
    sizes = [B.coli_moe_workspace_bytes_fp8(d, T) for T in list(range(0, 40)) + [64, 255, 256, 257, 2048]]
    assert sizes == sorted(sizes)
    sizes = [B.coli_fp8_workspace_bytes(T, 576, 1024) for T in range(0, 300)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    for bad in [(-1, 8, 16), (1, 0, 16), (1, 8, 8), (1, 8, 24), (1, 8, 0)]:
        assert B.coli_fp8_workspace_bytes(*bad) == 0


def test_norm_refusals(colimoe):
    f = B.lib().coli_rmsnorm_fp8
    ok = dict(hidden=64, T=1, x=FAKE, residual=None, dtype=0, gamma=None, eps=1e-5, sum=None, out=None, q=FAKE, scales=FAKE)

    def call(**over):
        a = {**ok, **over}
        return f(a["hidden"], a["T"], a["x"], a["residual"], a["dtype"], a["gamma"], a["eps"], a["sum"], a["out"], a["q"],
                 a["scales"], None)

    assert call(T=0) == B.COLI_OK
    for bad in [dict(hidden=0), dict(hidden=24), dict(T=-1), dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(x=None), dict(q=None), dict(scales=None), dict(x=MIS), dict(q=MIS), dict(scales=MIS),
                dict(residual=MIS), dict(gamma=MIS), dict(sum=MIS), dict(out=MIS)]:
        assert call(**bad) == B.COLI_EINVAL, bad
    assert call(hidden=32784) == B.COLI_EUNSUPPORTED


def test_matmul_refusals(colimoe):
    f = B.lib().coli_fp8_matmul
    ok = dict(T=1, N=8, K=16, xq=FAKE, xs=FAKE, wq=FAKE, ws_=FAKE, residual=None, y=FAKE, dtype=0, ws=FAKE, bytes=BIG)

    def call(**over):
        a = {**ok, **over}
        return f(a["T"], a["N"], a["K"], a["xq"], a["xs"], a["wq"], a["ws_"], a["residual"], a["y"], a["dtype"], a["ws"],
                 a["bytes"], None)

    assert call(T=0) == B.COLI_OK
    for bad in [dict(T=-1), dict(N=0), dict(K=0), dict(K=20), dict(K=8), dict(dtype=-1), dict(dtype=5)] + \
               [{k: v} for k in ("xq", "xs", "wq", "ws_", "y", "ws") for v in (None, MIS)] + [dict(residual=MIS)]:
        assert call(**bad) == B.COLI_EINVAL, bad
    assert call(bytes=B.coli_fp8_workspace_bytes(1, 8, 16) - 1) == B.COLI_ENOMEM
    for big in [dict(T=(1 << 24) + 1), dict(N=(1 << 24) + 1), dict(K=(1 << 24) + 16)]:
        assert call(**big) == B.COLI_EUNSUPPORTED, big


@pytest.mark.parametrize("which", ["gate_up", "down", "forward"])
def test_experts_refusals(colimoe, which):
    L = B.lib()
    d = B.make_dims(192, 320, 8, 3, 1)
    stride = (B.coli_moe_blob_bytes_fp8(192, 320) + 255) // 256 * 256
    good = B.Weights(None, None, FAKE, FAKE, stride)
    ok = dict(dims=d, weights=good, a=FAKE, as_=FAKE, T=2, w=FAKE, ids=FAKE, n=FAKE, off=FAKE, asg=FAKE, residual=None,
              o1=FAKE, o2=FAKE, ws=FAKE, bytes=BIG)

    def call(**over):
        v = {**ok, **over}
        dims, wts = ctypes.byref(v["dims"]), None if v["weights"] is None else ctypes.byref(v["weights"])
        lists = (v["ids"], v["n"], v["off"], v["asg"])
        if which == "gate_up":
            return L.coli_moe_gate_up_fp8(dims, wts, v["a"], v["as_"], v["T"], *lists, v["o1"], v["o2"], v["ws"], v["bytes"],
                                          None)
        f = L.coli_moe_down_fp8 if which == "down" else L.coli_moe_forward_fp8
        return f(dims, wts, v["a"], v["as_"], v["T"], v["w"], *lists, v["residual"], v["o1"], v["ws"], v["bytes"], None)

    assert call(T=0) == B.COLI_OK
    bad = [dict(dims=B.make_dims(200, 320, 8, 3, 1)), dict(dims=B.make_dims(192, 320, 8, 9, 1)),
           dict(dims=B.make_dims(192, 320, 2000, 3, 1)), dict(T=-1), dict(weights=None),
           dict(weights=B.Weights(None, None, None, FAKE, stride)), dict(weights=B.Weights(None, None, FAKE, None, stride)),
           dict(weights=B.Weights(None, None, FAKE, FAKE, stride - 256)), dict(weights=B.Weights(None, None, FAKE, FAKE, stride + 16)),
           dict(weights=B.Weights(None, None, MIS, FAKE, stride)), dict(weights=B.Weights(None, None, FAKE, MIS, stride)),
           dict(a=None), dict(a=MIS), dict(as_=None), dict(as_=MIS), dict(ids=None), dict(n=None), dict(off=None),
           dict(asg=None), dict(o1=None), dict(o1=MIS), dict(ws=None), dict(ws=MIS)]
    bad += [dict(o2=None), dict(o2=MIS)] if which == "gate_up" else [dict(w=None), dict(residual=MIS)]
    for b in bad:
        assert call(**b) == B.COLI_EINVAL, b
    assert call(bytes=B.coli_moe_workspace_bytes_fp8(d, 2) - 1) == B.COLI_ENOMEM
    assert call(T=(1 << 24) + 1) == B.COLI_EUNSUPPORTED


def test_e4m3_codes_are_torchs():
    # every code's value, and every midpoint between neighbours (ties), and what lies around them
    v = Q.e4m3_values(np.arange(256, dtype=np.uint8))
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    pos = np.sort(v[:127].astype(np.float64))
    mid = (pos[1:] + pos[:-1]) / 2
    x = np.concatenate([pos, mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9)), [1e-30, 448.0, 0.0]]).astype(np.float32)
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(Q.e4m3_codes(x), want)
    assert Q.e4m3_codes(np.float32([500.0, -1e30, np.inf, np.nan])).tolist() == [0x7E, 0xFE, 0x7E, 0x7F]


@pytest.mark.parametrize("rows,cols", [(128, 128), (64, 192), (300, 130)])
def test_quantize_matrix_fp8(rows, cols):
    rng = np.random.default_rng(rows)
    W = rng.standard_normal((rows, cols)).astype(np.float32) * np.exp(rng.standard_normal((rows, 1))).astype(np.float32)
    W[:, :8] = 0
    q, s = Q.quantize_matrix_fp8(W)
    assert q.shape == (rows, cols) and s.shape == ((rows + 127) // 128, (cols + 127) // 128) and s.dtype == np.float32
    sc = np.repeat(np.repeat(s, 128, 0)[:rows], 128, 1)[:, :cols].astype(np.float64)
    off = np.abs(Q.dequantize_matrix_fp8(q, s).astype(np.float64) - W)
    # half a step of 4 significant bits (and the scale's and quotient's roundings), or of the subnormals
    assert (off <= np.abs(W) * 2.0 ** -4 * (1 + 2.0 ** -20) + sc * 2.0 ** -10).all()
    z, zs = Q.quantize_matrix_fp8(np.zeros((130, 64), np.float32))
    assert (z == 0).all() and (zs == 0).all()


def test_expert_blob_fp8(colimoe):
    H, I = 192, 64
    rng = np.random.default_rng(0)
    mats = [rng.standard_normal(s).astype(np.float32) for s in ((I, H), (I, H), (H, I))]
    blob, deq = Q.expert_blob_fp8(*mats)
    assert blob.dtype == np.uint8 and blob.size == B.coli_moe_blob_bytes_fp8(H, I)
    q, s = Q.quantize_matrix_fp8(mats[1])
    assert np.array_equal(blob[I * H:2 * I * H], q.reshape(-1))
    at = 3 * I * H + 4 * 1 * 2
    assert np.array_equal(blob[at:at + 8], s.reshape(-1).view(np.uint8))
    assert np.array_equal(deq[1], Q.dequantize_matrix_fp8(q, s))
