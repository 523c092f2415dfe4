"""The fp8 calls (norm with 8-bit output, block-scaled product, the experts' two products) on the
GPU against 64-bit references, at the sizes where they can go wrong.

Bounds: a product is off by at most product_bound() times the sum of its terms' magnitudes
(derived in fp8ref.py), a rounding to bf16 by 2^-8 and to e4m3 by 2^-4 of the value (2^-10 of the
scale below the smallest normal code).
"""
import pytest
import torch

import fp8ref as R
from int4_routed_expert_gemv_b200 import binding as B

pytestmark = pytest.mark.gpu

NAN = float("nan")


def dense_ws(T, N, K):
    ws = torch.zeros(B.coli_fp8_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    B.check(B.coli_moe_workspace_init(ws))
    return ws


def run_matmul(T, N, K, dtype, residual, seed=0):
    g = torch.Generator().manual_seed(seed)
    xq, xs = R.activations(T, K, g)
    wq, s = R.weights(N, K, g)
    r = torch.randn(T, N, generator=g).to(dtype) if residual else None
    y = torch.full((T + 2, N), NAN, dtype=dtype, device="cuda")
    ws = dense_ws(T, N, K)
    B.check(B.coli_fp8_matmul(T, N, K, xq.cuda(), xs.cuda(), wq.cuda(), s.cuda(), None if r is None else r.cuda(), y, ws))
    assert B.coli_moe_read_status(ws) == (B.COLI_OK, 0)
    x, w = R.dequant(xq, xs), R.dequant_w(wq, s)
    ref, mag = x @ w.T, x.abs() @ w.abs().T
    if r is not None:
        ref, mag = ref + r.double(), mag + r.double().abs()
    got = y.cpu()
    assert torch.isnan(got[T:]).all(), "rows behind the last were written"
    bound = mag * R.product_bound(R.blocks(K), 1)
    if dtype == torch.bfloat16:
        bound = bound + (ref.abs() + bound) * 2.0 ** -8
    off = (got[:T].double() - ref).abs()
    worst = float((off / bound.clamp_min(1e-300)).max())
    assert worst <= 1, f"{worst:.2f} of the bound"
    return float(off.norm() / ref.norm())


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 64, 65, 77, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(1, 16), (64, 128), (129, 272), (576, 1024), (1000, 2064)])
def test_matmul_sizes(colimoe, T, N, K):
    rel = run_matmul(T, N, K, torch.float32, residual=(T + N) % 2 == 0)
    assert rel < 2e-5


@pytest.mark.parametrize("T,N,K,residual", [(1, 2048, 6144, False), (9, 300, 512, True), (200, 4096, 512, True),
                                            (1030, 640, 6144, False)])
def test_matmul_bf16(colimoe, T, N, K, residual):
    run_matmul(T, N, K, torch.bfloat16, residual)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", [(300, 5001, 640), (600, 4902, 400), (600, 5003, 272), (257, 5185, 16)])
@pytest.mark.parametrize("residual", [False, True])
def test_matmul_rows_of_any_length(colimoe, dtype, T, N, K, residual):
    # rows of y that do not begin on 16 bytes, of many tiles, whole and split, with many and with few K steps
    run_matmul(T, N, K, dtype, residual)


@pytest.mark.parametrize("T,N,K,residual", [(1382, 3081, 1776, True), (1382, 3081, 1776, False), (1382, 3080, 1776, True),
                                            (70, 12291, 640, True)])
def test_matmul_calls_in_a_row(colimoe, T, N, K, residual):
    # a warp with 6 rows of a tile, every tile split, one call behind the other
    g = torch.Generator().manual_seed(5)
    xq, xs = (t.cuda() for t in R.activations(T, K, g))
    wq, s = (t.cuda() for t in R.weights(N, K, g))
    r = torch.randn(T, N, generator=g).cuda() if residual else None
    ws = dense_ws(T, N, K)
    ys = [torch.empty(T, N, device="cuda") for _ in range(3)]
    for i in range(60):
        B.check(B.coli_fp8_matmul(T, N, K, xq, xs, wq, s, r, ys[i % 3], ws))
    assert B.coli_moe_read_status(ws) == (B.COLI_OK, 0)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_matmul_many_tiles(colimoe):
    # more tiles than CTAs, so whole tiles and split ones in one launch
    for T, N, K in [(1024, 6144, 256), (2049, 4100, 128)]:
        assert run_matmul(T, N, K, torch.float32, True) < 2e-5


def test_matmul_repeats_bitwise(colimoe):
    g = torch.Generator().manual_seed(3)
    for T, N, K in [(4, 1024, 6144), (130, 900, 4096)]:
        xq, xs = (t.cuda() for t in R.activations(T, K, g))
        wq, s = (t.cuda() for t in R.weights(N, K, g))
        ws = dense_ws(T, N, K)
        ys = []
        for _ in range(4):
            y = torch.empty(T, N, device="cuda")
            B.check(B.coli_fp8_matmul(T, N, K, xq, xs, wq, s, None, y, ws))
            ys.append(y)
        assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_matmul_more_than_32_bits_of_outputs(colimoe):
    # T * N passes 2^31: the last rows, and rows on both sides of the border
    T, N, K = 66000, 33000, 16
    g = torch.Generator().manual_seed(11)
    xq, xs = R.activations(T, K, g)
    wq, s = R.weights(N, K, g)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    B.check(B.coli_fp8_matmul(T, N, K, xq.cuda(), xs.cuda(), wq.cuda(), s.cuda(), None, y, dense_ws(T, N, K)))
    rows = torch.tensor([0, 65074, 65075, 65076, T - 1])
    x, w = R.dequant(xq[rows], xs[rows]), R.dequant_w(wq, s)
    ref, mag = x @ w.T, x.abs() @ w.abs().T
    bound = mag * R.product_bound(1) + (ref.abs() + mag * R.product_bound(1)) * 2.0 ** -8
    assert ((y[rows.cuda()].cpu().double() - ref).abs() <= bound).all()


def test_matmul_in_place_residual(colimoe):
    g = torch.Generator().manual_seed(4)
    for T, N, K in [(33, 257, 512), (5, 257, 512), (300, 5001, 640), (300, 5000, 640), (100, 257, 640)]:
        xq, xs = (t.cuda() for t in R.activations(T, K, g))
        wq, s = (t.cuda() for t in R.weights(N, K, g))
        ws = dense_ws(T, N, K)
        r = torch.randn(T, N, generator=g).cuda()
        y = torch.empty(T, N, device="cuda")
        B.check(B.coli_fp8_matmul(T, N, K, xq, xs, wq, s, r, y, ws))
        B.check(B.coli_fp8_matmul(T, N, K, xq, xs, wq, s, r, r, ws))
        assert torch.equal(r, y)


def test_matmul_non_finite_stays_in_its_row_and_column(colimoe):
    g = torch.Generator().manual_seed(5)
    for T, N, K in [(5, 300, 256), (150, 300, 256)]:
        xq, xs = R.activations(T, K, g)
        wq, s = R.weights(N, K, g)
        clean = torch.empty(T, N, device="cuda")
        y = torch.empty(T, N, device="cuda")
        ws = dense_ws(T, N, K)
        B.check(B.coli_fp8_matmul(T, N, K, xq.cuda(), xs.cuda(), wq.cuda(), s.cuda(), None, clean, ws))
        xq.view(torch.uint8)[3, 7] = 0x7F
        xs[4, 1] = float("inf")
        B.check(B.coli_fp8_matmul(T, N, K, xq.cuda(), xs.cuda(), wq.cuda(), s.cuda(), None, y, ws))
        keep = torch.ones(T, dtype=torch.bool)
        keep[[3, 4]] = False
        assert torch.equal(y.cpu()[keep], clean.cpu()[keep])
        assert torch.isnan(y[3]).all() and not torch.isfinite(y[4]).any()


# ------------------------------------------------------------------------------------------------
# norm
# ------------------------------------------------------------------------------------------------
def check_norm(x, r, gamma, eps, sum_, out, q, s):
    """Outputs (on the CPU) against the definition."""
    if r is not None:
        t = (x.float() + r.float()).to(x.dtype)
        if sum_ is not None:
            assert torch.equal(sum_, t)
    else:
        t = x
    d = t.double()
    gm = torch.ones(x.shape[1], dtype=torch.float64) if gamma is None else gamma.double()
    ref = d * gm / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    n = ref.float() if out is None else out
    assert ((n.double() - ref).abs() <= ref.abs() * R.U32 * (1 + 2.0 ** -16) + 1e-45).all()
    eq, es = R.quantize(n)
    if out is not None:
        assert torch.equal(s, es), "scales"
        assert torch.equal(q.view(torch.uint8), eq.view(torch.uint8)), "codes"
    else:      # n may be one rounding away from ref's
        assert ((s - es).abs() <= es * 4 * R.U32).all()
        assert ((R.dequant(q, s) - n.double()).abs() <= n.double().abs() * 2.0 ** -4 * (1 + 2.0 ** -20) +
                s.double().repeat_interleave(128, 1)[:, :n.shape[1]] * 2.0 ** -10).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(1, 16), (3, 64), (2, 144), (5, 576), (4, 6144), (2, 6160), (1, 12288), (1, 12304),
                                 (2, 32768)])
@pytest.mark.parametrize("residual,router", [(True, True), (False, False), (True, False)])
def test_norm(colimoe, dtype, T, H, residual, router):
    g = torch.Generator().manual_seed(T * H)
    x = (torch.randn(T, H, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))).to(dtype)
    r = torch.randn(T, H, generator=g).to(dtype) if residual else None
    gamma = 1 + 0.3 * torch.randn(H, generator=g) if T != 3 else None
    sm = torch.full((T + 1, H), NAN, dtype=dtype, device="cuda")
    out = torch.full((T + 1, H), NAN, device="cuda") if router else None
    q = torch.full((T + 1, H), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((T + 1, R.blocks(H)), NAN, device="cuda")
    B.check(B.coli_rmsnorm_fp8(H, T, x.cuda(), None if r is None else r.cuda(), None if gamma is None else gamma.cuda(),
                               1e-5, sm, out, q, s))
    torch.cuda.synchronize()
    assert torch.isnan(sm[T:]).all() and (q[T:] == 0x55).all() and torch.isnan(s[T:]).all()
    if r is None:
        assert torch.equal(sm[:T].cpu(), x)      # the sum of x alone is x
    check_norm(x, r, gamma, 1e-5, sm[:T].cpu() if residual else None, out[:T].cpu() if router else None,
               q[:T].cpu().view(R.E4M3), s[:T].cpu())


def test_norm_more_than_32_bits_of_elements(colimoe):
    T, H = 140000, 16384
    x = torch.randn(1000, H, device="cuda", dtype=torch.bfloat16, generator=torch.Generator("cuda").manual_seed(2))
    x = x.repeat(140, 1)
    x[T - 1] *= 3
    q = torch.empty(T, H, dtype=R.E4M3, device="cuda")
    s = torch.empty(T, H // 128, device="cuda")
    B.check(B.coli_rmsnorm_fp8(H, T, x, None, None, 1e-5, None, None, q, s))
    rows = torch.tensor([0, 131071, 131072, T - 1])
    check_norm(x[rows.cuda()].cpu(), None, None, 1e-5, None, None, q[rows.cuda()].cpu(), s[rows.cuda()].cpu())


@pytest.mark.parametrize("which", ["x", "residual"])
def test_norm_sum_in_place(colimoe, which):
    g = torch.Generator().manual_seed(9)
    x, r = torch.randn(7, 1040, generator=g).cuda(), torch.randn(7, 1040, generator=g).cuda()
    q, s = torch.empty(7, 1040, dtype=R.E4M3, device="cuda"), torch.empty(7, 9, device="cuda")
    want = x + r
    to = x if which == "x" else r
    B.check(B.coli_rmsnorm_fp8(1040, 7, x, r, None, 0.0, to, None, q, s))
    assert torch.equal(to, want)


def test_norm_zero_and_non_finite_rows(colimoe):
    H = 256
    x = torch.randn(6, H, generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1, :128] = 0                 # one block of zeros
    x[2, 5] = NAN
    x[3, 200] = float("inf")
    x[4] = 1e-42                   # denormals
    q, s = torch.empty(6, H, dtype=torch.uint8, device="cuda"), torch.empty(6, 2, device="cuda")
    out = torch.empty(6, H, device="cuda")
    B.check(B.coli_rmsnorm_fp8(H, 6, x.cuda(), None, None, 1e-6, None, out, q, s))
    q, s, out = q.cpu(), s.cpu(), out.cpu()
    assert (q[0] == 0).all() and (s[0] == 0).all() and (out[0] == 0).all()
    assert (q[1, :128] & 0x7F == 0).all() and s[1, 0] == 0 and (s[1, 1] > 0)
    assert torch.isnan(out[2]).all() and torch.isnan(s[2]).all() and ((q[2] & 0x7F) == 0x7F).all()
    # mean(x^2) is infinite: finite values go to 0, the infinite one to NaN, and so its block
    assert (out[3, :128] == 0).all() and s[3, 0] == 0 and torch.isnan(out[3, 200]) and torch.isnan(s[3, 1])
    assert (q[3, :128] & 0x7F == 0).all() and ((q[3, 128:] & 0x7F) == 0x7F).all()
    check_norm(x[4:], None, None, 1e-6, None, out[4:], q[4:].view(R.E4M3), s[4:])


def test_norm_codes_at_every_scale(colimoe):
    # 21 blocks whose values lie around 2^-149 .. 2^127, one of them with values far below its largest
    exps = [-149, -140, -126, -120, -101, -100, -99, -92, -91, -90, -89, -82, -10, 0, 82, 89, 98, 99, 100, 110, 125]
    H = 128 * len(exps)
    g = torch.Generator().manual_seed(3)
    gamma = torch.ldexp(torch.ones(H), torch.tensor(exps).repeat_interleave(128))
    x = torch.randn(4, H, generator=g)
    x[1] = x[1] * torch.exp(-4 * torch.rand(H, generator=g) ** 2 * 6)
    x[2, ::2] = 0
    x = x.clamp(-3.9, 3.9)
    q, s = torch.empty(4, H, dtype=torch.uint8, device="cuda"), torch.empty(4, len(exps), device="cuda")
    out = torch.empty(4, H, device="cuda")
    B.check(B.coli_rmsnorm_fp8(H, 4, x.cuda(), None, gamma.cuda(), 1e-6, None, out, q, s))
    n, s = out.cpu(), s.cpu()
    top = n.double().abs().view(4, -1, 128).amax(2) / 448
    assert torch.equal(s, top.float())
    want = torch.where(s[:, :, None] > 0, n.view(4, -1, 128).double() / s[:, :, None].double(), 0.0).float()
    want = want.clamp(-448, 448).view(4, H).to(R.E4M3).view(torch.uint8)
    same = (q.cpu() == want) | ((q.cpu() | want) & 0x7F == 0)
    assert same.all(), (~same).nonzero()[:8]


# ------------------------------------------------------------------------------------------------
# experts
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,H", [(16, 128), (60, 1024), (60, 128), (400, 128)])
def test_swiglu_over_its_range(colimoe, T, H):
    # one column of h: g = u = +-xs, so its scale is silu(g) * g / 448 with all of fp32
    I, E = 64, 4
    v = torch.cat([torch.linspace(-79, 200, T - 8), torch.tensor([0.0, 1e-30, -1e-30, 1e-3, -1e-3, 1e4, -1e4, -95.0])])
    x = torch.zeros(T, H, dtype=torch.uint8)
    x[:, 0] = torch.where(v < 0, 0xB8, 0x38).to(torch.uint8)               # e4m3 -1 and 1
    one = torch.zeros(I, H, dtype=torch.uint8)
    one[0, 0] = 0x38
    blob = torch.cat([one.reshape(-1), one.reshape(-1), torch.zeros(H * I, dtype=torch.uint8),
                      torch.ones(3 * R.blocks(H)).view(torch.uint8)])
    stride = (blob.numel() + 255) // 256 * 256
    experts = torch.zeros(E, stride, dtype=torch.uint8)
    experts[0, :blob.numel()] = blob
    experts = experts.cuda()
    dims, weights = B.make_dims(H, I, E, 1, 0), B.make_weights(None, None, experts, None, stride)
    lst = [t.cuda() for t in R.lists(torch.zeros(T, 1, dtype=torch.int32), E)]
    ws = torch.zeros(B.coli_moe_workspace_bytes_fp8(dims, T), dtype=torch.uint8, device="cuda")
    B.check(B.coli_moe_workspace_init(ws))
    hq, hs = torch.empty(T, I, dtype=torch.uint8, device="cuda"), torch.empty(T, 1, device="cuda")
    xs = v.abs()[:, None].repeat(1, R.blocks(H)).cuda()
    B.check(B.coli_moe_gate_up_fp8(dims, weights, x.cuda(), xs, T, *lst, hq, hs, ws))
    assert B.coli_moe_read_status(ws) == (B.COLI_OK, 0)
    g = v.double()
    h = g * torch.sigmoid(g) * g
    got = hs.cpu()[:, 0].double() * 448
    # beside silu_bound one rounding for the scale; below 2^-126 and at g = -95 the smallest normal number counts
    off = (got - h.abs()).abs()
    bound = h.abs() * (R.silu_bound(g) + R.U32) + 448 * 2.0 ** -126
    assert (off <= bound).all(), (float((off / bound).max()), float(v[(off / bound).argmax()]))


class Case:
    """A layer on the device with lists, outputs and a workspace."""

    def __init__(self, H, I, E, k, n_shared, T, seed=0, hot=False, e0=0, e1=None):
        self.L = L = R.make_layer(H, I, E, k, n_shared, seed)
        self.T = T
        g = torch.Generator().manual_seed(seed + 100)
        score = torch.rand(T, E, generator=g)
        if hot:                       # every token takes expert 0
            score[:, 0] = 2
        self.idx = score.topk(k, 1).indices.to(torch.int32)
        self.w = torch.softmax(torch.randn(T, k, generator=g), 1)
        self.xq, self.xs = R.activations(T, H, g)
        self.res = torch.randn(T, H, generator=g)
        e1 = E if e1 is None else e1
        self.lst = R.lists(self.idx, E, e0, e1)
        if e0 or e1 < E:
            L = self.L = R.Layer(H, I, e1 - e0, k, n_shared, L.mats[e0:e1] + L.mats[E:], L.blobs[e0:e1].contiguous(),
                                 L.shared, L.stride)
        self.dims = B.make_dims(H, I, L.E, min(k, L.E), n_shared)
        self.dims.top_k = k
        self.blobs, self.shared = L.blobs.cuda(), None if L.shared is None else L.shared.cuda()
        self.weights = B.make_weights(None, None, self.blobs, self.shared, L.stride)
        self.dl = [t.cuda() for t in self.lst]
        self.ws = torch.zeros(max(B.coli_moe_workspace_bytes_fp8(self.dims, T), 1), dtype=torch.uint8, device="cuda")
        B.check(B.coli_moe_workspace_init(self.ws))
        self.rows = T * (k + n_shared)
        self.hq = torch.full((self.rows + 1, I), 0x55, dtype=torch.uint8, device="cuda")
        self.hs = torch.full((self.rows + 1, R.blocks(I)), -7.0, device="cuda")
        self.y = torch.full((T + 1, H), NAN, device="cuda")

    def gate_up(self):
        B.check(B.coli_moe_gate_up_fp8(self.dims, self.weights, self.xq.cuda(), self.xs.cuda(), self.T, *self.dl, self.hq,
                                       self.hs, self.ws))
        assert B.coli_moe_read_status(self.ws) == (B.COLI_OK, 0)
        return self.hq.cpu(), self.hs.cpu()

    def check_gate_up(self):
        hq, hs = self.gate_up()
        h, err, named = R.gate_up(self.L, self.xq, self.xs, self.lst)
        n = self.rows
        left = torch.ones(n + 1, dtype=torch.bool)
        left[:n] = ~named
        assert (hq[left] == 0x55).all() and (hs[left] == -7.0).all(), "rows outside the lists were written"
        q, s = hq[:n][named].view(R.E4M3), hs[:n][named]
        h, err = h[named], err[named]
        pad = torch.zeros(h.shape[0], R.blocks(self.L.I) * 128, dtype=torch.float64)
        pad[:, :self.L.I] = h.abs()
        top = pad.view(h.shape[0], -1, 128).amax(2)
        pad[:, :self.L.I] = err
        terr = pad.view(h.shape[0], -1, 128).amax(2)
        assert ((s.double() - top / 448).abs() <= terr / 448 + top / 448 * 2 * R.U32).all(), "scales"
        sd = s.double().repeat_interleave(128, 1)[:, :self.L.I]
        bound = err + (h.abs() + err) * 2.0 ** -4 * (1 + 2.0 ** -20) + sd * 2.0 ** -10
        off = (R.dequant(q, s) - h).abs()
        assert (off <= bound).all(), float((off / bound).max())
        assert float(off.norm() / h.norm()) < 2.0 ** -5, "no better than a code's last bit"

    def check_down(self, residual=True, in_place=False):
        g = torch.Generator().manual_seed(77)
        hq, hs = R.activations(self.rows, self.L.I, g)
        named = torch.zeros(self.rows, dtype=torch.bool)
        for _, at, _ in R.groups(self.L, self.lst, self.T):
            named[at] = True
        hq.view(torch.uint8)[~named] = 0x7F          # rows that the lists leave out are not read
        res = self.res if residual else None
        y = self.y
        rd = None if res is None else res.cuda()
        if in_place:
            y = rd
        B.check(B.coli_moe_down_fp8(self.dims, self.weights, hq.cuda(), hs.cuda(), self.T, self.w.cuda(), *self.dl, rd, y,
                                    self.ws))
        assert B.coli_moe_read_status(self.ws) == (B.COLI_OK, 0)
        ref, bound = R.down(self.L, hq, hs, self.w, self.lst, res)
        got = y.cpu()
        if not in_place:
            assert torch.isnan(got[self.T:]).all()
        off = (got[:self.T].double() - ref).abs()
        assert (off <= bound).all(), float((off / bound.clamp_min(1e-300)).max())


LAYERS = [
    # H, I, E, k, n_shared
    (64, 64, 4, 1, 0),
    (192, 320, 8, 3, 1),
    (1024, 512, 16, 4, 1),
    (640, 128, 5, 5, 1),
]


@pytest.mark.parametrize("H,I,E,k,ns", LAYERS)
@pytest.mark.parametrize("T", [1, 4, 16, 17, 70, 200])
def test_gate_up(colimoe, H, I, E, k, ns, T):
    Case(H, I, E, k, ns, T, seed=T, hot=T % 2 == 0).check_gate_up()


@pytest.mark.parametrize("H,I,E,k,ns", LAYERS)
@pytest.mark.parametrize("T", [1, 4, 16, 17, 70, 200])
def test_down(colimoe, H, I, E, k, ns, T):
    Case(H, I, E, k, ns, T, seed=T, hot=T % 2 == 0).check_down(residual=T % 3 != 0)


@pytest.mark.parametrize("T", [17, 70, 150])
@pytest.mark.parametrize("hot", [False, True])
@pytest.mark.parametrize("I", [64, 320])
def test_batches_in_between(colimoe, T, hot, I):
    # few rows an expert on the average, and one expert with all tokens; odd sizes of K and of the last row block
    c = Case(1088, I, 16, 2, 1, T, seed=T, hot=hot)
    c.check_gate_up()
    c.check_down()


@pytest.mark.parametrize("T", [100, 330])
def test_many_rows_of_few_experts(colimoe, T):
    # every kernel that a batch of experts can take: few rows per expert, some, many
    for E in (3, 24):
        c = Case(192, 320, E, 2, 1, T, seed=E)
        c.check_gate_up()
        c.check_down()


def test_glm_shape(colimoe):
    for T in (1, 3):
        c = Case(6144, 2048, 10, 8, 1, T, seed=2)
        c.check_gate_up()
        c.check_down(in_place=T == 3)


@pytest.mark.parametrize("T", [5, 40])
def test_lists_that_leave_out(colimoe, T):
    # one rank's share: experts 2 .. 4 of 6; some tokens have none of them, some slots are left out
    c = Case(256, 192, 6, 2, 1, T, seed=6, e0=2, e1=5)
    assert int(c.lst[2][-1]) < T * 2
    c.check_gate_up()
    c.check_down()
    # lists without an expert, with and without the shared one
    for ns in (0, 1):
        c = Case(256, 192, 6, 2, ns, T, seed=6)
        c.lst = (torch.full((6,), -1, dtype=torch.int32), torch.tensor([0], dtype=torch.int32),
                 torch.zeros(7, dtype=torch.int32), c.lst[3])
        c.dl = [t.cuda() for t in c.lst]
        c.check_down()
        if ns:
            c.check_gate_up()


def test_bad_lists_are_flagged_and_not_followed(colimoe):
    for T in (3, 40):
        c = Case(256, 192, 6, 2, 1, T, seed=8)
        union, n, off, asg = [t.clone() for t in c.lst]
        for bad in ("expert", "offset", "assign", "count"):
            u, m, o, a = union.clone(), n.clone(), off.clone(), asg.clone()
            if bad == "expert":
                u[0] = 1 << 20
            elif bad == "offset":
                o[1] = 1 << 20
            elif bad == "assign":
                a[0] = -5
                a[1] = 1 << 30
            else:
                m[0] = 1 << 20
            B.check(B.coli_moe_workspace_init(c.ws))
            lst = [t.cuda() for t in (u, m, o, a)]
            hq, hs = R.activations(c.rows, 192, torch.Generator().manual_seed(1))
            B.check(B.coli_moe_gate_up_fp8(c.dims, c.weights, c.xq.cuda(), c.xs.cuda(), T, *lst, c.hq, c.hs, c.ws))
            st = B.coli_moe_read_status(c.ws)
            assert st == (B.COLI_EDEVICE, B.DEV_BAD_INDEX), (bad, st)
            B.check(B.coli_moe_workspace_init(c.ws))
            B.check(B.coli_moe_down_fp8(c.dims, c.weights, hq.cuda(), hs.cuda(), T, c.w.cuda(), *lst, None, c.y, c.ws))
            st = B.coli_moe_read_status(c.ws)
            assert st == (B.COLI_EDEVICE, B.DEV_BAD_INDEX), (bad, st)


def test_a_token_twice_in_a_list(colimoe):
    # up to 16 tokens it is flagged (coli_moe_union flags the routing already); above, every position counts
    for T in (3, 40):
        c = Case(256, 192, 6, 2, 1, T, seed=8)
        c.idx[1] = c.idx[1, 0]
        c.lst = R.lists(c.idx, 6)
        c.dl = [t.cuda() for t in c.lst]
        if T > 16:
            c.check_gate_up()
            c.check_down()
            continue
        hq, hs = R.activations(c.rows, 192, torch.Generator().manual_seed(1))
        for call in (lambda: B.coli_moe_gate_up_fp8(c.dims, c.weights, c.xq.cuda(), c.xs.cuda(), T, *c.dl, c.hq, c.hs, c.ws),
                     lambda: B.coli_moe_down_fp8(c.dims, c.weights, hq.cuda(), hs.cuda(), T, c.w.cuda(), *c.dl, None, c.y,
                                                 c.ws)):
            B.check(B.coli_moe_workspace_init(c.ws))
            B.check(call())
            assert B.coli_moe_read_status(c.ws) == (B.COLI_EDEVICE, B.DEV_BAD_INDEX)


@pytest.mark.parametrize("T", [3, 40, 150])
def test_two_graphs_share_a_workspace(colimoe, T):
    # replayed in turn on one stream: one's counters and parts are done with when the other begins
    c = Case(512, 256, 6, 2, 1, T, seed=9)
    g = torch.Generator().manual_seed(10)
    hq, hs = (t.cuda() for t in R.activations(c.rows, 256, g))
    w, res, xq, xs = c.w.cuda(), c.res.cuda(), c.xq.cuda(), c.xs.cuda()

    def up():
        B.check(B.coli_moe_gate_up_fp8(c.dims, c.weights, xq, xs, T, *c.dl, c.hq, c.hs, c.ws))

    def down():
        B.check(B.coli_moe_down_fp8(c.dims, c.weights, hq, hs, T, w, *c.dl, res, c.y, c.ws))

    up()
    down()
    want = c.hq.clone(), c.hs.clone(), c.y.clone()
    graphs = []
    for f in (up, down):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for _ in range(3):
        c.hq[:c.rows] = 0
        c.hs[:c.rows] = 0
        c.y[:T] = 0
        graphs[0].replay()
        graphs[1].replay()
        assert torch.equal(c.hq, want[0]) and torch.equal(c.hs, want[1]) and torch.equal(c.y[:T], want[2][:T])
    assert B.coli_moe_read_status(c.ws) == (B.COLI_OK, 0)


# ------------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 6, 90])
def test_norm_route_experts_together(colimoe, T):
    """A residual layer as a program runs it: norm (sum, n, codes) -> route and union on n -> experts -> y = sum + MoE."""
    H, I, E, k = 256, 192, 12, 3
    L = R.make_layer(H, I, E, k, 1, 21)
    g = torch.Generator().manual_seed(22)
    x, r = torch.randn(T, H, generator=g).cuda(), torch.randn(T, H, generator=g).cuda()
    wr = (torch.randn(E, H, generator=g) * 0.1).cuda()
    gamma = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    dims = B.make_dims(H, I, E, k, 1)
    blobs, shared = L.blobs.cuda(), L.shared.cuda()
    weights = B.make_weights(wr, None, blobs, shared, L.stride)
    b = B.LayerBuffers(dims, T)
    ws = torch.zeros(B.coli_moe_workspace_bytes_fp8(dims, T), dtype=torch.uint8, device="cuda")
    B.check(B.coli_moe_workspace_init(ws))
    sm, n = torch.empty_like(x), torch.empty_like(x)
    q, s = torch.empty(T, H, dtype=R.E4M3, device="cuda"), torch.empty(T, 2, device="cuda")
    y = torch.empty_like(x)

    def step():
        B.check(B.coli_rmsnorm_fp8(H, T, x, r, gamma, 1e-6, sm, n, q, s))
        B.check(B.coli_moe_route_union(dims, wr, None, n, T, b.idx, b.w, None, b.union_ids, b.n_union, b.offsets, b.assign,
                                       b.ws))
        B.check(B.coli_moe_forward_fp8(dims, weights, q, s, T, b.w, b.union_ids, b.n_union, b.offsets, b.assign, sm, y, ws))

    step()
    assert B.coli_moe_read_status(ws) == (B.COLI_OK, 0) and B.coli_moe_read_status(b.ws) == (B.COLI_OK, 0)
    # the halves called one by one give the same bits
    hq = torch.empty(T * (k + 1), I, dtype=R.E4M3, device="cuda")
    hs = torch.empty(T * (k + 1), R.blocks(I), device="cuda")
    y2 = torch.empty_like(y)
    lst = (b.union_ids, b.n_union, b.offsets, b.assign)
    B.check(B.coli_moe_gate_up_fp8(dims, weights, q, s, T, *lst, hq, hs, ws))
    B.check(B.coli_moe_down_fp8(dims, weights, hq, hs, T, b.w, *lst, sm, y2, ws))
    assert torch.equal(y, y2)
    # against 64 bits, from the codes that the calls made
    lh = tuple(t.cpu() for t in lst)
    lh = (lh[0], lh[1][:1], lh[2], lh[3])
    ref, bound = R.down(L, hq.cpu(), hs.cpu(), b.w[:T].cpu(), lh, sm.cpu())
    assert ((y.cpu().double() - ref).abs() <= bound).all()
    # captured once and replayed on new inputs
    graph = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for seed in (30, 31):
        x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        got = y.clone()
        step()
        assert torch.equal(got, y)


def test_quantised_layer_is_near_the_layer(colimoe):
    """fp32 expert weights through the host quantiser, and the experts on the quantised rows of a norm: within the
    codes' precision of the fp32 layer (each product's terms are off by 2^-4 at most on either side, and h's codes
    by 2^-4 again; independent errors of a sum of many terms come out far below their sum)."""
    import numpy as np
    from int4_routed_expert_gemv_b200 import quantize as Q
    H, I, E, k, T = 256, 192, 6, 2, 20
    rng = np.random.default_rng(5)
    mats = [[rng.standard_normal(s).astype(np.float32) / s[1] ** 0.5 for s in ((I, H), (I, H), (H, I))] for _ in range(E)]
    stride = (B.coli_moe_blob_bytes_fp8(H, I) + 255) // 256 * 256
    blobs = torch.zeros(E, stride, dtype=torch.uint8)
    for e in range(E):
        b, _ = Q.expert_blob_fp8(*mats[e])
        blobs[e, :b.size] = torch.from_numpy(b)
    idx = torch.from_numpy(rng.permuted(np.tile(np.arange(E), (T, 1)), axis=1)[:, :k].astype(np.int32))
    w = torch.softmax(torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)), 1)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
    dims = B.make_dims(H, I, E, k, 0)
    dev = blobs.cuda()
    weights = B.make_weights(None, None, dev, None, stride)
    ws = torch.zeros(B.coli_moe_workspace_bytes_fp8(dims, T), dtype=torch.uint8, device="cuda")
    B.check(B.coli_moe_workspace_init(ws))
    n, q, s = torch.empty_like(x), torch.empty(T, H, dtype=R.E4M3, device="cuda"), torch.empty(T, 2, device="cuda")
    y = torch.empty_like(x)
    B.check(B.coli_rmsnorm_fp8(H, T, x, None, None, 1e-6, None, n, q, s))
    B.check(B.coli_moe_forward_fp8(dims, weights, q, s, T, w.cuda(), *[t.cuda() for t in R.lists(idx, E)], None, y, ws))
    nn = n.cpu().double().numpy()
    ref = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            G, U, D = (m.astype(np.float64) for m in mats[int(idx[t, j])])
            g = G @ nn[t]
            ref[t] += float(w[t, j]) * (D @ (g / (1 + np.exp(-g)) * (U @ nn[t])))
    assert np.linalg.norm(y.cpu().double().numpy() - ref) < 2.0 ** -3 * np.linalg.norm(ref)


def test_other_streams(colimoe):
    # calls on two streams with a workspace each
    g = torch.Generator().manual_seed(40)
    T, N, K = 20, 700, 1024
    sets = []
    for _ in range(2):
        xq, xs = (t.cuda() for t in R.activations(T, K, g))
        wq, s = (t.cuda() for t in R.weights(N, K, g))
        sets.append((xq, xs, wq, s, torch.empty(T, N, device="cuda"), dense_ws(T, N, K), torch.cuda.Stream()))
    want = []
    for xq, xs, wq, s, y, ws, _ in sets:
        B.check(B.coli_fp8_matmul(T, N, K, xq, xs, wq, s, None, y, ws))
        want.append(y.clone())
        y.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for xq, xs, wq, s, y, ws, st in sets:
            B.check(B.coli_fp8_matmul(T, N, K, xq, xs, wq, s, None, y, ws, stream=st))
    torch.cuda.synchronize()
    for w, (_, _, _, _, y, _, _) in zip(want, sets):
        assert torch.equal(w, y)
