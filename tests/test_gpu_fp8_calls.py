"""The fp8 calls on the GPU where one kernel's launch, its tiles and its neighbours meet: launches that take
seconds, tiles split between workers, lists that name wrong things, values that are not finite.

References are in 64 bits and the bounds those of fp8ref.py."""
import pytest
import torch

import fp8ref as R
import test_gpu_fp8 as F
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
    del codes, y
    torch.cuda.empty_cache()
    assert ((got - ref).abs() <= bound).all()


def device_inputs(T, N, K, dtype, residual, seed):
    g = torch.Generator().manual_seed(seed)
    xq, xs = R.activations(T, K, g)
    wq, s = R.weights(N, K, g)
    r = torch.randn(T, N, generator=g).to(dtype) if residual else None
    return [None if t is None else t.cuda() for t in (xq, xs, wq, s, r)]


def check_matmul(y, xq, xs, wq, s, r):
    """y [T][N] against 64 bits, on the device."""
    x, w = (q.double() * t.double().repeat_interleave(128, 1)[:, :q.shape[1]]
            for q, t in ((xq, xs), (wq, s.repeat_interleave(128, 0)[:wq.shape[0]])))
    ref, mag = x @ w.T, x.abs() @ w.abs().T
    if r is not None:
        ref, mag = ref + r.double(), mag + r.double().abs()
    bound = mag * R.product_bound(R.blocks(xq.shape[1]), 1)
    if y.dtype == torch.bfloat16:
        bound = bound + (ref.abs() + bound) * 2.0 ** -8
    off = (y.double() - ref).abs()
    assert (off <= bound).all(), float((off / bound.clamp_min(1e-300)).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", [(4096, 6144, 2048), (3001, 5128, 1168)])
def test_matmul_several_tiles_a_pair(colimoe, dtype, T, N, K):
    # five whole tiles a pair and more, onto a residual (whose copies are asked for while a tile's sums are formed) and alone
    for residual in (True, False):
        xq, xs, wq, s, r = device_inputs(T, N, K, dtype, residual, T)
        y = torch.full((T + 1, N), float("nan"), dtype=dtype, device="cuda")
        ws = dense_ws(T, N, K)
        B.check(B.coli_fp8_matmul(T, N, K, xq, xs, wq, s, r, y, ws))
        assert B.coli_moe_read_status(ws) == (B.COLI_OK, 0)
        assert torch.isnan(y[T]).all()
        check_matmul(y[:T], xq, xs, wq, s, r)


def test_matmul_repeats_over_many_tiles(colimoe):
    # 21 tiles a pair and operands that do not stay in L2: a tile that a step does not wait for is missing now and then
    T, N, K = 16384, 6144, 2048
    xq, xs, wq, s, r = device_inputs(T, N, K, torch.float32, True, 1)
    ws = dense_ws(T, N, K)
    want, y = (torch.empty(T, N, device="cuda") for _ in range(2))
    B.check(B.coli_fp8_matmul(T, N, K, xq, xs, wq, s, r, want, ws))
    check_matmul(want[-600:], xq[-600:], xs[-600:], wq, s, r[-600:])
    differ = []
    for i in range(60):
        y.fill_(float("nan"))
        B.check(B.coli_fp8_matmul(T, N, K, xq, xs, wq, s, r, y, ws))
        differ.append((y != want).sum())
    assert [int(d) for d in differ] == [0] * 60
    assert B.coli_moe_read_status(ws) == (B.COLI_OK, 0)


@pytest.mark.parametrize("T,H,E", [(3, 1024, 8), (40, 1088, 16), (150, 512, 4), (600, 1024, 6)])
def test_other_inputs_call_after_call(colimoe, T, H, E):
    # norm and experts on two batches in turn, through the same buffers and workspace and with nothing in between: what
    # one kernel writes the next, which begins before it ends, has to read
    c = F.Case(H, 320, E, 2, 1, T, seed=T)
    g = torch.Generator().manual_seed(3)
    xs = [torch.randn(T, H, generator=g).cuda() * m for m in (1, 40)]
    q, s = torch.empty(T, H, dtype=R.E4M3, device="cuda"), torch.empty(T, R.blocks(H), device="cuda")
    wq, wsc = (t.cuda() for t in R.weights(264, H, g))
    y, z = torch.empty(T, H, device="cuda"), torch.empty(T, 264, device="cuda")
    gammas = [torch.randn(H, generator=g).cuda() for _ in range(2)]
    w, zws = c.w.cuda(), dense_ws(T, 264, H)

    def step(j):
        B.check(B.coli_rmsnorm_fp8(H, T, xs[j], None, gammas[j], 1e-6, None, None, q, s))
        B.check(B.coli_moe_gate_up_fp8(c.dims, c.weights, q, s, T, *c.dl, c.hq, c.hs, c.ws))
        B.check(B.coli_moe_forward_fp8(c.dims, c.weights, q, s, T, w, *c.dl, xs[j], y, c.ws))
        B.check(B.coli_fp8_matmul(T, 264, H, q, s, wq, wsc, None, z, zws))

    want = []
    for j in range(2):
        step(j)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (c.hq, c.hs, y, z)])
    for i in range(40):
        step(i % 2)
        step((i + 1) % 2)
        for a, b in zip((c.hq, c.hs, y, z), want[(i + 1) % 2]):
            assert torch.equal(a, b)
    # the two batches' products one behind the other, without the norm
    qs = []
    for j in range(2):
        B.check(B.coli_rmsnorm_fp8(H, T, xs[j], None, gammas[j], 1e-6, None, None, q, s))
        qs.append((q.clone(), s.clone()))
    outs = [(torch.full_like(c.hq, 0x55), torch.full_like(c.hs, -7.0)) for _ in range(20)]
    for i, (hq, hs) in enumerate(outs):
        B.check(B.coli_moe_gate_up_fp8(c.dims, c.weights, *qs[i % 2], T, *c.dl, hq, hs, c.ws))
    for i, (hq, hs) in enumerate(outs):
        assert torch.equal(hq, want[i % 2][0]) and torch.equal(hs, want[i % 2][1])
    assert B.coli_moe_read_status(c.ws) == (B.COLI_OK, 0)


@pytest.mark.parametrize("T", [4, 40, 300])
def test_a_gate_that_overflows(colimoe, T):
    # every kernel: silu(+inf) * u is an infinity of u's sign, which takes its block's scale with it and no other value
    H, I, E = 1024, 192, 4
    G = torch.zeros(I, H, dtype=torch.uint8)
    U = torch.zeros(I, H, dtype=torch.uint8)
    G[0, 0], G[1, 0], G[130, 0] = 0x7E, 0x01, 0x7E             # 448, 2^-9, 448
    U[0, 0], U[1, 0], U[130, 0] = 0x38, 0x38, 0x38             # 1
    U[0, 1] = 0xFE                                             # -448
    sc = [torch.ones(2, 8), torch.ones(2, 8), torch.ones(8, 2)]
    sc[0][0], sc[0][1] = 1e38, 2.0 ** -20
    sc[1][:] = 2.0 ** -20
    blob = torch.cat([G.reshape(-1), U.reshape(-1), torch.zeros(H * I, dtype=torch.uint8)] +
                     [t.reshape(-1).view(torch.uint8) for t in sc])
    stride = (blob.numel() + 255) // 256 * 256
    experts = torch.zeros(E, stride, dtype=torch.uint8)
    experts[0, :blob.numel()] = blob
    experts = experts.cuda()
    dims, weights = B.make_dims(H, I, E, 1, 0), B.make_weights(None, None, experts, None, stride)
    lst = [t.cuda() for t in R.lists(torch.zeros(T, 1, dtype=torch.int32), E)]
    ws = torch.zeros(B.coli_moe_workspace_bytes_fp8(dims, T), dtype=torch.uint8, device="cuda")
    B.check(B.coli_moe_workspace_init(ws))
    x = torch.zeros(T, H, dtype=torch.uint8)
    x[:, 0] = 0x7E
    x[2, 1] = 0x7E                                             # u of row 0 negative
    x[3, 0] = 0x7F                                             # a NaN of its own
    xs = torch.ones(T, 8)
    xs[1] = xs[4:] = 2.0 ** -60                                # these gates stay finite
    hq, hs = torch.full((T, I), 0x55, dtype=torch.uint8, device="cuda"), torch.empty(T, 2, device="cuda")
    B.check(B.coli_moe_gate_up_fp8(dims, weights, x.cuda(), xs.cuda(), T, *lst, hq, hs, ws))
    assert B.coli_moe_read_status(ws) == (B.COLI_OK, 0)
    hq, hs = hq.cpu(), hs.cpu()
    inf = float("inf")
    for t in (0, 2):
        assert hs[t, 0] == inf and hq[t, 0] & 0x7F == 0x7F, t
        assert (hq[t, 1:128] & 0x7F == 0).all(), t
    g, u = 448 * 448 * 2.0 ** -20, 448 * 2.0 ** -20            # the second block of token 0
    h = g / (1 + 2.718281828459045 ** -g) * u
    assert abs(float(hs[0, 1]) * 448 - h) <= h * 20 * R.U32 and hq[0, 130] == 0x7E
    assert torch.isnan(hs[3, 0]) and (hq[3, :128] & 0x7F == 0x7F).all()
    for t in [1] + list(range(4, T)):
        h = 448 * 448 * 1e38 * 2.0 ** -60 * (448 * 2.0 ** -80)
        assert abs(float(hs[t, 0]) * 448 - h) <= h * 20 * R.U32 and hq[t, 0] == 0x7E, t


# ------------------------------------------------------------------------------------------------
# lists
# ------------------------------------------------------------------------------------------------
def taken(c, lst):
    """What the calls take of any lists: (matrices, rows, positions) of each list that lies within the batch, and of
    those the positions that are the batch's; the shared expert last."""
    union, n, off, asg = (t.tolist() for t in lst)
    P, out = c.T * c.L.k, []
    for u in range(min(max(n[0], 0), c.L.E)):
        if 0 <= union[u] < c.L.E and 0 <= off[u] <= off[u + 1] <= P:
            at = [p for p in range(off[u], off[u + 1]) if 0 <= asg[p] < P]
            out.append((c.L.mats[union[u]], torch.tensor(at, dtype=torch.long),
                        torch.tensor([asg[p] for p in at], dtype=torch.long)))
    if c.L.n_shared:
        out.append((c.L.mats[c.L.E], torch.arange(P, P + c.T), None))
    return out


def check_lists(c, lst, monkeypatch, status, zeros=()):
    """Both products over any lists, against 64 bits.  zeros: positions whose row of h may be zeros."""
    with monkeypatch.context() as m:
        m.setattr(R, "groups", lambda L, l, T: taken(c, lst))
        dl = [t.cuda() for t in lst]
        n, I = c.rows, c.L.I
        # another batch first: nothing of it may be left in what the next call reads
        B.check(B.coli_moe_gate_up_fp8(c.dims, c.weights, c.xq.flip(0).cuda(), (c.xs * 3).cuda(), c.T, *c.dl, c.hq, c.hs,
                                       c.ws))
        B.check(B.coli_moe_workspace_init(c.ws))
        c.hq.fill_(0x55)
        c.hs.fill_(-7.0)
        B.check(B.coli_moe_gate_up_fp8(c.dims, c.weights, c.xq.cuda(), c.xs.cuda(), c.T, *dl, c.hq, c.hs, c.ws))
        assert B.coli_moe_read_status(c.ws) == status
        hq, hs = c.hq.cpu(), c.hs.cpu()
        h, err, named = R.gate_up(c.L, c.xq, c.xs, lst)
        left = torch.cat([~named, torch.ones(1, dtype=torch.bool)])
        for p in zeros:
            assert not named[p]
            assert (hq[p] == 0x55).all() and (hs[p] == -7).all() or (hq[p] & 0x7F == 0).all() and (hs[p] == 0).all()
            left[p] = False
        assert (hq[left] == 0x55).all() and (hs[left] == -7.0).all(), "rows outside the lists were written"
        q, s, h, err = hq[:n][named].view(R.E4M3), hs[:n][named], h[named], err[named]
        sd = s.double().repeat_interleave(128, 1)[:, :I]
        bound = err + (h.abs() + err) * 2.0 ** -4 * (1 + 2.0 ** -20) + sd * 2.0 ** -10
        assert ((R.dequant(q, s) - h).abs() <= bound).all()
        top = torch.nn.functional.pad(h.abs(), (0, s.shape[1] * 128 - I)).view(h.shape[0], -1, 128).amax(2)
        terr = torch.nn.functional.pad(err, (0, s.shape[1] * 128 - I)).view(h.shape[0], -1, 128).amax(2)
        assert ((s.double() - top / 448).abs() <= terr / 448 + top / 448 * 2 * R.U32).all()

        hq, hs = R.activations(n, I, torch.Generator().manual_seed(77))
        hq.view(torch.uint8)[~named] = 0x7F          # rows that the lists leave out are not read
        B.check(B.coli_moe_workspace_init(c.ws))
        c.y.fill_(float("nan"))
        B.check(B.coli_moe_down_fp8(c.dims, c.weights, hq.cuda(), hs.cuda(), c.T, c.w.cuda(), *dl, c.res.cuda(), c.y, c.ws))
        assert B.coli_moe_read_status(c.ws) == status
        ref, bound = R.down(c.L, hq, hs, c.w, lst, c.res)
        assert ((c.y[:c.T].cpu().double() - ref).abs() <= bound).all()
        assert torch.isnan(c.y[c.T:]).all()


# of 6 experts, 2 each: the 16-token kernel, the 64-token one and the pairs, in both products
LIST_SIZES = [(3, 256), (40, 1024), (300, 256)]


@pytest.mark.parametrize("T,H", LIST_SIZES)
@pytest.mark.parametrize("bad", ["expert", "offset", "assign", "count", "tail"])
def test_bad_lists_leave_the_others_right(colimoe, monkeypatch, T, H, bad):
    c = F.Case(H, 192, 6, 2, 1, T, seed=8)
    u, m, o, a = [t.clone() for t in c.lst]
    zeros = ()
    if bad == "expert":
        u[0] = 1 << 20
    elif bad == "offset":
        o[1] = 1 << 20
    elif bad == "assign":
        a[0], a[1] = -5, 1 << 30
        zeros = (0, 1)
    elif bad == "count":
        m[0] = 1 << 20
    else:      # the last list ends before the ones in front of it
        assert int(m[0]) >= 3 and int(o[2]) > 1
        m[0], o[3] = 3, 1
    check_lists(c, (u, m, o, a), monkeypatch, (B.COLI_EDEVICE, B.DEV_BAD_INDEX), zeros)


@pytest.mark.parametrize("T,H", LIST_SIZES)
def test_lists_of_one_rank_in_every_kernel(colimoe, monkeypatch, T, H):
    # experts 2 .. 4 of 6: some tokens have none of them, some slots are left out; then no expert at all
    c = F.Case(H, 192, 6, 2, 1, T, seed=6, e0=2, e1=5)
    check_lists(c, c.lst, monkeypatch, (B.COLI_OK, 0))
    none = (torch.full((3,), -1, dtype=torch.int32), torch.tensor([0], dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
            c.lst[3])
    check_lists(c, none, monkeypatch, (B.COLI_OK, 0))


@pytest.mark.parametrize("T,H,E", [(500, 64, 300), (500, 1088, 300), (700, 64, 1024), (16, 64, 1024)])
def test_many_lists(colimoe, T, H, E):
    # more lists than a block of the gather has threads, up to the most
    c = F.Case(H, 64, E, 2, 1, T, seed=T)
    assert int(c.lst[1]) > 256 or T == 16
    c.check_gate_up()
    c.check_down()


@pytest.mark.parametrize("T,H", LIST_SIZES)
@pytest.mark.parametrize("where", ["one list", "two lists"])
def test_a_position_named_twice_is_flagged(colimoe, T, H, where):
    c = F.Case(H, 192, 6, 2, 1, T, seed=8)
    a, off = c.lst[3].clone(), c.lst[2].tolist()
    # the first entry of a list in place of the last of the same list, or of the last list
    n = int(c.lst[1][0])
    u = max(range(n), key=lambda i: off[i + 1] - off[i])
    first, last = (off[u], off[u + 1] - 1) if where == "one list" else (off[0], off[n] - 1)
    assert first != last
    twice = int(a[first])
    a[last] = twice
    lst = [c.dl[0], c.dl[1], c.dl[2], a.cuda()]
    hq, hs = R.activations(c.rows, 192, torch.Generator().manual_seed(1))
    ys = []
    for _ in range(3):
        B.check(B.coli_moe_workspace_init(c.ws))
        B.check(B.coli_moe_down_fp8(c.dims, c.weights, hq.cuda(), hs.cuda(), T, c.w.cuda(), *lst, c.res.cuda(), c.y, c.ws))
        assert B.coli_moe_read_status(c.ws) == (B.COLI_EDEVICE, B.DEV_BAD_INDEX)
        ys.append(c.y.clone())
    assert torch.equal(ys[0][:T], ys[1][:T]) and torch.equal(ys[0][:T], ys[2][:T])
    # tokens that neither entry belongs to are right
    ref, bound = R.down(c.L, hq, hs, c.w, c.lst, c.res)
    keep = torch.ones(T, dtype=torch.bool)
    keep[[twice // 2, int(c.lst[3][last]) // 2]] = False
    off_ = (ys[0][:T].cpu().double() - ref).abs()
    assert (off_[keep] <= bound[keep]).all()


# ------------------------------------------------------------------------------------------------
# range
# ------------------------------------------------------------------------------------------------
def tiny(t, g):
    """Scales 2^-85 .. 2^-60 in place of t's: products of two of them lie on both sides of 2^-126 and of 2^-149."""
    return torch.ldexp(1 + torch.rand(t.shape, generator=g), torch.randint(-85, -60, t.shape, generator=g))


@pytest.mark.parametrize("T,N,K", [(5, 300, 1040), (40, 300, 1040), (300, 300, 1040), (300, 301, 528)])
def test_scale_products_below_the_normal_numbers(colimoe, T, N, K):
    # every kernel: beside the usual bound, 2^-125 for each block (and a denormal result's own rounding, one a block)
    g = torch.Generator().manual_seed(T)
    xq, xs = R.activations(T, K, g)
    wq, s = R.weights(N, K, g)
    xs, s = tiny(xs, g), tiny(s, g)
    y = torch.empty(T, N, device="cuda")
    B.check(B.coli_fp8_matmul(T, N, K, xq.cuda(), xs.cuda(), wq.cuda(), s.cuda(), None, y, dense_ws(T, N, K)))
    x, w = R.dequant(xq, xs), R.dequant_w(wq, s)
    bound = (x.abs() @ w.abs().T) * R.product_bound(R.blocks(K)) + R.blocks(K) * (2.0 ** -125 + 2.0 ** -149)
    off = (y.cpu().double() - x @ w.T).abs()
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("T,H", LIST_SIZES)
def test_scale_products_below_the_normal_numbers_down(colimoe, T, H):
    c = F.Case(H, 192, 6, 2, 1, T, seed=8)
    g = torch.Generator().manual_seed(T)
    hq, hs = R.activations(c.rows, 192, g)
    hs = torch.ldexp(1 + torch.rand(hs.shape, generator=g), torch.randint(-130, -100, hs.shape, generator=g))
    B.check(B.coli_moe_down_fp8(c.dims, c.weights, hq.cuda(), hs.cuda(), T, c.w.cuda(), *c.dl, None, c.y, c.ws))
    ref, bound = R.down(c.L, hq, hs, c.w, c.lst, None)
    more = 3 * R.blocks(192) * (2.0 ** -125 + 2.0 ** -149)
    assert ((c.y[:T].cpu().double() - ref).abs() <= bound + more).all()


# ------------------------------------------------------------------------------------------------
# tiles whose K steps are split between workers, which add the parts up
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,N,K,dtype,residual", [
    (64, 38400, 2048, torch.float32, True),        # 150 tiles for 148 CTAs, all split
    (130, 12801, 2064, torch.bfloat16, True),      # 153 tiles, ragged rows of y
    (600, 6400, 2064, torch.float32, True),        # 75 tiles for 74 pairs
    (600, 6400, 2048, torch.bfloat16, False),
    (1100, 7688, 1808, torch.bfloat16, True),      # 155 tiles: 74 whole ones beside 81 in parts
])
def test_matmul_split_tiles(colimoe, T, N, K, dtype, residual):
    xq, xs, wq, s, r = device_inputs(T, N, K, dtype, residual, T)
    ws = dense_ws(T, N, K)
    ys = [torch.full((T + 1, N), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    for y in ys:
        B.check(B.coli_fp8_matmul(T, N, K, xq, xs, wq, s, r, y, ws))
    assert B.coli_moe_read_status(ws) == (B.COLI_OK, 0)
    check_matmul(ys[0][:T], xq, xs, wq, s, r)
    assert torch.isnan(ys[0][T]).all() and torch.equal(ys[0][:T], ys[1][:T])


@pytest.mark.parametrize("T,H,I,E", [(40, 4096, 2048, 9),       # 160 tiles for 148 CTAs in both products
                                     (150, 4864, 2432, 3)])     # 76 tiles for 74 pairs in both
def test_experts_split_tiles(colimoe, T, H, I, E):
    c = F.Case(H, I, E, 2, 1, T, seed=4)
    assert all(0 < n <= 256 for n in (c.lst[2][1:] - c.lst[2][:-1])[:E].tolist()) and int(c.lst[1]) == E
    c.check_gate_up()
    c.check_down()
    c.check_down(in_place=True)


@pytest.mark.parametrize("T,H,I,E", [(40, 1024, 192, 6), (300, 256, 192, 6), (150, 1024, 2432, 3)])
def test_two_graphs_on_one_workspace_in_every_kernel(colimoe, T, H, I, E):
    # replayed in turn, and each twice in a row
    c = F.Case(H, I, E, 2, 1, T, seed=9)
    hq, hs = (t.cuda() for t in R.activations(c.rows, I, torch.Generator().manual_seed(10)))
    w, res, xq, xs = c.w.cuda(), c.res.cuda(), c.xq.cuda(), c.xs.cuda()

    def up():
        B.check(B.coli_moe_gate_up_fp8(c.dims, c.weights, xq, xs, T, *c.dl, c.hq, c.hs, c.ws))

    def down():
        B.check(B.coli_moe_down_fp8(c.dims, c.weights, hq, hs, T, w, *c.dl, res, c.y, c.ws))

    c.check_gate_up()
    up()
    down()
    want = c.hq.clone(), c.hs.clone(), c.y.clone()
    graphs = []
    for f in (up, down):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for order in ((0, 1), (1, 0), (0, 0, 1, 1), (1, 1, 0, 0)):
        c.hq[:c.rows] = 0
        c.hs[:c.rows] = 0
        c.y[:T] = 0
        for i in order:
            graphs[i].replay()
        assert torch.equal(c.hq, want[0]) and torch.equal(c.hs, want[1]) and torch.equal(c.y[:T], want[2][:T])
    assert B.coli_moe_read_status(c.ws) == (B.COLI_OK, 0)


@pytest.mark.parametrize("T,H", LIST_SIZES)
def test_two_streams_in_every_kernel(colimoe, T, H):
    # two layers at once, each with its workspace on a stream of its own
    layers, want = [F.Case(H, 320, 6, 2, 1, T, seed=20 + i) for i in range(2)], []
    args = []
    for c in layers:
        w, xq, xs, res = c.w.cuda(), c.xq.cuda(), c.xs.cuda(), c.res.cuda()
        args.append((w, xq, xs, res, torch.cuda.Stream()))

    def run(c, a, stream):
        w, xq, xs, res, _ = a
        B.check(B.coli_moe_forward_fp8(c.dims, c.weights, xq, xs, T, w, *c.dl, res, c.y, c.ws, stream=stream))

    for c, a in zip(layers, args):
        run(c, a, None)
        want.append(c.y[:T].clone())
        c.y.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for c, a in zip(layers, args):
            run(c, a, a[4])
    torch.cuda.synchronize()
    for c, y in zip(layers, want):
        assert torch.equal(c.y[:T], y) and B.coli_moe_read_status(c.ws) == (B.COLI_OK, 0)
