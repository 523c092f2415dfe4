"""Reference for the 8-bit floating point path in 64 bits (torch on the CPU), and seeded inputs.

Every expected value is computed from the codes and scales themselves in double; beside each
product the sum of its terms' magnitudes is returned, which the error bounds are multiples of.
"""
from __future__ import annotations

import dataclasses

import torch

E4M3 = torch.float8_e4m3fn
U32 = 2.0 ** -24          # half a step of fp32, relative
# A product's inner sum: 128 terms on the tensor cores in some order, each addition off by a
# whole step at most (2^-23); then one addition per scale block and the scale products, each
# rounded to nearest (2^-24).
def product_bound(kb: int, more: int = 0) -> float:
    return 128 * 2 * U32 + (kb + 3 + more) * U32


# silu(g) * u, relative, in half steps of fp32: 4 for the power of two (2^-22), 1 for its product
# with 1 + c, |g| / 20 for ln 2 as a float in c (off by 1.9e-9, times |g| / ln 2), 1 each for 1 + e^-g, the
# corrected quotient and the product with u.
def silu_bound(g: torch.Tensor) -> torch.Tensor:
    return (8 + g.abs() / 20) * U32 * (1 + 2.0 ** -16)


def blocks(n: int) -> int:
    return (n + 127) // 128


def quantize(v: torch.Tensor):
    """fp32 rows -> (codes, scales): the definition, in fp32 steps."""
    rows, cols = v.shape
    nb = blocks(cols)
    p = torch.zeros(rows, nb * 128)
    p[:, :cols] = v
    p = p.view(rows, nb, 128)
    s = p.abs().amax(2) / 448.0
    q = torch.where(s[:, :, None] > 0, p / torch.where(s > 0, s, torch.ones_like(s))[:, :, None], torch.zeros(()))
    return q.clamp(-448, 448).view(rows, nb * 128)[:, :cols].to(E4M3).contiguous(), s


def dequant(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    """Activation codes [rows][cols] and scales [rows][C(cols)] in double."""
    return q.double() * s.double().repeat_interleave(128, 1)[:, :q.shape[1]]


def dequant_w(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    """Weight codes [rows][cols] and scales [C(rows)][C(cols)] in double."""
    return q.double() * s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def activations(rows: int, cols: int, g: torch.Generator):
    return quantize(torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g)))


def weights(rows: int, cols: int, g: torch.Generator):
    q = (torch.randn(rows, cols, generator=g) * 110).clamp(-448, 448).to(E4M3)
    s = (0.5 + torch.rand(blocks(rows), blocks(cols), generator=g)) / (110 * cols ** 0.5)
    return q, s


@dataclasses.dataclass
class Layer:
    H: int
    I: int
    E: int
    k: int
    n_shared: int
    mats: list            # per expert (the shared one last): (G, U, D) in double
    blobs: torch.Tensor   # [E][stride] uint8
    shared: torch.Tensor  # [stride] uint8 or None
    stride: int


def blob_bytes(H: int, I: int) -> int:
    return 3 * H * I + 12 * blocks(H) * blocks(I)


def make_layer(H, I, E, k, n_shared, seed) -> Layer:
    g = torch.Generator().manual_seed(seed)
    stride = (blob_bytes(H, I) + 255) // 256 * 256 + 256 * (seed % 2)      # padded blobs too
    mats, rows = [], []
    for _ in range(E + n_shared):
        parts = [weights(I, H, g), weights(I, H, g), weights(H, I, g)]
        mats.append([dequant_w(q, s) for q, s in parts])
        b = torch.full((stride,), 0x7F, dtype=torch.uint8)      # NaN codes behind the blob
        raw = torch.cat([q.view(torch.uint8).reshape(-1) for q, _ in parts] +
                        [s.reshape(-1).view(torch.uint8) for _, s in parts])
        b[:raw.numel()] = raw
        rows.append(b)
    return Layer(H, I, E, k, n_shared, mats, torch.stack(rows[:E]), rows[E] if n_shared else None, stride)


def lists(idx: torch.Tensor, E: int, e0: int = 0, e1: int = None):
    """Union lists of idx [T][k] (optionally only experts e0 .. e1 - 1, renumbered)."""
    e1 = E if e1 is None else e1
    T, k = idx.shape
    ids, off, asg = [], [0], []
    flat = idx.reshape(-1).tolist()
    for e in range(e0, e1):
        at = [i for i, v in enumerate(flat) if v == e]
        if at:
            ids.append(e - e0)
            asg += at
            off.append(len(asg))
    n = len(ids)
    E_l = e1 - e0
    union = torch.full((E_l,), -1, dtype=torch.int32)
    union[:n] = torch.tensor(ids, dtype=torch.int32)
    offsets = torch.full((E_l + 1,), off[-1], dtype=torch.int32)
    offsets[:n + 1] = torch.tensor(off, dtype=torch.int32)
    assign = torch.full((max(T * k, 1),), 0, dtype=torch.int32)
    assign[:len(asg)] = torch.tensor(asg, dtype=torch.int32)
    return union, torch.tensor([n], dtype=torch.int32), offsets, assign


def groups(L: Layer, lst, T: int):
    """(matrices, rows of h, positions t * k + slot or None) of each list and the shared expert."""
    union, n, off, asg = (t.tolist() for t in lst)
    out = [(L.mats[union[u]], torch.arange(off[u], off[u + 1]), torch.tensor(asg[off[u]:off[u + 1]]))
           for u in range(n[0])]
    if L.n_shared:
        out.append((L.mats[L.E], torch.arange(T * L.k, T * L.k + T), None))
    return out


def gate_up(L: Layer, xq, xs, lst):
    """h in double, a bound on the error of a kernel's h, and which rows the lists name."""
    T = xq.shape[0]
    x = dequant(xq, xs)
    rows = T * (L.k + L.n_shared)
    h, err = torch.zeros(rows, L.I, dtype=torch.float64), torch.zeros(rows, L.I, dtype=torch.float64)
    named = torch.zeros(rows, dtype=torch.bool)
    rel = product_bound(blocks(L.H))
    for (G, U, _), at, asg in groups(L, lst, T):
        xe = x if asg is None else x[asg // L.k]
        ge, ue = xe @ G.T, xe @ U.T
        dg, du = rel * (xe.abs() @ G.abs().T), rel * (xe.abs() @ U.abs().T)
        s = ge * torch.sigmoid(ge)
        h[at] = s * ue
        # |silu'| <= 1.1; the rest as silu_bound has it
        err[at] = 1.1 * ue.abs() * dg + s.abs() * du + 1.1 * dg * du + silu_bound(ge) * (s * ue).abs()
        named[at] = True
    return h, err, named


def down(L: Layer, hq, hs, w, lst, residual):
    T = w.shape[0]
    h = dequant(hq, hs)
    y = residual.double().clone() if residual is not None else torch.zeros(T, L.H, dtype=torch.float64)
    mag = y.abs()
    for (_, _, D), at, asg in groups(L, lst, T):
        z, m = h[at] @ D.T, h[at].abs() @ D.abs().T
        if asg is None:
            y += z
            mag += m
        else:
            wt = w.double().reshape(-1)[asg][:, None]
            y.index_add_(0, asg // L.k, z * wt)
            mag.index_add_(0, asg // L.k, m * wt)
    return y, mag * product_bound(blocks(L.I), L.k + 2)
