"""Host-side quantisation of fp32 expert weights into the library's blob containers.

Symmetric absmax scaling, round to nearest (ties to even), clipped to the container's code
range:
  gs64 int4: one fp16 scale per 64 input columns, codes [-8, 7],     scale = absmax / 7;
  gs64 int8: one fp16 scale per 64 input columns, codes [-128, 127], scale = absmax / 127;
  per-row int4: one fp16 scale per row,           codes [-8, 7],     scale = absmax / 7;
  gs64 int2: one fp16 scale per 64 input columns, codes [-2, 1],     scale = absmax / 2.
The scale is rounded to fp16 first and the codes are taken against the rounded scale.  Blob
order: Gq | Uq | Dq | Gs | Us | Ds, payload packed with the lowest-index column in the
lowest bits (the layout of coli_moe_blob_bytes_fmt).  The fp8 container (e4m3 codes, one fp32
scale per 128 rows and 128 columns, scale = absmax / 448) is made by the functions with fp8
in their names (the layout of coli_moe_blob_bytes_fp8).  This is a weight preparation tool;
the forward itself runs on the GPU only.
"""
import numpy as np

FMT_INT4_G64, FMT_INT8_G64, FMT_INT4_ROW, FMT_INT2_G64 = 0, 1, 2, 3
BITS = {FMT_INT4_G64: 4, FMT_INT8_G64: 8, FMT_INT4_ROW: 4, FMT_INT2_G64: 2}
QRANGE = {FMT_INT4_G64: (-8, 7), FMT_INT8_G64: (-128, 127), FMT_INT4_ROW: (-8, 7), FMT_INT2_G64: (-2, 1)}
QDIV = {FMT_INT4_G64: 7.0, FMT_INT8_G64: 127.0, FMT_INT4_ROW: 7.0, FMT_INT2_G64: 2.0}


def quantize_matrix(W: np.ndarray, fmt: int):
    """W [rows][in] float -> (codes [rows][in] int8, scales [rows][in/64] or [rows][1] fp16)."""
    W = np.asarray(W, np.float32)
    rows, cols = W.shape
    assert cols % 64 == 0
    g = 1 if fmt == FMT_INT4_ROW else cols // 64
    Wg = W.reshape(rows, g, cols // g)
    amax = np.abs(Wg).max(axis=2)
    s16 = (amax / QDIV[fmt]).astype(np.float16)
    s = s16.astype(np.float32)
    safe = np.where(s > 0, s, 1.0)
    lo, hi = QRANGE[fmt]
    q = np.clip(np.rint(Wg / safe[:, :, None]), lo, hi)
    q = np.where(s[:, :, None] > 0, q, 0).astype(np.int8).reshape(rows, cols)
    return q, s16


def dequantize_matrix(q: np.ndarray, s16: np.ndarray) -> np.ndarray:
    rows, cols = q.shape
    g = s16.shape[1]
    return (q.reshape(rows, g, cols // g).astype(np.float32) * s16.astype(np.float32)[:, :, None]).reshape(rows, cols)


def pack_codes(q: np.ndarray, bits: int) -> np.ndarray:
    rows, cols = q.shape
    per = 8 // bits
    mask = (1 << bits) - 1
    u = (q.astype(np.int64) & mask).reshape(rows, cols // per, per)
    out = np.zeros((rows, cols // per), np.int64)
    for j in range(per):
        out |= u[:, :, j] << (bits * j)
    return out.astype(np.uint8).reshape(-1)


def expert_blob(G: np.ndarray, U: np.ndarray, D: np.ndarray, fmt: int):
    """G, U [I][H] and D [H][I] float -> (blob uint8, dequantised (G, U, D))."""
    parts, scs, deq = [], [], []
    for M in (G, U, D):
        q, s = quantize_matrix(M, fmt)
        parts.append(pack_codes(q, BITS[fmt]))
        scs.append(s.view(np.uint8).reshape(-1))
        deq.append(dequantize_matrix(q, s))
    return np.concatenate(parts + scs), tuple(deq)


# ------------------------------------------------------------------------------------
# e4m3 codes with one fp32 scale per 128 x 128 block
# ------------------------------------------------------------------------------------
FP8_MAX, FP8_BLOCK = 448.0, 128


def e4m3_codes(v: np.ndarray) -> np.ndarray:
    """float values -> e4m3 codes (uint8): to nearest, ties to even, clipped to +-448, NaN to 0x7F."""
    v = np.asarray(v, np.float32).astype(np.float64)
    a = np.minimum(np.abs(v), FP8_MAX)
    _, e = np.frexp(np.where(np.isnan(a), 0.0, a))
    e = np.maximum(e - 1, -6)                       # exponent of the leading bit, subnormals at -6
    m = np.rint(np.ldexp(np.nan_to_num(a), 3 - e)).astype(np.int64)   # 0 .. 16 eighths of 2^e
    # m = 16 carries into the next exponent; m < 8 only occurs at e = -6 (subnormals)
    code = np.where(m >= 8, ((e + 7) << 3) + (m - 8), m)
    code = np.where(np.isnan(v), 0x7F, code)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    """e4m3 codes (uint8) -> float32 values."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, np.ldexp(8.0 + m, e - 10), np.ldexp(m.astype(np.float64), -9))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v).astype(np.float32)


def _fp8_blocks(n: int) -> int:
    return (n + FP8_BLOCK - 1) // FP8_BLOCK


def quantize_matrix_fp8(W: np.ndarray):
    """W [rows][cols] float -> (codes [rows][cols] uint8, scales [C(rows)][C(cols)] fp32).  A block with a NaN has a NaN
    scale and NaN codes throughout; one with an infinity an infinite scale, NaN codes there and 0 elsewhere."""
    W = np.asarray(W, np.float32)
    rows, cols = W.shape
    rb, cb = _fp8_blocks(rows), _fp8_blocks(cols)
    P = np.zeros((rb * FP8_BLOCK, cb * FP8_BLOCK), np.float32)
    P[:rows, :cols] = W
    P = P.reshape(rb, FP8_BLOCK, cb, FP8_BLOCK)
    s = (np.abs(P).max(axis=(1, 3)) / np.float32(FP8_MAX)).astype(np.float32)
    safe = np.where(s == 0, np.float32(1.0), s)
    with np.errstate(invalid="ignore"):
        q = e4m3_codes(P / safe[:, None, :, None])
    return np.ascontiguousarray(q.reshape(rb * FP8_BLOCK, cb * FP8_BLOCK)[:rows, :cols]), s


def dequantize_matrix_fp8(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    rows, cols = q.shape
    full = np.repeat(np.repeat(s, FP8_BLOCK, 0)[:rows], FP8_BLOCK, 1)[:, :cols]
    return e4m3_values(q) * full


def expert_blob_fp8(G: np.ndarray, U: np.ndarray, D: np.ndarray):
    """G, U [I][H] and D [H][I] float -> (blob uint8, dequantised (G, U, D))."""
    parts, scs, deq = [], [], []
    for M in (G, U, D):
        q, s = quantize_matrix_fp8(M)
        parts.append(q.reshape(-1))
        scs.append(s.reshape(-1).view(np.uint8))
        deq.append(dequantize_matrix_fp8(q, s))
    return np.concatenate(parts + scs), tuple(deq)
