"""Plain NumPy forms of the norm, its gradient, the block quantiser and the
fp8 matrix product, for the tests.  Written from the definitions in
include/ar.h; shares no code with the library.

Values are computed in 64 bits, except where a test compares bits: the rank
sum and the quantiser follow the stated binary32 steps one by one.
"""
import numpy as np

U32 = 2.0 ** -24          # unit roundoff of binary32
U16 = 2.0 ** -8           # of bf16, which has 8 significand bits


def bf16_bits(x) -> np.ndarray:
    """binary32 array -> bf16 patterns, nearest even, NaN as 0x7FC0."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    r[np.isnan(x)] = 0x7FC0
    return r


def bf16_val(b) -> np.ndarray:
    return (np.ascontiguousarray(b, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32)


def as_bf16(x) -> np.ndarray:
    """Values rounded to bf16, as binary32."""
    return bf16_val(bf16_bits(x)).reshape(np.shape(x))


def _e4m3_table() -> np.ndarray:
    v = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = -x if s else x
    v[0x7F] = v[0xFF] = np.nan
    return v


E4M3 = _e4m3_table()
_POS = E4M3[:0x7F]                                   # 0 .. 448, ascending
_MID = (_POS[1:] + _POS[:-1]) / 2


def e4m3_codes(x) -> np.ndarray:
    """Nearest code of each value (|x| <= 448 after rounding), ties to even;
    0x7F for what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    with np.errstate(invalid="ignore"):
        lo = np.searchsorted(_MID, a, side="left")   # a at a midpoint stays below
        tie = np.isin(a, _MID)
        lo = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.int64)
    c = (np.minimum(lo, 0x7E) | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)
    c[~np.isfinite(x)] = 0x7F
    return c


def block_amax(f, block_rows: int) -> np.ndarray:
    """Largest finite magnitude of each block_rows x 128 block."""
    rows, cols = f.shape
    a = np.where(np.isfinite(f), np.abs(f), 0)
    R, C = -(-rows // block_rows), -(-cols // 128)
    p = np.zeros((R * block_rows, C * 128), dtype=f.dtype)
    p[:rows, :cols] = a
    return p.reshape(R, block_rows, C, 128).max(axis=(1, 3))


def spread(s, shape, block_rows: int) -> np.ndarray:
    """A scale for each element."""
    return np.repeat(np.repeat(s, block_rows, 0)[:shape[0]], 128, 1)[:, :shape[1]]


def quantise(f, block_rows: int, e8m0: bool):
    """(codes, scales) by the stated binary32 steps; scales as kept."""
    f = np.asarray(f, dtype=np.float32)
    amax = block_amax(f, block_rows)
    if e8m0:
        k = np.full(amax.shape, -127, dtype=np.int64)
        for e in range(-127, 128):                   # smallest k with amax <= 448 * 2^k
            k = np.where(amax.astype(np.float64) > 448.0 * 2.0 ** e, e + 1, k)
        inv = 2.0 ** -k.astype(np.float64)
        kept = (k + 127).astype(np.uint8)
    else:
        kept = np.maximum(amax / np.float32(448), np.float32(2.0 ** -126)).astype(np.float32)
        inv = (np.float32(1) / kept).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = f * spread(inv, f.shape, block_rows).astype(np.float32)
    return e4m3_codes(q), kept


def scale_val(s) -> np.ndarray:
    """Scales as kept -> 64-bit values."""
    s = np.asarray(s)
    if s.dtype == np.uint8:
        return np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return s.astype(np.float64)


def dequantise(codes, scales, block_rows: int) -> np.ndarray:
    return E4M3[codes] * spread(scale_val(scales), codes.shape, block_rows)


def rank_sum(xs, residual=None) -> np.ndarray:
    """binary32, rank order, the residual last."""
    h = xs[0].astype(np.float32)
    for x in list(xs[1:]) + ([] if residual is None else [residual]):
        h = (h + x.astype(np.float32)).astype(np.float32)
    return h


def norm(h, weight, eps) -> np.ndarray:
    h = h.astype(np.float64)
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return y if weight is None else y * weight.astype(np.float64)


def norm_bwd(dy, h, weight, dres, eps):
    """(dx, dweight) in 64 bits."""
    dy, h = dy.astype(np.float64), h.astype(np.float64)
    w = np.ones(h.shape[1]) if weight is None else weight.astype(np.float64)
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    x, g = h * r, dy * w
    dx = r * (g - x * (g * x).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + dres.astype(np.float64)
    return dx, (dy * x).sum(0)
