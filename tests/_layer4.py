"""Plain float64 implementation of the 4-bit layer's format (numpy only)."""
import numpy as np

B = 32
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def blocks(n, size=B):
    return -(-n // size)


def scale_bytes(x):
    """127 + the least e >= -125 with the block's largest magnitude <= 6 * 2^e; 255 where the block is not finite."""
    rows, cols = x.shape
    a = np.pad(np.abs(x), ((0, 0), (0, blocks(cols) * B - cols))).reshape(rows, -1, B)
    fine = np.isfinite(a).all(axis=2)
    amax = np.where(fine[:, :, None], a, 0.0).max(axis=2)
    e = np.full(amax.shape, -125)
    while (amax > 6.0 * 2.0 ** e.astype(np.float64)).any():
        e = e + (amax > 6.0 * 2.0 ** e.astype(np.float64))
    return np.where(fine, e + 127, 255).astype(np.uint8)


def spread(scales, cols):
    """The scale of every element."""
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return np.repeat(s, B, axis=1)[:, :cols]


def nearest_code(v):
    """Codes of float64 values in [-6, 6]: to nearest, ties to the even code; 0 for NaN."""
    a = np.abs(np.where(np.isnan(v), 0.0, v))
    hi = np.clip(np.searchsorted(VALUES[:8], a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - VALUES[lo], VALUES[hi] - a
    q = np.where((dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isnan(v), 0, np.where(np.signbit(v), q + 8, q)).astype(np.uint8)


def pairs(codes):
    """Two codes a byte, the earlier one in the low half."""
    rows, cols = codes.shape
    p = np.pad(codes, ((0, 0), (0, cols % 2)))
    return (p[:, 0::2] | p[:, 1::2] << 4).astype(np.uint8)


def tile_place(r, j, cols):
    """Byte that row r's block j has among the scales."""
    return (r // 128 * blocks(cols, 128) + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4


def tiled(scales, cols):
    rows = scales.shape[0]
    out = np.full(blocks(rows, 128) * blocks(cols, 128) * 512, 127, np.uint8)
    out[tile_place(np.arange(rows)[:, None], np.arange(scales.shape[1])[None], cols)] = scales
    return out


def pack(x):
    """Code bytes and scale bytes as they lie in memory, and the values they stand for."""
    x = x.astype(np.float64)
    s = scale_bytes(x)
    with np.errstate(invalid="ignore"):
        codes = nearest_code(x / spread(s, x.shape[1]))
    return pairs(codes), tiled(s, x.shape[1]), VALUES[codes] * spread(s, x.shape[1])
