"""Plain float64 implementation of the 8-bit layer's format and operators (numpy only)."""
import numpy as np

B = 128


def code_values():
    """The 256 e4m3 codes as float64: sign, 4 exponent bits with bias 7, 3 mantissa bits; 0x7f and 0xff NaN."""
    v = np.empty(256)
    for c in range(256):
        ex, man = (c >> 3) & 15, c & 7
        v[c] = man * 2.0 ** -9 if ex == 0 else (1 + man / 8) * 2.0 ** (ex - 7)
        if ex == 15 and man == 7:
            v[c] = np.nan
        if c & 128:
            v[c] = -v[c]
    return v


VALUES = code_values()


def blocks(n):
    return -(-n // B)


def block_amax(x, tiles):
    """Largest finite magnitude of each block (0 where there is none)."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    rows, cols = a.shape
    a = np.pad(a, ((0, blocks(rows) * B - rows if tiles else 0), (0, blocks(cols) * B - cols)))
    h = B if tiles else 1
    return a.reshape(a.shape[0] // h, h, a.shape[1] // B, B).max(axis=(1, 3))


def scale_bytes(x, tiles):
    """127 + the least e >= -117 with amax <= 448 * 2^e."""
    amax = block_amax(x, tiles)
    e = np.full(amax.shape, -117)
    while (amax > 448.0 * 2.0 ** e.astype(np.float64)).any():
        e = e + (amax > 448.0 * 2.0 ** e.astype(np.float64))
    return (e + 127).astype(np.uint8)


def spread(scales, rows, cols, tiles):
    """The scale of every element."""
    s = np.exp2(scales.astype(np.float64) - 127)
    s = np.repeat(s, B, axis=1)[:, :cols]
    return np.repeat(s, B, axis=0)[:rows] if tiles else s


def nearest_code(v):
    """Codes of float64 values in [-448, 448] (round to nearest, ties to the even code); NaN for the rest."""
    grid = VALUES[:127]  # nonnegative codes, ascending
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, np.where(np.isfinite(a), a, 0.0)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - grid[lo], grid[hi] - a
    up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    q = np.where(up, hi, lo)
    q = np.where(np.signbit(v), q | 128, q)
    return np.where(np.isfinite(v), q, 0x7f).astype(np.uint8)


def pack(x, tiles):
    x = x.astype(np.float64)
    s = scale_bytes(x, tiles)
    return nearest_code(x / spread(s, *x.shape, tiles)), s


def unpack(codes, scales, tiles):
    return VALUES[codes] * spread(scales, *codes.shape, tiles)
