"""Plain fp64 form of the microscaled 4-bit formats, written from the formats' definition (test
infrastructure: NumPy on the host, no code of the library)."""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
# E4M3 values 0 .. 448, code order
E4M3 = np.array([(1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) if c > 7 else c / 8 * 2.0 ** -6 for c in range(127)])


def nearest_even(table, v):
    """Index of the entry of an ascending table nearest to each v >= 0, ties to the even index."""
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    d_lo, d_hi = v - table[lo], table[hi] - v
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantize(x, fmt):
    """(codes rows x cols, scale bytes rows x blocks, global scale) of a float64 matrix."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    b = BLOCK[fmt]
    n = -(-cols // b)
    p = np.zeros((rows, n * b))
    p[:, :cols] = x
    p = p.reshape(rows, n, b)
    ok = np.isfinite(p).all(axis=2)
    mag = np.where(np.isfinite(p), np.abs(p), 0.0)
    g = 1.0
    if fmt == MX:
        top = np.where(ok, mag.max(axis=2), 0.0)
        e = np.where(top > 0, np.frexp(top)[1] - 3, -127).clip(-127, 125)
        scale = 2.0 ** e.astype(np.float64)
        byte = e + 127
    else:
        most = mag.max() if mag.size else 0.0
        if most > 0:
            g = 2.0 ** -126
            while most > 2688 * g:
                g *= 2
        top = np.where(ok, mag.max(axis=2), 0.0)
        byte = nearest_even(E4M3, np.minimum(top / (6 * g), 448.0))
        scale = E4M3[byte]
    unit = (scale * g)[:, :, None]
    q = np.divide(mag, unit, out=np.zeros_like(mag), where=unit > 0)
    code = nearest_even(MAGNITUDES, np.minimum(q, 6.0)) + 8 * np.signbit(p)
    code = np.where(ok[:, :, None], code, 0)
    byte = np.where(ok, byte, 255 if fmt == MX else 127)
    return code.reshape(rows, -1)[:, :cols].astype(np.uint8), byte.astype(np.uint8), g


def values(code, byte, g, fmt):
    b = BLOCK[fmt]
    v = MAGNITUDES[code % 8] * np.where(code > 7, -1.0, 1.0)
    if fmt == MX:
        s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    else:
        s = np.where(byte == 127, np.nan, E4M3[np.minimum(byte, 126)])
    return v * np.repeat(s, b, axis=1)[:, :code.shape[1]] * g


def pack(code):
    rows, cols = code.shape
    p = np.zeros((rows, -(-cols // 128) * 128), dtype=np.uint8)
    p[:, :cols] = code
    return p[:, 0::2] | (p[:, 1::2] << 4)


def tile_scales(byte, rows, cols, fmt):
    """Scale bytes in the order of the format: padding blocks zero."""
    wide = -(-cols // 128) * 128 // BLOCK[fmt]
    out = np.zeros(-(-rows // 128) * 128 * wide, dtype=np.uint8)
    r = np.arange(rows)[:, None]
    s = np.arange(byte.shape[1])[None, :]
    out[((r // 128) * (wide // 4) + s // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + s % 4] = byte
    return out
