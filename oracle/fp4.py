"""Microscaled 4-bit floating point in 64 bits: plain numpy, one matrix at a time, no code shared with the GPU path.

A block of values along a row shares a scale d, and each value is held as the nearest of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} d
(ties to the even code, magnitudes above 6 d as 6 d).
  nvfp4: blocks of 16, d = g s; g the smallest power of two (at least 2^-126) with max |X| <= 6 * 448 g, 0 for X = 0;
         s = max |block| / (6 g), the nearest e4m3 number, ties to even, at most 448
  mxfp4: blocks of 32, d = 2^e, e = floor(log2(max |block|)) - 2, at least -127
A block that holds Inf or NaN has the scale NaN and codes of 0; g is that of the finite values.
"""
import numpy as np

BLOCK = {"nvfp4": 16, "mxfp4": 32}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# index = the bits: 4 of exponent (bias 7), 3 of significand; the last (0x7F) is NaN and left out
E4M3 = np.array([(m / 8.0 * 2.0**-6) if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:-1])


def nearest(a, grid):
    """Index of the value of `grid` nearest to each a >= 0, ties to the even index, the last one above all."""
    hi = np.clip(np.searchsorted(grid, a, side="left"), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    to_lo, to_hi = a - grid[lo], grid[hi] - a
    take_lo = (to_lo < to_hi) | ((to_lo == to_hi) & (lo % 2 == 0))
    return np.where(a >= grid[-1], len(grid) - 1, np.where(take_lo, lo, hi))


def tensor_scale(most):
    """g of a largest magnitude."""
    if most == 0.0:
        return 0.0
    e = -126
    while 2688.0 * 2.0**e < most:
        e += 1
    return 2.0**e


def quantize(x, fmt, amax=None):
    """(codes (rows, cols) 0 .. 15, scales' bytes (rows, blocks), g or None) of x (rows, cols) in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    n = BLOCK[fmt]
    blocks = -(-cols // n)
    v = np.zeros((rows, blocks * n))
    v[:, :cols] = x
    v = v.reshape(rows, blocks, n)
    bad = ~np.isfinite(v).all(2)
    most = np.abs(np.where(bad[..., None], 0.0, v)).max(2)
    if fmt == "nvfp4":
        finite = np.abs(x[np.isfinite(x)])
        if amax is None:
            g = tensor_scale(finite.max() if finite.size else 0.0)
        else:
            g = tensor_scale(amax) if amax > 0 and np.isfinite(amax) else 1.0
        byte = nearest(most / g / 6.0, E4M3) if g else np.zeros(most.shape, dtype=np.int64)
        d = E4M3[byte] * g
    else:
        g = None
        e = np.where(most > 0, np.frexp(most)[1] - 3, -127).clip(-127)
        byte = e + 127
        d = 2.0**e
    v = np.where(bad[..., None], 0.0, v)
    code = nearest(np.divide(np.abs(v), d[..., None], out=np.zeros_like(v), where=d[..., None] > 0), E2M1)
    code = np.where(np.signbit(v) & (d[..., None] > 0), code + 8, code)
    code = np.where(bad[..., None], 0, code)
    byte = np.where(bad, 0x7F if fmt == "nvfp4" else 0xFF, byte).astype(np.uint8)
    return code.reshape(rows, -1)[:, :cols].astype(np.uint8), byte, g


def values(code, byte, g, fmt):
    """What codes and scales stand for, in 64 bits."""
    rows, cols = code.shape
    s = np.append(E4M3, [np.nan])[byte & 0x7F] * g if fmt == "nvfp4" else np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    v = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    return v * np.repeat(s, BLOCK[fmt], axis=1)[:, :cols]


def pack_codes(code, width=None):
    """Two codes a byte, the first in the low half; rows of `width` bytes (default: ceil(cols / 32) * 16)."""
    rows, cols = code.shape
    width = -(-cols // 32) * 16 if width is None else width
    c = np.zeros((rows, 2 * width), dtype=np.uint8)
    c[:, :cols] = code
    return c[:, 0::2] | (c[:, 1::2] << 4)


def pack_scales(byte):
    """(row tiles, block tiles, 512): row r, block k at (r % 32) * 16 + (r % 128) / 32 * 4 + k % 4 of its tile."""
    rows, blocks = byte.shape
    t = np.zeros((-(-rows // 128), -(-blocks // 4), 512), dtype=np.uint8)
    r, k = np.arange(rows)[:, None], np.arange(blocks)[None, :]
    t[r // 128, k // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4] = byte
    return t
