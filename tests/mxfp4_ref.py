"""MXFP4 in 64 bits on the CPU, for the tests: the format's definition (values,
nearest-even rounding, scale rule, tiled scale bytes) in plain numpy."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_bytes(x):
    """x [rows, cols] float64 -> scale byte per block of 32 [rows, cols / 32]."""
    b = np.abs(x.reshape(x.shape[0], -1, 32))
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 1.0, b.max(-1, initial=0.0, where=np.isfinite(b)))
    e = np.full(amax.shape, -127.0)
    e[amax > 0] = np.floor(np.log2(amax[amax > 0])) - 2
    s = np.clip(e, -127, 127) + 127
    s[bad] = 255
    return s.astype(np.uint8)


def codes_of(x, s):
    """e2m1 codes [rows, cols] of x under its blocks' scale bytes."""
    sb = np.repeat(s, 32, axis=1).astype(np.float64)
    nan = sb == 255
    y = np.where(nan, 0.0, x) * np.exp2(127.0 - sb)
    a = np.abs(y)
    hi = np.clip(np.searchsorted(GRID, a, side="left"), 1, 7)
    lo = hi - 1
    mid = (GRID[lo] + GRID[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    c = np.where(up, hi, lo).astype(np.uint8) | (np.signbit(y).astype(np.uint8) << 3)
    c[nan] = 0
    return c


def pack(c):
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def unpack(p):
    return np.stack((p & 15, p >> 4), -1).reshape(p.shape[0], -1)


def tile(s, fill=0):
    """Scale bytes [rows, blocks] in the tiled byte order, rows padded with `fill`."""
    rows, nb = s.shape
    out = np.full((rows + 127) // 128 * 128 * nb, fill, np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[((r // 128) * (nb // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = s
    return out


def values(c, s):
    """float64 values of codes [rows, cols] under scale bytes [rows, cols / 32]."""
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    sb = np.repeat(s, 32, axis=1).astype(np.float64)
    return np.where(sb == 255, np.nan, v * np.exp2(sb - 127.0))


def quantize(x):
    """x [rows, cols] -> (packed codes, tiled scales, float64 values)."""
    s = scale_bytes(x)
    c = codes_of(x, s)
    return pack(c), tile(s), values(c, s)
