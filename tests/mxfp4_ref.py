"""MXFP4 in 64 bits on the CPU: the definition, evaluated with numpy.

A block of 32 has the scale 2^(floor(log2 max|x|) - 2), not below 2^-127, and its codes are
the nearest of 0 0.5 1 1.5 2 3 4 6 to |x| / scale, ties to the even code, with the sign bit;
a block with a NaN or an infinity has the scale byte 255 and codes 0.  Written for the
tests alone: it shares nothing with the library.
"""

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def blocks(cols):
    return -(-cols // 32)


def encode(x):
    """x (float64, rows x cols) -> (codes 0..15, rows x cols; scale bytes, rows x blocks)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = blocks(cols)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    bad = ~np.isfinite(b).all(2)
    top = np.abs(np.where(bad[:, :, None], 0, b)).max(2)
    e = np.frexp(top)[1] - 1  # top = 1.m * 2^e
    s = np.where(top > 0, np.clip(e - 2 + 127, 0, 254), 0)
    v = np.ldexp(np.where(bad[:, :, None], 0, b), (127 - s)[:, :, None])
    # nearest with ties to even: the distance to each value, the even code first among equals
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    dist = np.abs(np.minimum(np.abs(v), 6)[..., None] - GRID[order])
    code = order[dist.argmin(-1)] + 8 * np.signbit(v)
    code = np.where(bad[:, :, None], 0, code)
    return code.reshape(rows, nb * 32)[:, :cols].astype(np.uint8), np.where(bad, 255, s).astype(np.uint8)


def values(code, s):
    """What codes (rows x cols) and scale bytes (rows x blocks) stand for, in float64."""
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    scale = np.ldexp(1.0, s.astype(int) - 127)
    scale[s == 255] = np.nan
    return v * np.repeat(scale, 32, 1)[:, :code.shape[1]]


def pack_codes(code, ld=None, fill=0):
    """Codes in the library's layout: (rows, ld) bytes; bytes beyond the blocks hold `fill`."""
    rows, cols = code.shape
    nb = blocks(cols)
    full = np.zeros((rows, nb * 32), np.uint8)
    full[:, :cols] = code
    out = np.full((rows, ld or 16 * nb), fill, np.uint8)
    out[:, :16 * nb] = full[:, 0::2] | (full[:, 1::2] << 4)
    return out


def pack_scales(s):
    """Scale bytes in the library's layout, one element at a time by its stated address."""
    rows, nb = s.shape
    atoms = -(-nb // 4)
    out = np.zeros(-(-rows // 128) * atoms * 512, np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[512 * ((r // 128) * atoms + b // 4) + 16 * (r % 32) + 4 * ((r % 128) // 32) + b % 4] = s
    return out


def through(x):
    """x quantised along its rows and back, in float64."""
    return values(*encode(x))


def random_codes(rng, rows, cols, lo=126, hi=129):
    """Random codes and scale bytes in [lo, hi)."""
    return (rng.integers(0, 16, (rows, cols)).astype(np.uint8),
            rng.integers(lo, hi, (rows, blocks(cols))).astype(np.uint8))
