"""Microscaled 4-bit blocks from their definition, in numpy and 64 bits."""
import numpy as np

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_bytes(rows, K):
    return -(-rows // 128) * -(-K // 128) * 512


def tiles(grid, K):
    """Scale bytes [rows, K / 32] in tiles of 128 rows by 4 blocks, zeros outside."""
    rows = grid.shape[0]
    R, C = -(-rows // 128), -(-K // 128)
    out = np.zeros(R * C * 512, np.uint8)
    for r in range(rows):
        for k in range(grid.shape[1]):
            tile = (r // 128) * C + k // 4
            out[tile * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4] = grid[r, k]
    return out


def grid(scales, rows, K):
    """The scale bytes [rows, K / 32] of tiles."""
    C = -(-K // 128)
    r = np.arange(rows)[:, None]
    k = np.arange(K // 32)[None]
    return scales[((r // 128) * C + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4]


def quantize(x):
    """x float64 [rows, K] -> (codes uint8 [rows, K], scale bytes [rows, K / 32])."""
    rows, K = x.shape
    b = x.reshape(rows, K // 32, 32)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(top)
    e = np.full(top.shape, -127)
    for i in np.ndindex(top.shape):
        if bad[i] or top[i] == 0:
            continue
        k = -127  # the least exponent that holds the block
        while 6.0 * 2.0 ** k < top[i]:
            k += 1
        e[i] = k
    q = b / np.exp2(e.astype(np.float64))[..., None]
    q = np.where(bad[..., None], 0.0, q)
    a = np.abs(q)
    lower = np.searchsorted(MAGS, a, side="right") - 1
    upper = np.minimum(lower + 1, 7)
    down, up = a - MAGS[lower], MAGS[upper] - a
    code = np.where(down == up, lower + lower % 2, np.where(down < up, lower, upper))
    code = np.where(a >= 6.0, 7, code) + 8 * np.signbit(q)
    return code.reshape(rows, K).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def values(packed, scale_grid):
    """Packed codes and scale bytes [rows, K / 32] -> float64 [rows, K]."""
    rows = packed.shape[0]
    codes = np.empty((rows, 2 * packed.shape[1]), np.int64)
    codes[:, 0::2], codes[:, 1::2] = packed & 15, packed >> 4
    v = MAGS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scale_grid == 255, np.nan, np.exp2(scale_grid.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)
