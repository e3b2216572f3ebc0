"""Microscaled 8-bit blocks from their definition, in numpy and 64 bits."""
import math

import numpy as np
import torch

# every e4m3 magnitude by its code: 2^-9 m below 2^-6, (1 + m / 8) 2^(E - 7) from there on
MAGS = np.array([(m * 2.0 ** -9 if E == 0 else (1 + m / 8) * 2.0 ** (E - 7))
                 for E in range(16) for m in range(8)][:127])


def scale_bytes(rows, K):
    return -(-rows // 128) * -(-K // 128) * 512


def tiles(grid, K):
    """Scale bytes [rows, K / 32] in tiles of 128 rows by 4 blocks, zeros outside."""
    rows = grid.shape[0]
    R, C = -(-rows // 128), -(-K // 128)
    out = np.zeros(R * C * 512, np.uint8)
    r, k = np.arange(rows)[:, None], np.arange(grid.shape[1])[None]
    out[((r // 128) * C + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4] = grid
    return out


def grid(scales, rows, K):
    """The scale bytes [rows, K / 32] of tiles."""
    C = -(-K // 128)
    r, k = np.arange(rows)[:, None], np.arange(K // 32)[None]
    return scales[((r // 128) * C + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4]


def exponents(top):
    """Per block maximum the least e with top <= 448 * 2^e, e >= -127 (by its definition)."""
    e = np.full(top.shape, -127)
    fine = np.isfinite(top) & (top > 0)
    guess = np.floor(np.log2(np.where(fine, top, 1.0))).astype(int) - 10
    for step in range(4):  # up from a start that is too low until the block fits
        guess = np.where(448.0 * np.exp2(guess.astype(np.float64)) < top, guess + 1, guess)
    return np.where(fine, np.maximum(guess, e), e)


def nearest(q):
    """Codes of float64 values of at most 448 (nearest, ties to the even code)."""
    a = np.abs(q)
    lower = np.clip(np.searchsorted(MAGS, a, side="right") - 1, 0, 126)
    upper = np.minimum(lower + 1, 126)
    down, up = a - MAGS[lower], MAGS[upper] - a
    code = np.where(down == up, lower + lower % 2, np.where(down < up, lower, upper))
    code = np.where(a >= 448.0, 126, code)
    return (code + 128 * np.signbit(q)).astype(np.uint8)


def quantize(x):
    """x float64 [rows, K] -> (codes uint8 [rows, K], scale bytes [rows, K / 32])."""
    rows, K = x.shape
    b = x.reshape(rows, K // 32, 32)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(top)
    e = exponents(top)
    q = np.where(bad[..., None], 0.0, b) / np.exp2(e.astype(np.float64))[..., None]
    return nearest(q).reshape(rows, K), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scale_grid):
    """Codes and scale bytes [rows, K / 32] -> float64 [rows, K]."""
    mag = np.append(MAGS, np.nan)[codes & 127]
    v = np.where(codes & 128, -mag, mag)
    s = np.where(scale_grid == 255, np.nan, np.exp2(scale_grid.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)


def across(codes, scale_grid):
    """The values of [rows, K] in blocks along the rows: codes [K, R], scale bytes [K, R / 32]."""
    v = values(codes, scale_grid).T
    short = -v.shape[1] % 32
    return quantize(np.concatenate([v, np.zeros((v.shape[0], short))], axis=1))


def held(rm, codes, scale_grid, device="cuda"):
    """The library's matrix of such codes and scales."""
    K = codes.shape[1]
    return rm.Mxfp8(torch.from_numpy(codes).view(torch.float8_e4m3fn).to(device),
                    torch.from_numpy(tiles(scale_grid, K)).to(device))


def shown(q):
    """-> (codes uint8 [rows, K], scale bytes [rows, K / 32], all scale bytes) of the library's."""
    K = q.codes.shape[-1]
    codes = q.codes.view(torch.uint8).reshape(-1, K).cpu().numpy()
    flat = q.scales.cpu().numpy()
    return codes, grid(flat, codes.shape[0], K), flat


def decoded(q):
    """The library's matrix in 64 bits, as a CUDA tensor of its shape."""
    codes, g, _ = shown(q)
    return torch.from_numpy(values(codes, g)).view(q.codes.shape).to(q.codes.device)


def random_codes(rng, rows, K, lo=118, hi=130):
    """Codes of every kind but NaN, and scales of some magnitudes."""
    codes = rng.integers(0, 127, (rows, K)) + 128 * rng.integers(0, 2, (rows, K))
    return codes.astype(np.uint8), rng.integers(lo, hi, (rows, K // 32)).astype(np.uint8)


def activation(name, z):
    """act(z) and its derivative, float64."""
    if name is None:
        return z, torch.ones_like(z)
    if name == "gelu":
        phi = 0.5 * torch.erfc(-z * math.sqrt(0.5))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    a, slope = (z, 1.0) if name == "silu" else (c * (z + 0.044715 * z ** 3),
                                               c * (1 + 3 * 0.044715 * z * z))
    p = torch.sigmoid(a)
    return z * p, p + z * p * torch.sigmoid(-a) * slope


ACTIVATIONS = [None, "silu", "gelu", "gelu_tanh"]


def step_of(v, dtype):
    """Half a step of `dtype` at v, its subnormals' included."""
    f = torch.finfo(dtype)
    return f.eps / 2 * v.abs() + f.smallest_normal * f.eps / 2


def check_held(q, want, slack):
    """q holds `want` (float64, the shape of its codes) in 8-bit blocks, each value of which the kernel
    may have seen off by `slack` before it was rounded: the scale is that of a maximum within its
    block's slack, and a code is off by half a step of its binade under that scale, and the slack."""
    codes, g, flat = shown(q)
    rows, K = codes.shape
    C = -(-K // 128)
    assert flat.size == scale_bytes(rows, K)
    want, slack = (t.reshape(rows, K).double().cpu().numpy() for t in (want, slack))
    assert np.array_equal(tiles(g, K), flat)  # zeros outside the matrix
    b, s = np.abs(want).reshape(rows, -1, 32), slack.reshape(rows, -1, 32)
    low, high = exponents(np.maximum(b - s, 0.0).max(-1)), exponents((b + s).max(-1))
    e = g.astype(int) - 127
    assert ((e >= low) & (e <= high)).all()
    scale = np.repeat(np.exp2(e.astype(np.float64)), 32, axis=1)
    got = values(codes, g)
    # half a step at the larger of the two magnitudes: 2^-4 of its power of two, 2^-10 at least
    near = np.maximum(np.abs(got), np.abs(want) + slack) / scale
    half = np.exp2(np.floor(np.log2(np.maximum(near, 2.0 ** -6))) - 4) * scale
    off = np.abs(got - want) - half - slack
    assert (off <= 1e-12 * scale).all(), float(off.max())
