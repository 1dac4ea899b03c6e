"""The 4-bit operators in 64 bits, from their formulas (numpy, CPU): the
reference of the 4-bit tests.  It shares nothing with the library."""
from __future__ import annotations

import numpy as np

BLOCK = {"mxfp4": 32, "nvfp4": 16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
_c = np.arange(127)
E4M3 = np.where(_c < 8, _c * 2.0**-9, (1 + _c % 8 / 8) * 2.0 ** (_c // 8 - 7.0))


def nearest(v, grid):
    """Index of the nearest grid value of v >= 0 (ties to the even index, beyond the last to it)."""
    v = np.minimum(v, grid[-1])
    hi = np.searchsorted(grid, v)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - v, v - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantize(x, fmt, t=None):
    """(codes, scale bytes) of a [M, K] float32 array: 4-bit codes [M, 32 ceil(K / 32)] one a
    byte, scale bytes [M, ceil(K / B)]."""
    B = BLOCK[fmt]
    M, K = x.shape
    Kp = -(-K // 32) * 32
    xb = np.zeros((M, Kp), np.float32)
    xb[:, :K] = x
    xb = xb.reshape(M, Kp // B, B)
    with np.errstate(all="ignore"):
        a = np.abs(xb).max(-1)                      # NaN propagates
        bad = ~np.isfinite(a)
        a = np.where(bad, np.float32(0), a)
        if fmt == "mxfp4":
            m, e = np.frexp(a.astype(np.float64))
            S = np.where(a > 0, np.clip(e - 1 - 2, -127, 127), -127)
            scale = (S + 127).astype(np.uint8)
            v = xb.astype(np.float64) * 2.0 ** -S[..., None].astype(np.float64)
        else:
            t32 = np.float32(1 if t is None else t)
            want = np.minimum((a / np.float32(6)) / t32, np.float32(448))  # fp32 divisions
            scale = nearest(want.astype(np.float64), E4M3).astype(np.uint8)
            d = E4M3[scale].astype(np.float32) * t32
            r = np.where(d > 0, np.float32(1) / np.where(d > 0, d, np.float32(1)), np.float32(0))
            r = np.minimum(r, np.finfo(np.float32).max).astype(np.float32)
            v = (xb * r[..., None]).astype(np.float64)                      # one fp32 rounding
        code = nearest(np.abs(np.where(bad[..., None], 0, v)), E2M1[:8])
    code = code + 8 * (np.signbit(xb) & ~bad[..., None])
    scale = np.where(bad, 0xFF if fmt == "mxfp4" else 0x7F, scale).astype(np.uint8)
    return code.astype(np.uint8).reshape(M, Kp), scale[:, : -(-K // B)]


def pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpack(codes):
    out = np.empty((codes.shape[0], 2 * codes.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = codes & 15, codes >> 4
    return out


def tile(scale):
    """[M, blocks] -> [ceil(M / 128), ceil(blocks / 4), 32, 16], zeros beyond."""
    M, nb = scale.shape
    out = np.zeros((-(-M // 128), -(-nb // 4), 32, 16), np.uint8)
    r, j = np.meshgrid(np.arange(M), np.arange(nb), indexing="ij")
    out[r // 128, j // 4, r % 32, (r % 128) // 32 * 4 + j % 4] = scale
    return out


def untile(tiles, M, nb):
    r, j = np.meshgrid(np.arange(M), np.arange(nb), indexing="ij")
    return tiles[r // 128, j // 4, r % 32, (r % 128) // 32 * 4 + j % 4]


def scale_values(scale, fmt):
    if fmt == "mxfp4":
        with np.errstate(all="ignore"):
            return np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    s = scale.astype(int)
    return np.where(s == 127, np.nan, E4M3[np.minimum(s, 126)])


def values(code, scale, fmt):
    """float64 values [M, columns] of codes (one a byte) and scale bytes, without a tensor scale."""
    B = BLOCK[fmt]
    full = np.zeros((code.shape[0], code.shape[1] // B))
    full[:, : scale.shape[1]] = scale_values(scale, fmt)
    return E2M1[code] * np.repeat(full, B, axis=1)


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))
