"""The 4-bit cache format and the norm + rotation of rows, from their
definitions, in numpy and 64 bits: what the GPU tests compare with."""
from __future__ import annotations

import numpy as np

PAGE = 16
MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALES = np.array([b * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18) for b in range(0xE3)])


def _nearest(v, grid):
    """Index of the nearest grid value, ties to the even index, values past the end to the last."""
    i = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    below, above = v - grid[i - 1], grid[i] - v
    return np.where((below < above) | ((below == above) & ((i - 1) % 2 == 0)), i - 1, i)


def quantise(x):
    """(codes uint8 [..., D], scale bytes uint8 [..., D / 16]) of rows [..., D]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (-1, 16))
    nan = np.isnan(g).any(-1)
    a = np.where(np.isnan(g), 0.0, np.abs(g))
    byte = _nearest(np.minimum(a.max(-1) / 6.0, 1e30), SCALES)
    s = SCALES[byte][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(s > 0, a / s, 0.0)
    mag = _nearest(np.minimum(r, 1e30), MAGS)
    codes = mag | (np.signbit(g).astype(np.int64) << 3)
    return codes.reshape(x.shape).astype(np.uint8), np.where(nan, 0xFF, byte).astype(np.uint8)


def values(codes, scales):
    """float64 values of codes and scale bytes (bytes above 0xF8 are NaN, 0xF8 is infinite)."""
    c, b = codes.astype(np.int64), scales.astype(np.int64)
    s = np.where(b < 8, b * 2.0 ** -17, (8 + b % 8) * 2.0 ** (b // 8 - 18))
    s = np.where(b > 0xF8, np.nan, np.where(b == 0xF8, np.inf, s))
    v = MAGS[c & 7].reshape(c.shape[:-1] + (-1, 16))
    with np.errstate(invalid="ignore"):
        v = (v * s[..., None]).reshape(c.shape)
    return np.where(c >= 8, -v, v)


def places(D, is_v):
    """(code byte, nibble [16, D]; scale byte [16, D / 16]) of a block, from the header's text."""
    tok, col = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
    tok2, grp = np.meshgrid(np.arange(PAGE), np.arange(D // 16), indexing="ij")
    if not is_v:
        return tok * D // 2 + col // 2, col % 2, 8 * D + tok2 * D // 16 + grp
    hi, t, n = tok // 8, tok % 8 // 2, tok % 2
    g, p, i = col // (D // 8), col % (D // 8) // 8, col % 8
    hi2, t2, n2 = tok2 // 8, tok2 % 8 // 2, tok2 % 2
    return 512 * p + 16 * (4 * g + t) + 2 * i + hi, n, 8 * D + 4 * (4 * grp + t2) + 2 * hi2 + n2


def unpack(pool, is_v):
    """Pool bytes [blocks, Hkv, 9 D] to codes [blocks, 16, Hkv, D] and scale bytes [blocks, 16, Hkv, D / 16]."""
    D = pool.shape[-1] // 9
    at, nib, sc = places(D, is_v)
    codes = (pool[..., at] >> (4 * nib).astype(np.uint8)) & 15
    return np.ascontiguousarray(codes.transpose(0, 2, 1, 3)), np.ascontiguousarray(pool[..., sc].transpose(0, 2, 1, 3))


def pack(codes, scales, is_v):
    """The inverse of unpack."""
    nb, _, H, D = codes.shape
    at, nib, sc = places(D, is_v)
    pool = np.zeros((nb, H, 9 * D), np.uint8)
    c = codes.transpose(0, 2, 1, 3).astype(np.uint8)
    for n in (0, 1):
        m = nib == n
        pool[..., at[m]] |= c[..., m] << np.uint8(4 * n)
    pool[..., sc] = scales.transpose(0, 2, 1, 3)
    return pool


def pool_values(pool, is_v):
    return values(*unpack(pool, is_v))


def norm_rope(x, weight, eps, inv_freq, pos, mscale=1.0, interleaved=False):
    """Rows [rows, H, D] in float64: norm (weight not None), then rotation by pos * inv_freq."""
    x = np.asarray(x, np.float64).copy()
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if inv_freq is None:
        return x
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = mscale * np.cos(ang)[:, None, :], mscale * np.sin(ang)[:, None, :]
    r = 2 * len(inv_freq)
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    u, w = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = u * c - w * s, w * c + u * s
    return x
