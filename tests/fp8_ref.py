"""The 8-bit cache format and its append, from their definitions, in numpy and
64 bits: what the GPU tests compare with."""
from __future__ import annotations

import numpy as np

PAGE = 16


def _e4m3():
    v = []
    for c in range(128):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


MAGS = _e4m3()          # of the codes 0 .. 127; 127 is no number of the format
FINITE = MAGS[:127]
MAX = 448.0
assert FINITE[-1] == MAX


def scale(b):
    b = np.asarray(b, np.int64)
    return np.where(b > 0, 2.0 ** (b - 127.0), 0.0)


def exponent(amax):
    """Biased exponent of the smallest scale by which amax fits, at most 2^119."""
    out = np.zeros(np.shape(amax), np.int64)
    for i, a in np.ndenumerate(np.asarray(amax, np.float64)):
        if a > 0:
            out[i] = next((b for b in range(1, 247) if a <= MAX * 2.0 ** (b - 127)), 246)
    return out


def codes_of(x, b):
    """Codes of x (no NaN) under the biased exponents b (broadcast): nearest, ties to the even code, saturating."""
    x = np.asarray(x, np.float64)
    s = np.broadcast_to(scale(b), x.shape)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(s > 0, np.abs(x) / s, 0.0)
    r = np.minimum(np.where(np.isnan(r), 0.0, r), MAX)
    i = np.clip(np.searchsorted(FINITE, r), 1, 126)
    below, above = r - FINITE[i - 1], FINITE[i] - r
    i = np.where((below < above) | ((below == above) & ((i - 1) % 2 == 0)), i - 1, i)
    return (i | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)


def values_of(codes, b):
    c = codes.astype(np.int64)
    v = MAGS[c & 127] * np.broadcast_to(scale(b), codes.shape)
    return np.where(c >= 128, -v, v)


def places(D):
    """Byte of (token, column) in a block, from the header's text."""
    t, col = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
    return t * D + 16 * ((col // 16) ^ (((t & 6) ^ ((t & 1) << 2)) % (D // 16))) + col % 16


def unpack(pool):
    """Pool bytes [blocks, H, 16 D + 16] to codes [blocks, 16, H, D], exponents [blocks, H] and NaN masks [blocks, H]."""
    D = pool.shape[-1] // 16 - 1
    codes = pool[..., places(D)]
    word = pool[..., 16 * D:].astype(np.int64)
    return np.ascontiguousarray(codes.transpose(0, 2, 1, 3)), word[..., 0], word[..., 2] | word[..., 3] << 8


def pack(codes, b, mask, old=None):
    nb, _, H, D = codes.shape
    pool = np.zeros((nb, H, 16 * D + 16), np.uint8) if old is None else old.copy()
    pool[..., places(D)] = codes.transpose(0, 2, 1, 3)
    pool[..., 16 * D] = b
    pool[..., 16 * D + 1] = 0
    pool[..., 16 * D + 2], pool[..., 16 * D + 3] = np.asarray(mask) & 255, np.asarray(mask) >> 8
    return pool


def pool_values(pool):
    """[blocks, 16, H, D] in float64, tokens with a NaN all NaN."""
    c, b, m = unpack(pool)
    v = values_of(c, b[:, None, :, None])
    nan = (m[:, None, :] >> np.arange(PAGE)[None, :, None] & 1).astype(bool)
    return np.where(nan[..., None], np.nan, v)


def write_page(block, new, kept):
    """One block [16 D + 16] after new rows {slot: row [D]} come in and the slots `kept` stay.  Returns (block, rows as held)."""
    D = block.shape[-1] // 16 - 1
    c, b0, m0 = (x[0] for x in unpack(block[None, None]))
    c, b0, m0 = c[:, 0], int(b0[0]), int(m0[0])
    rows = {t: np.asarray(x, np.float64) for t, x in new.items()}
    nan = {t for t, x in rows.items() if np.isnan(x).any()}
    clean = {t: np.where(np.isnan(x), 0.0, x) for t, x in rows.items()}
    b = int(exponent(max(np.abs(x).max() for x in clean.values())))
    mask = sum(1 << t for t in nan)
    if kept:
        b = max(b, b0)
        mask |= m0 & sum(1 << t for t in kept)
        if b > b0 > 0:
            for t in kept:
                c[t] = codes_of(np.where(c[t] >= 128, -1.0, 1.0) * MAGS[c[t] & 127] * 2.0 ** (b0 - b), 127)
    for t, x in clean.items():
        # (a NaN's code is a plain 0)
        c[t] = np.where(np.isnan(rows[t]), 0, codes_of(x, b))
    held = {t: np.full(D, np.nan) if t in nan else values_of(c[t], b) for t in rows}
    return pack(c[None, :, None], np.array([[b]]), np.array([[mask]]), block[None, None])[0, 0], held


def append(pool, table, seq_info, rows, ring_rows=0):
    """Valid segments' rows [rows, H, D] into pool [blocks, H, 16 D + 16] in place; the rows as held.

    The segments that write one page of one column write it together, a later
    one's rows before an earlier one's."""
    H = pool.shape[1]
    held = np.full(rows.shape, 9.0)
    pages = {}  # (col, table page) -> {slot: row}
    for q0, n, col, kend in np.asarray(seq_info).tolist():
        for i in range(n):
            p = kend - n + i
            at = p % ring_rows if ring_rows else p
            pages.setdefault((col, at // PAGE), {})[at % PAGE] = q0 + i
    for (col, tp), slots in pages.items():
        block = int(table[col, tp])
        kept = [t for t in range(PAGE) if t not in slots and (ring_rows or t < max(slots))]
        for h in range(H):
            pool[block, h], out = write_page(pool[block, h], {t: rows[r, h] for t, r in slots.items()}, kept)
            for t, r in slots.items():
                held[r, h] = out[t]
    return held
