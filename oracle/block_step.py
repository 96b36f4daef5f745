"""The 8-bit cache with block scales in plain numpy: E4M3 codes, a power-of-two scale for each 16 tokens of a page and
head that grows with what is appended.  Shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

from .paged_step import e4m3_values, to_e4m3

BLOCK = 16


def encode(x):
    """E4M3 codes of numbers of at most 448: to nearest, ties to the even code; NaN for what is not finite."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    code = to_e4m3(np.where(fine, np.abs(x), 0.0)) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(fine, code, 0x7F).astype(np.uint8)


def decode(code):
    code = np.asarray(code, np.uint8)
    v = np.concatenate([e4m3_values(), [np.nan]])
    return v[code & 0x7F] * np.where(code & 0x80, -1.0, 1.0)


def scale_for(top):
    """The smallest power of two s >= 2^-64 with top <= 448 s."""
    top = np.asarray(top, np.float64)
    s = np.full(top.shape, 2.0 ** -64)
    for _ in range(190):
        s = np.where(top > 448 * s, 2 * s, s)
    return s


def values(pool, scales):
    """[pages, Hkv, P, D] of codes [pages, Hkv, P, D] and scales [pages, Hkv, P / 16]."""
    with np.errstate(invalid="ignore"):
        return decode(pool) * np.repeat(scales.astype(np.float64), BLOCK, -1)[..., None]


def make_pool(y):
    """(codes, scales) that hold y [pages, Hkv, P, D], each block written at once."""
    pages, hkv, P, D = y.shape
    s = scale_for(np.abs(y).reshape(pages, hkv, P // BLOCK, -1).max(-1))
    return encode(y / np.repeat(s, BLOCK, -1)[..., None]), s.astype(np.float32)


def append(y, slot, pool, scales):
    """Rows y [N, Hkv, D] (fp32 values) appended to copies of pool and scales.  Returns (pool, scales, what
    the cache then holds of each row)."""
    pool, scales = pool.copy(), scales.copy()
    pages, hkv, P, D = pool.shape
    held = np.zeros(y.shape)
    blocks = {}
    for i, s in enumerate(slot):
        if 0 <= s < pages * P:
            blocks.setdefault(int(s) // BLOCK, []).append(i)
    for block, rows in blocks.items():
        page, lo = block * BLOCK // P, block * BLOCK % P
        first = any(slot[i] % BLOCK == 0 for i in rows)
        for h in range(hkv):
            x = y[rows, h].astype(np.float64)
            top = np.abs(x[np.isfinite(x)]).max(initial=0.0)
            old = float(scales[page, h, lo // BLOCK])
            if first or not (0 < old < np.inf):
                old = 0.0
            s = max(float(scale_for(top)), old)
            if s > old > 0:
                at = pool[page, h, lo:lo + BLOCK]
                # one product rounded to fp32, then to E4M3
                pool[page, h, lo:lo + BLOCK] = encode((decode(at) * np.float64(np.float32(old / s))).astype(np.float32))
            scales[page, h, lo // BLOCK] = s
            for i in rows:
                with np.errstate(invalid="ignore"):
                    c = encode((y[i, h].astype(np.float64) / s).astype(np.float32))
                pool[page, h, int(slot[i]) % P] = c
                held[i, h] = decode(c) * s
    return pool, scales, held
