"""The device-side step in plain numpy: page planning, head norms + rotation + 4-bit
append, and attention over a 4-bit paged cache.  Shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values() -> np.ndarray:
    """The values of the 127 codes 0x00..0x7e (0x7f is NaN)."""
    c = np.arange(127)
    e, m = c >> 3, (c & 7) / 8.0
    return np.where(e == 0, m * 2.0 ** -6, (1 + m) * 2.0 ** (e - 7.0))


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Codes of x >= 0: to nearest, ties to the even code, saturating at 448."""
    v = e4m3_values()
    x = np.minimum(np.asarray(x, np.float64), 448.0)
    lo = np.clip(np.searchsorted(v, x, side="right") - 1, 0, 125)
    below, above = x - v[lo], v[lo + 1] - x
    up = (above < below) | ((above == below) & (lo % 2 == 1))
    return (lo + up).astype(np.uint8)


def from_e4m3(c: np.ndarray) -> np.ndarray:
    v = np.concatenate([e4m3_values(), [np.nan]])
    return v[c & 0x7F] * np.where(c & 0x80, -1.0, 1.0)


def to_e2m1(x: np.ndarray) -> np.ndarray:
    """4-bit codes of x: to nearest, ties to the even code, saturating at 6."""
    a = np.minimum(np.abs(np.asarray(x, np.float64)), 6.0)
    lo = np.clip(np.searchsorted(E2M1, a, side="right") - 1, 0, 6)
    below, above = a - E2M1[lo], E2M1[lo + 1] - a
    up = (above < below) | ((above == below) & (lo % 2 == 1))
    return ((lo + up) | (np.signbit(x).astype(np.int64) << 3)).astype(np.uint8)


def from_e2m1(c: np.ndarray) -> np.ndarray:
    return E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)


def quantise(y: np.ndarray):
    """Codes [..., D] and scale codes [..., D/16] of fp32 rows y, as the format defines them."""
    b = np.asarray(y, np.float32).reshape(*y.shape[:-1], -1, 16)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(amax)
    sc = to_e4m3(np.where(bad, np.float32(0), amax) / np.float32(6))
    s = from_e4m3(sc).astype(np.float32)
    with np.errstate(all="ignore"):
        t = np.where((s > 0)[..., None] & ~bad[..., None], b / s[..., None], np.float32(0))
    code = to_e2m1(t)
    return code.reshape(y.shape), np.where(bad, 0x7F, sc).astype(np.uint8)


def dequantise(code: np.ndarray, scale: np.ndarray) -> np.ndarray:
    b = from_e2m1(code).reshape(*code.shape[:-1], -1, 16) * from_e4m3(scale)[..., None]
    return b.reshape(code.shape)


def pool_views(pool: np.ndarray, D: int):
    """(codes [pages, Hkv, P, D/2], scales [pages, Hkv, P, D/16]) views of a uint8 pool."""
    pages, hkv, nbytes = pool.shape
    P = nbytes * 16 // (9 * D)
    cut = P * D // 2
    return pool[:, :, :cut].reshape(pages, hkv, P, D // 2), pool[:, :, cut:].reshape(pages, hkv, P, D // 16)


def make_pool(values: np.ndarray) -> np.ndarray:
    """A pool that holds values [pages, Hkv, P, D] quantised."""
    code, scale = quantise(values)
    pages, hkv, P, D = values.shape
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    return np.ascontiguousarray(np.concatenate(
        [packed.reshape(pages, hkv, -1), scale.reshape(pages, hkv, -1)], -1))


def read_pool(pool: np.ndarray, D: int) -> np.ndarray:
    """[pages, Hkv, P, D] values of a pool."""
    raw, scale = pool_views(pool, D)
    code = np.stack([raw & 15, raw >> 4], -1).reshape(*raw.shape[:-1], D)
    return dequantise(code, scale)


def plan(lengths, new, table, free, free_count, P, max_rows):
    """One step planned in a loop over sequences; returns a dict (inputs are not changed)."""
    B, max_pages = table.shape
    table, free = table.copy(), free.copy()
    lengths = np.maximum(lengths, 0)
    held = [-(-int(n) // P) for n in lengths]
    stack = [int(x) for x in free[:free_count]]
    kv, ok = [], True
    for b in range(B):
        k = 0 if new[b] < 0 else int(lengths[b]) + int(new[b])
        ok &= int(lengths[b]) <= max_pages * P and k <= max_pages * P
        kv.append(k)
    rows = sum(int(n) for n in new if n > 0)
    need = sum(-(-kv[b] // P) - held[b] for b in range(B) if new[b] >= 0)
    back = sum(held[b] for b in range(B) if new[b] < 0)
    ok &= rows <= max_rows and need <= free_count + back and free_count + back <= len(free)
    pos, slot = np.zeros(max_rows, np.int32), np.full(max_rows, -1, np.int32)
    start = np.zeros(B + 1, np.int32)
    if not ok:
        return dict(table=table, free=free, row_start=start, pos=pos, slot=slot,
                    kv_len=lengths.astype(np.int32), free_left=free_count,
                    report=[3, 0, 0, int(lengths.max())])
    for b in range(B):
        if new[b] < 0:
            stack += [int(x) for x in table[b, :held[b]]]
    free[:len(stack)] = stack
    r = 0
    for b in range(B):
        if new[b] >= 0:
            for c in range(held[b], -(-kv[b] // P)):
                table[b, c] = stack.pop()
            for t in range(int(new[b])):
                at = int(lengths[b]) + t
                page = int(table[b, at // P])
                pos[r], slot[r] = at, page * P + at % P if 0 <= page < len(free) else -1
                r += 1
        start[b + 1] = r
    return dict(table=table, free=free, row_start=start, pos=pos, slot=slot,
                kv_len=np.array(kv, np.int32), free_left=len(stack), report=[0, rows, need, max(kv)])


def turn(x, gamma, eps, cos_sin, pos, inter):
    """Norm and rotation of x [rows, heads, D] (fp32 values): fp32 with each operation rounded,
    the mean in 64 bits.  Returns (result, the magnitude that each element's rounding goes by)."""
    f = np.float32
    y = np.asarray(x, f)
    if gamma is not None:
        ms = (y.astype(np.float64) ** 2).mean(-1, keepdims=True) + float(f(eps))
        with np.errstate(all="ignore"):
            y = (y * (1.0 / np.sqrt(ms)).astype(f)).astype(f) * np.asarray(gamma, f)
    mag = np.abs(y)
    if cos_sin is None:
        return y, mag
    half = cos_sin.shape[1] // 2
    c, s = cos_sin[pos, :half][:, None], cos_sin[pos, half:][:, None]
    i = slice(0, 2 * half, 2) if inter else slice(0, half)
    j = slice(1, 2 * half, 2) if inter else slice(half, 2 * half)
    a, b = y[..., i], y[..., j]
    out, mag = y.copy(), mag.copy()
    out[..., i] = (a * c).astype(f) - (b * s).astype(f)
    out[..., j] = (b * c).astype(f) + (a * s).astype(f)
    mag[..., i] = np.abs(a * c) + np.abs(b * s)
    mag[..., j] = np.abs(b * c) + np.abs(a * s)
    return out, mag


def attend(q, k_vals, v_vals, table, kv_len, row_start, scale, v_scale=1.0):
    """fp64 attention of q [rows, Hq, D] over pool values [pages, Hkv, P, D].  Returns a dict: out,
    lse, and what error bounds need: wabs = sum w|v|, vabs = sum |v|, smax = the largest
    scale * sum |q k| of a row, keys = keys seen."""
    N, Hq, D = q.shape
    pages, Hkv, P, _ = k_vals.shape
    G = Hq // Hkv
    r = {n: np.zeros((N, Hq, D)) for n in ("out", "wabs", "vabs")}
    r["lse"], r["smax"], r["keys"] = np.zeros((N, Hq)), np.zeros((N, Hq)), np.zeros((N, Hq))
    r["live"] = np.zeros(N, bool)
    for b, kv in enumerate(kv_len):
        n = row_start[b + 1] - row_start[b]
        at = np.arange(kv)
        pg = table[b, at // P]
        ok = (pg >= 0) & (pg < pages)
        for i in range(n):
            row = row_start[b] + i
            r["live"][row] = True
            see = ok & (at <= kv - n + i)
            sl = pg[see], at[see] % P
            for h in range(Hq):
                k, v = k_vals[sl[0], h // G, sl[1]], v_vals[sl[0], h // G, sl[1]]
                if len(k) == 0:
                    r["lse"][row, h] = -np.inf
                    continue
                s = scale * (k @ q[row, h])
                m = s.max()
                w = np.exp(s - m)
                l = w.sum()
                w /= l
                r["lse"][row, h] = m + np.log(l)
                r["out"][row, h] = v_scale * (w @ v)
                r["wabs"][row, h] = abs(v_scale) * (w @ np.abs(v))
                r["vabs"][row, h] = abs(v_scale) * np.abs(v).sum(0)
                r["smax"][row, h] = abs(scale) * (np.abs(k) @ np.abs(q[row, h])).max()
                r["keys"][row, h] = len(k)
    return r
