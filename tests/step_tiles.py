"""Cases of the paged attention that a lost, doubled or misplaced tile of keys cannot pass: keys and values are
constant over tiles of 128 keys, values are positive, so that outputs are means whose size every tile shapes, and
the reference is a sum over tiles."""
import numpy as np

from oracle import paged_step as step

TILE, P, T = 128, 64, 97  # keys of a tile, tokens of a page, different tiles in the pool
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


class Tiles:
    """Sequence b's tile i is tile (i + 7 b) % T of the pool.  Query head h is constant: 0, .5, 1 or -.5 in turn."""

    def __init__(self, lens, rows, Hq, Hkv, D, dtype):
        self.lens, self.rows, self.Hq, self.Hkv, self.D, self.dtype = lens, rows, Hq, Hkv, D, dtype
        c, h = np.arange(T)[:, None], np.arange(Hkv)
        level = step.E2M1[1 + (c * 5 + h * 3 + c // 7) % 7]  # [T, Hkv]
        high = (np.arange(D) // 16) == ((c + h) % (D // 16))[..., None]
        fill = lambda x: np.ascontiguousarray(np.broadcast_to(  # noqa: E731
            x[:, None, :, None, :], (T, TILE // P, Hkv, P, D)).reshape(-1, Hkv, P, D).astype(np.float32))
        self.pools = [step.make_pool(fill(np.broadcast_to(level[..., None], (T, Hkv, D)))),
                      step.make_pool(fill(np.where(high, 6.0, 1.5)))]
        k, v = [step.read_pool(p, D)[::TILE // P, :, 0] for p in self.pools]
        self.level, self.v = k[..., 0], v  # as the format holds them
        B, per = len(lens), TILE // P
        pages = max(1, max(-(-n // P) for n in lens))
        j, b = np.arange(pages), np.arange(B)[:, None]
        self.table = ((j // per + 7 * b) % T * per + j % per).astype(np.int32)
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.scale = 1.0 / D
        self.q = np.array([0.0, 0.5, 1.0, -0.5])[np.arange(Hq) % 4]

    def reference(self, b, without=(0, 0), twice=(0, 0)):
        """(out [rows, Hq, D], lse [rows, Hq]) of sequence b, whose tiles [without) are lost and [twice) counted twice."""
        n, keys, G = self.rows[b], self.lens[b], self.Hq // self.Hkv
        at = np.arange(max(1, -(-keys // TILE)))
        seen = np.clip(keys - n + 1 + np.arange(n), 0, None)[:, None]
        count = np.clip(seen - at * TILE, 0, TILE).astype(np.float64)  # [rows, tiles]
        count[:, without[0]:without[1]] = 0
        count[:, twice[0]:twice[1]] *= 2
        c = (at + 7 * b) % T
        out, lse = np.zeros((n, self.Hq, self.D)), np.zeros((n, self.Hq))
        for h in range(self.Hq):
            w = np.exp(self.scale * self.D * self.q[h] * self.level[c, h // G])
            total = count @ w
            with np.errstate(all="ignore"):
                out[:, h] = np.where(total[:, None] > 0, (count * w) @ self.v[c, h // G] / total[:, None], 0.0)
                lse[:, h] = np.log(total)
        return out, lse

    def bad(self, b, out, lse, want):
        """Outputs and lse of sequence b that are off by more than the arithmetic allows, counted.

        Heads with q = 0: every weight is the same power of two and every fp32 sum exact (multiples of half of
        it, fewer than 2^24 of them), so only the output's own rounding and the quotient's are left, and for
        lse the logarithm's of a number below 32 (2^-18).  Other heads: weights rounded to fp16, 2^-11; fp32
        sums of at most 32769 keys of one CTA, added 16 or more at a time, and of 608 pieces, 2^-23 each
        addition: 2^-11 and less for the output's two sums, 2^-13 for lse; scores of 6 at most, 2^-18."""
        half = HALF[self.dtype]
        flat = self.q == 0
        tol = np.where(flat, half + 2.0 ** -21, half + 2.0 ** -10)[:, None] * np.abs(want[0])
        low = np.where(flat, 2.0 ** -18, 2.0 ** -13)
        none = np.isneginf(want[1])
        with np.errstate(all="ignore"):
            far = ~(np.abs(lse - want[1]) <= low)
        return int((~(np.abs(out - want[0]) <= tol)).sum()), int(np.where(none, ~np.isneginf(lse), far).sum())


_rng = np.random.default_rng(48)
CASES = {
    # few rows: one item over all CTAs (joined in groups), some items, items of which a CTA holds several
    "one_head_64": ([320_011], [1], 1, 1, 64, "fp16"),
    "one_head_128": ([60_001], [1], 4, 1, 128, "fp16"),
    "rows_16": ([40_003], [16], 1, 1, 128, "bf16"),
    "rows_10": ([60_001], [10], 2, 1, 64, "fp16"),
    "rows_8": ([131_072], [8], 4, 1, 64, "bf16"),
    "long_4": ([131_073] * 4, [1] * 4, 32, 8, 128, "bf16"),
    "ragged_48": ([int(x) for x in _rng.integers(0, 8194, 48)], [1] * 48, 32, 32, 64, "fp16"),
    "drafts": ([int(x) for x in _rng.integers(5, 12006, 16)], [int(x) for x in _rng.integers(0, 6, 16)], 32, 8, 128, "bf16"),
    # many rows
    "rows_33": ([60_001], [33], 1, 1, 128, "fp16"),
    "rows_64": ([131_072], [16], 32, 8, 128, "bf16"),
    "rows_200": ([20_011], [200], 3, 1, 64, "fp16"),
    "chunk": ([8192], [1031], 8, 2, 128, "bf16"),
    # a prompt's chunk beside single tokens and drafts, as one call
    "mixed": ([34_816, 32_769, 1, 32_769, 0, 129, 20_000, 32_769], [2048, 1, 1, 1, 1, 0, 5, 1], 16, 4, 128, "bf16"),
    "mixed_64": ([300, 16_385, 16_385, 16_384, 40, 9_000], [300, 1, 1, 0, 33, 1], 8, 8, 64, "fp16"),
}
