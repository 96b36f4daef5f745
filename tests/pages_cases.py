"""Batches of sequences over a pool whose pages some of them share."""
import numpy as np

from oracle import pages as op


def batch(seed, B, P, max_len, spare, share=0.3, extra=0):
    """(lengths, table, free stack, its count): sequences of up to max_len rows; with probability `share` one begins
    with full pages of the one before it.  `extra`: pages of the pool that nobody has and that are not on the stack."""
    rng = np.random.default_rng(seed)
    length = rng.integers(0, max_len + 1, B).astype(np.int32)
    max_pages = -(-max_len // P) + 1
    table = np.full((B, max_pages), -1, np.int32)
    pool = rng.permutation(B * max_pages + spare + extra).astype(np.int32)
    at = 0
    for b in range(B):
        n = op.held(length[b], P)
        same = 0
        if b and rng.random() < share:
            same = int(rng.integers(0, min(length[b], length[b - 1]) // P + 1))
            table[b, :same] = table[b - 1, :same]
        table[b, same:n] = pool[at:at + n - same]
        at += n - same
    pages = at + spare + extra  # the pool, numbered anew
    number = np.full(len(pool), -1, np.int64)
    number[pool[:pages]] = rng.permutation(pages)
    table = np.where(table >= 0, number[np.maximum(table, 0)], -1).astype(np.int32)
    free = np.full(pages, -1, np.int32)
    free[:spare] = number[pool[at:at + spare]]
    return length, table, free, spare


def cut_batch(seed, B, P, max_len, spare):
    """The same after a fork in which many rows became copies of others, and with half of the rows then cut back to any
    length: partly filled pages that other rows hold in full, or in part."""
    rng = np.random.default_rng(seed + 7)
    length, table, free, count = batch(seed, B, P, max_len, spare + 2 * B)
    r = op.fork(table, length, rng.integers(0, max(1, B // 3), B), free, count, P)
    assert r["report"][0] == 0
    n = r["lengths"]
    n = np.where(rng.random(B) < 0.5, rng.integers(0, n + 1), n).astype(np.int32)
    return n, r["table"], r["free"], r["free_left"]
