"""The life of a cache's pages without a GPU: the oracle's invariants, and every refusal of the entry points (they
return before anything is enqueued)."""
import ctypes

import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from oracle import pages as op
from tests.pages_cases import batch
from zero_copy_offloaded_gb300 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return dkv.lib()


# ---- the oracle -------------------------------------------------------------------------

@pytest.mark.parametrize("seed", range(20))
def test_fork_keeps_every_sequence_and_every_page(seed):
    length, table, free, count = batch(seed, 9, 4, 50, spare=12)
    rng = np.random.default_rng(seed)
    src = rng.integers(-1, 9, 9)
    content = {}  # what a page holds: of the sequence's own pages, itself
    r = op.fork(table, length, src, free, count, 4)
    assert r["report"][0] == 0
    content = {int(to): int(frm) for frm, to in r["copies"] if to >= 0}
    seen_partial = {}
    for b in range(9):
        n = op.held(r["lengths"][b], 4)
        assert r["lengths"][b] == (length[src[b]] if src[b] >= 0 else 0)
        if src[b] >= 0:  # reads the same bytes
            assert [content.get(int(p), int(p)) for p in r["table"][b, :n]] == list(table[src[b], :n])
        if r["lengths"][b] % 4:
            assert int(r["table"][b, n - 1]) not in seen_partial  # nobody else appends there
            seen_partial[int(r["table"][b, n - 1])] = b
    now = {int(p) for b in range(9) for p in r["table"][b, :op.held(r["lengths"][b], 4)]}
    stack = [int(x) for x in r["free"][:r["free_left"]]]
    before = {int(p) for b in range(9) for p in table[b, :op.held(length[b], 4)]} | {int(x) for x in free[:count]}
    assert len(set(stack)) == len(stack) and not now & set(stack) and now | set(stack) == before


def test_fork_closed_forms():
    table = np.array([[5, 6, -1], [7, -1, -1]], np.int32)
    free = np.array([9, 8, -1, -1, -1, -1, -1, -1, -1, -1], np.int32)
    # both go on as the first, which keeps its half page; the second's page goes back
    r = op.fork(table, [6, 3], [0, 0], free, 2, 4)
    assert r["table"].tolist() == [[5, 6, -1], [5, 7, -1]] and r["copies"].tolist() == [[-1, -1], [6, 7]]
    assert r["free"][:3].tolist() == [9, 8, 7] and r["free_left"] == 2 and r["report"] == [0, 1, 1, 6]
    # they change places: nothing to copy
    r = op.fork(table, [6, 3], [1, 0], free, 2, 4)
    assert r["table"].tolist() == [[7, -1, -1], [5, 6, -1]] and r["report"] == [0, 0, 0, 6]
    # both end
    r = op.fork(table, [6, 3], [-1, -1], free, 2, 4)
    assert r["free"][:5].tolist() == [9, 8, 5, 6, 7] and r["free_left"] == 5


@pytest.mark.parametrize("seed", range(20))
def test_compact_leaves_no_holes(seed):
    length, table, free, count = batch(seed, 9, 4, 50, spare=12, share=0.5)
    r = op.compact(table, length, len(free), 4, len(free) // 2)
    live = {int(p) for b in range(9) for p in r["table"][b, :op.held(length[b], 4)]}
    assert live == set(range(r["report"][2]))
    assert sorted(r["free"][:r["free_left"]]) == list(range(r["report"][2], len(free)))
    back = {int(to): int(frm) for frm, to in r["moves"] if frm >= 0}
    for b in range(9):
        n = op.held(length[b], 4)
        assert [back.get(int(p), int(p)) for p in r["table"][b, :n]] == list(table[b, :n])


# ---- refusals ---------------------------------------------------------------------------

FORK = dict(table=4096, len=4096, src=4096, free=4096, count=4096, batch=4, max_pages=8, page_tokens=16, pages=64,
            table_out=8192, len_out=4096, left=4096, copies=4096, report=4096, ws=4096, size=1 << 20, stream=None)
COMPACT = dict(table=4096, len=4096, batch=4, max_pages=8, page_tokens=16, pages=64, table_out=8192, free=4096,
               left=4096, moves=4096, max_moves=32, report=4096, ws=4096, size=1 << 20, stream=None)


@pytest.mark.parametrize("change", [
    {"table": None}, {"len": None}, {"src": None}, {"free": None}, {"count": None}, {"table_out": None},
    {"len_out": None}, {"left": None}, {"copies": None}, {"report": None}, {"ws": None}, {"batch": 0}, {"batch": 1025},
    {"max_pages": 0}, {"max_pages": 1 << 27}, {"page_tokens": 0}, {"page_tokens": 24}, {"page_tokens": 8192},
    {"pages": 0}, {"pages": 1 << 27}, {"ws": 4096 + 16}, {"copies": 4100}, {"size": 100}])
def test_fork_refuses(L, change):
    assert L.dkv_pages_fork(*{**FORK, **change}.values()) == 1
    assert dkv.dkv_last_error()


@pytest.mark.parametrize("change", [
    {"table": None}, {"len": None}, {"free": None}, {"table_out": None}, {"left": None}, {"moves": None},
    {"report": None}, {"ws": None}, {"batch": 0}, {"batch": 1025}, {"max_pages": 0}, {"page_tokens": 3}, {"pages": 0},
    {"max_moves": 31}, {"ws": 4096 + 128}, {"moves": 4100}, {"size": 100}])
def test_compact_refuses(L, change):
    assert L.dkv_pages_compact(*{**COMPACT, **change}.values()) == 1
    assert dkv.dkv_last_error()


@pytest.mark.parametrize("pairs,n,pools,count", [
    (None, 4, (4096, 4096, 64, 8, 8), 1), (4096, -1, (4096, 4096, 64, 8, 8), 1), (4100, 4, (4096, 4096, 64, 8, 8), 1),
    (4096, 4, None, 1), (4096, 4, (4096, 4096, 64, 8, 8), 0), (4096, 4, (0, 4096, 64, 8, 8), 1),
    (4096, 4, (4096, 0, 64, 8, 8), 1), (4096, 4, (4096, 4096, 0, 8, 8), 1), (4096, 4, (4096, 4096, 66, 8, 8), 1),
    (4096, 4, (4097, 4096, 64, 8, 8), 1), (4096, 4, (4096, 4098, 64, 8, 8), 1), (4096, 4, (4096, 4096, 64, 0, 8), 1),
    (4096, 4, (4096, 4096, 64, 8, -1), 1), (4096, 4, (4096, 4096, (1 << 30) + 4, 8, 8), 1), (4096, 1 << 31, (4096, 4096, 64, 8, 8), 1)])
def test_copy_refuses(L, pairs, n, pools, count):
    packed = ctypes.create_string_buffer(dkv._PAGE_POOL.pack(*pools)) if pools else None
    n = n if n < 1 << 31 else -(1 << 31)
    assert L.dkv_pages_copy(pairs, n, ctypes.addressof(packed) if packed else None, count, None) == 1


def test_no_pairs_are_nothing_to_do(L):
    packed = ctypes.create_string_buffer(dkv._PAGE_POOL.pack(4096, 4096, 64, 8, 8))
    assert L.dkv_pages_copy(None, 0, ctypes.addressof(packed), 1, None) == 0


def test_workspace(L):
    assert dkv.dkv_pages_workspace(0, 8, 64) == dkv.dkv_pages_workspace(1025, 8, 64) == 0
    assert dkv.dkv_pages_workspace(4, 0, 64) == dkv.dkv_pages_workspace(4, 8, 0) == 0
    # two marks or a mark and a rank for each page, a row each, the old table
    assert dkv.dkv_pages_workspace(4, 8, 64) >= 64 * 5 + 4 * 16 + 4 * 8 * 4
    assert dkv.dkv_pages_workspace(1024, 1 << 16, 1 << 20) >= (5 << 20) + (1 << 28)


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="current CUDA device"):
        dkv.dkv_pages_fork(i(4, 8), i(4), i(4), i(64), i(1), 16, i(4, 8), i(4), i(1), i(4, 2), i(4))
    with pytest.raises(ValueError, match="page_table is"):
        dkv.dkv_pages_fork(i(32), i(4), i(4), i(64), i(1), 16, i(4, 8), i(4), i(1), i(4, 2), i(4))
    with pytest.raises(ValueError, match="moves"):
        dkv.dkv_pages_compact(i(4, 8), i(4), 16, i(4, 8), i(64), i(1), i(64), i(4))
    with pytest.raises(ValueError, match="pairs"):
        dkv.dkv_pages_copy(i(4), [i(8, 4)])
    with pytest.raises(ValueError, match="1 pools into 2"):
        dkv.dkv_pages_copy(i(4, 2), [i(8, 4)], [i(8, 4)] * 2)
    with pytest.raises(ValueError, match="does not go into"):
        dkv.dkv_pages_copy(i(4, 2), [i(8, 4)], [i(8, 5)])
    with pytest.raises(ValueError, match="contiguous"):
        dkv.dkv_pages_copy(i(4, 2), [i(8, 4).t()])
