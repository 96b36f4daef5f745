"""Sequences that are cut back to a page that others hold, without a GPU: what the oracle of a fork makes of them."""
import numpy as np
import pytest

from oracle import pages as op
from tests.pages_cases import cut_batch


def test_a_cut_row_gets_a_page_of_its_own():
    # both go on as the first, which ends with its second page
    table = np.array([[0, 1, -1], [2, -1, -1]], np.int32)
    free = np.array([3, 4, 5, 6, 7, -1, -1, -1], np.int32)
    r = op.fork(table, [32, 5], [0, 0], free, 5, 16)
    assert r["table"].tolist() == [[0, 1, -1], [0, 1, -1]]
    # the second is cut back to 30 rows: it would append to a page of the first
    again = op.fork(r["table"], [32, 30], [0, 1], r["free"], r["free_left"], 16)
    assert again["table"].tolist() == [[0, 1, -1], [0, 2, -1]] and again["copies"].tolist() == [[-1, -1], [1, 2]]
    assert again["report"] == [0, 0, 1, 32]
    # both are: the lower one keeps it; and one that ends leaves it to the other
    again = op.fork(r["table"], [31, 30], [0, 1], r["free"], r["free_left"], 16)
    assert again["table"].tolist() == [[0, 1, -1], [0, 2, -1]]
    again = op.fork(r["table"], [32, 30], [-1, 1], r["free"], r["free_left"], 16)
    assert again["table"].tolist()[1] == [0, 1, -1] and again["report"] == [0, 0, 0, 30]
    # a full page that nobody fills in part stays shared
    again = op.fork(r["table"], [32, 16], [0, 1], r["free"], r["free_left"], 16)
    assert again["report"] == [0, 0, 0, 32]


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("seed", range(20))
def test_no_page_that_is_appended_to_has_two_holders(seed, same):
    B, P = 12, 4
    length, table, free, count = cut_batch(seed, B, P, 50, spare=40)
    src = np.arange(B) if same else np.random.default_rng(seed).integers(-1, B, B)
    r = op.fork(table, length, src, free, count, P)
    assert r["report"][0] == 0
    rows = [list(map(int, r["table"][b, :op.held(r["lengths"][b], P)])) for b in range(B)]
    was = {int(to): int(frm) for frm, to in r["copies"] if to >= 0}
    for b in range(B):
        if src[b] >= 0:  # reads the same bytes
            assert [was.get(x, x) for x in rows[b]] == list(table[src[b], :len(rows[b])])
        if r["lengths"][b] % P:
            assert sum(rows[b][-1] in other for other in rows) == 1
    stack = [int(x) for x in r["free"][:r["free_left"]]]
    now = {x for row in rows for x in row}
    before = {int(p) for b in range(B) for p in table[b, :op.held(length[b], P)]} | {int(x) for x in free[:count]}
    assert len(set(stack)) == len(stack) and not now & set(stack) and now | set(stack) == before
    # copies come from pages that keep their bytes: none of them is the target of another copy
    assert not set(was) & set(was.values()) and len(was) == sum(r["copies"][:, 1] >= 0)
