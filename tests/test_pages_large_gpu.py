"""What a fork and a compaction refuse or leave alone, on tables on either side of the size up to which one launch takes
them: whole numbers, equal to the oracle's."""
import numpy as np
import pytest

from tests.pages_cases import batch
from tests.test_pages_gpu import check_compact, check_fork

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# table entries and pages that one launch takes: of a fork, of a compaction
FORK_IN_ONE, COMPACT_IN_ONE = 1 << 18, 1 << 17


def half_empty(large, extra=9):
    """Sequences of which every other is empty, so that a fork into these takes pages and releases none."""
    B, max_len = (1024, 3000) if large else (20, 2500)
    length, table, free, count = batch(3, B, 16, max_len, spare=B, share=0.0, extra=extra)
    assert (table.size + len(free) > FORK_IN_ONE) == large and (table.size + len(free) > COMPACT_IN_ONE) == large
    length[1::2] = 0
    length[0::2] = np.where(length[0::2] % 16, length[0::2], length[0::2] // 16 * 16 + 5)
    src = np.arange(B)
    src[1::2] = np.random.default_rng(4).permutation(np.arange(0, B, 2))
    return length, table, free, count, src


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("large", [False, True])
def test_fork_one_page_short(large, inplace):
    length, table, free, count, src = half_empty(large)
    need = check_fork(length, table, src, free, count, 16, inplace)["report"]
    assert need[:3] == [0, 0, len(length) // 2]  # none released
    need = need[2]
    for spare, status in ((need, 0), (need - 1, 3), (0, 3)):
        want = check_fork(length, table, src, free, spare, 16, inplace)
        assert want["report"][0] == status and want["free_left"] == (0 if status == 0 else spare)
        assert status == 0 or np.array_equal(want["lengths"], length)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("large", [False, True])
def test_fork_refused_on_the_device(large, inplace):
    length, table, free, count, src = half_empty(large)
    B = len(length)
    # pages go back, and more than the pool would be on the stack
    assert check_fork(length, table, np.full(B, -1), free, len(free), 16, inplace)["report"][0] == 3
    for bad in (B, B + 7, 2 ** 31 - 1):
        odd = src.copy()
        odd[B // 2] = bad
        assert check_fork(length, table, odd, free, count, 16, inplace)["report"][0] == 1
    far = length.copy()
    far[B - 2] = table.shape[1] * 16 + 1
    assert check_fork(far, table, src, free, count, 16, inplace)["report"][0] == 3
    # and both: the source is named
    assert check_fork(far, table, odd, free, count, 16, inplace)["report"][0] == 1


def with_odd_rows(large):
    length, table, free, count, src = half_empty(large)
    rng = np.random.default_rng(5)
    rows = np.argwhere(length >= 64)[:, 0]
    for value in (len(free), len(free) + 5, 2 ** 31 - 1, -1, -9, -2 ** 31):
        b = rng.choice(rows)
        table[b, rng.integers(0, length[b] // 16)] = value
        b = rng.choice(rows)
        table[b, length[b] // 16] = value  # the last page, filled in part
    length[1::4] = -rng.integers(1, 1000, len(length[1::4]))
    return length, table, free, count, src


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("large", [False, True])
def test_lengths_below_zero_and_foreign_pages(large, inplace):
    length, table, free, count, src = with_odd_rows(large)
    B = len(length)
    for s in (src, np.arange(B), np.full(B, -1), np.full(B, int(np.argmax(length))), np.roll(np.arange(B), 3)):
        assert check_fork(length, table, s, free, count, 16, inplace)["report"][0] == 0
    assert check_fork(length, table, src, free, 3, 16, inplace)["report"][0] == 3
    assert check_compact(length, table, len(free), 16, inplace)["report"][0] == 0


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("large", [False, True])
def test_compact_refused_on_the_device(large, inplace):
    length, table, free, *_ = half_empty(large, extra=40)
    assert check_compact(length, table, len(free), 16, inplace)["report"][:2] != [0, 0]
    for b in (0, len(length) // 2, len(length) - 1):
        far = length.copy()
        far[b] = table.shape[1] * 16 + 1
        want = check_compact(far, table, len(free), 16, inplace)
        assert want["report"] == [3, 0, 0, int(far[b])] and want["free_left"] is None
