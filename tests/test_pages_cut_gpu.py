"""Sequences that are cut back to a page that others hold, on the GPU: the fork's tables against the oracle, and appends
behind it that leave the others' rows alone."""
import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from tests.pages_cases import cut_batch
from tests.test_pages_gpu import check_fork, i32, sources

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

IN_ONE = 1 << 18  # table entries and pages that a fork takes in one launch


@pytest.mark.parametrize("B,P,max_len", [(2, 4, 30), (9, 16, 300), (64, 16, 3000), (700, 4, 400), (1024, 16, 200), (512, 16, 12000)])
@pytest.mark.parametrize("kind", ["same", "mixed", "one", "turn", "end"])
@pytest.mark.parametrize("inplace", [False, True])
def test_fork_of_cut_rows(B, P, max_len, kind, inplace):
    length, table, free, count = cut_batch(B + P, B, P, max_len, spare=2 * B)
    assert (table.size + len(free) > IN_ONE) == (max_len == 12000)
    want = check_fork(length, table, sources(B, B, kind), free, count, P, inplace)
    assert want["report"][0] == 0 and (kind != "same" or B < 64 or want["report"][2] > 0)


@pytest.mark.parametrize("large", [False, True])
def test_too_few_pages_for_cut_rows(large):
    B, P, max_len = (512, 16, 12000) if large else (64, 16, 3000)
    length, table, free, count = cut_batch(3, B, P, max_len, spare=2 * B)
    assert (table.size + len(free) > IN_ONE) == large
    need = check_fork(length, table, np.arange(B), free, count, P)["report"][2]
    assert need > 0
    for inplace in (False, True):
        assert check_fork(length, table, np.arange(B), free, need, P, inplace)["report"][0] == 0
        assert check_fork(length, table, np.arange(B), free, need - 1, P, inplace)["report"][0] == 3


def test_appends_behind_a_cut_leave_the_others_alone():
    """Two sequences share two full pages; the second is cut back into the second page, forked onto itself and appended to,
    with larger values than the block holds, so that its scale grows."""
    B, P, Hkv, D, pages = 2, 16, 2, 64, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = lambda n, size=1.0: (size * torch.randn((n, Hkv, D), generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    pools = [torch.zeros((pages, Hkv, P, D), dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.ones((pages, Hkv, 1), device="cuda") for _ in "kv"]
    table, free, count = i32([[0, 1, -1], [0, 1, -1]]), i32([7, 6, 5, 4, 3, 2, -1, -1]), i32([6])
    every = torch.arange(32, dtype=torch.int32, device="cuda")
    k, v = rows(32), rows(32)
    dkv.dkv_block_append(None, k, v, every, every, *pools, *scales)
    had = [t[:2].clone() for t in (*pools, *scales)]
    length, report, copies = i32([32, 30]), i32([0] * 4), i32([[0, 0]] * B)
    dkv.dkv_pages_fork(table, length, i32([0, 1]), free, count, P, table, length, count, copies, report)
    dkv.dkv_pages_copy(copies, [*pools, *scales])
    start, pos, slot, kv, left = i32([0] * 3), i32([0] * 5), i32([0] * 5), i32([0, 0]), i32([0])
    dkv.dkv_step_plan(length, i32([0, 5]), table, free, count, P, start, pos, slot, kv, left, report)
    assert int(report[0]) == 0 and kv.tolist() == [32, 35]
    dkv.dkv_block_append(None, rows(5, 100.0), rows(5, 100.0), pos, slot, *pools, *scales)
    for now, was in zip((*pools, *scales), had):
        assert torch.equal(now[:2], was)  # the first sequence
    page = int(table[1, 1])
    assert page not in (0, 1) and copies.tolist() == [[-1, -1], [1, page]]
    for pool, scale, old in zip(pools, scales, (k, v)):  # and the second still has its 30 rows, to the grown scale's step
        held = pool[page].view(torch.float8_e4m3fn).float() * scale[page][..., None]
        want = old[16:30].float().transpose(0, 1)
        assert torch.all((held[:, :14] - want).abs() <= want.abs() * 2.0 ** -3 + scale[page][..., None] * 2.0 ** -9)
