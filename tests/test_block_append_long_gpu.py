"""Long appends of whole blocks, where a warp takes several heads of a block one after the other: the oracle's bytes and
scales, equal."""
import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from tests.test_block_append_gpu import check, filled, rows_of, slots_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# rows times heads decide how many heads: 2 for the first of each head size, 4 for the others, whose heads they divide or not
@pytest.mark.parametrize("rows,Hkv,D,dtype,P", [
    (4096, 5, 128, "bf16", 16), (4096, 8, 128, "fp16", 64), (2050, 18, 128, "bf16", 32),
    (8192, 9, 64, "bf16", 64), (8200, 17, 64, "fp16", 16)])
@pytest.mark.parametrize("mix", ["one", "many"])
def test_whole_blocks_of_many_heads(rows, Hkv, D, dtype, P, mix):
    """One sequence, or many of 7 to 70 rows beside short ones: blocks begun and continued in the middle, half of
    the latter with a scale that has to grow."""
    rng = np.random.default_rng(31)
    lens = [rows - 40, 33, 7]
    if mix == "many":
        lens = []
        while sum(lens) < rows:
            lens.append(int(rng.choice([1, 5, 6, 7, 8, 15, 16, 17, 30, 70])))
    slot, pages = slots_of(32, lens, P)
    _, k, v = rows_of(33, len(slot), 1, Hkv, D, dtype)
    pos = rng.integers(0, 300, len(slot)).astype(np.int32)
    table = dkv.rope_table(300, D // 2, device="cpu").numpy()
    pools = filled(34, pages, Hkv, P, D)
    for _, s in pools:  # some blocks hold small values, some large ones
        s *= np.exp2(rng.integers(-12, 12, s.shape)).astype(np.float32)
    check(None, k, v, slot, pos, table, pools, norm=True, dtype=dtype)
