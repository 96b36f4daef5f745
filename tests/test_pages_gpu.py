"""The life of a cache's pages on the GPU against the oracle: whole numbers and bytes, equal."""
import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from oracle import pages as op
from tests.pages_cases import batch

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def host(d):
    return {k: v.cpu().numpy() for k, v in d.items()}


def run_fork(length, table, src, free, count, P, inplace=False, workspace=None):
    B = len(length)
    d = dict(table=i32(table), lengths=i32(length), src=i32(src), free=i32(free), count=i32([count]),
             out=i32(np.full_like(table, 77)), len_out=i32([77] * B), left=i32([77]), copies=i32(np.full((B, 2), 77)),
             report=i32([77] * 4))
    if inplace:
        d["out"], d["len_out"], d["left"] = d["table"], d["lengths"], d["count"]
    dkv.dkv_pages_fork(d["table"], d["lengths"], d["src"], d["free"], d["count"], P, d["out"], d["len_out"], d["left"],
                       d["copies"], d["report"], workspace=workspace)
    return host(d)


def check_fork(length, table, src, free, count, P, inplace=False, workspace=None):
    want = op.fork(table, length, src, free, count, P, table if inplace else np.full_like(table, 77))
    got = run_fork(length, table, src, free, count, P, inplace, workspace)
    for a, b in (("report", "report"), ("len_out", "lengths"), ("out", "table"), ("free", "free"), ("copies", "copies")):
        assert np.array_equal(got[a], want[b]), (a, got[a], want[b])
    assert got["left"][0] == want["free_left"]
    if not inplace:
        assert np.array_equal(got["table"], table) and np.array_equal(got["lengths"], length) and got["count"][0] == count
    assert np.array_equal(got["src"], src)
    return want


def sources(seed, B, kind):
    rng = np.random.default_rng(seed + 1000)
    if kind == "same":
        return np.arange(B)
    if kind == "end":
        return np.full(B, -1)
    if kind == "one":
        return np.full(B, rng.integers(0, B))
    if kind == "turn":
        return np.roll(np.arange(B), 1)
    return np.where(rng.random(B) < 0.2, -1, np.where(rng.random(B) < 0.4, np.arange(B), rng.integers(0, B, B)))


@pytest.mark.parametrize("B,P,max_len", [
    (1, 16, 40), (2, 1, 9), (5, 16, 700), (31, 4, 300), (33, 64, 5000), (257, 16, 900), (1024, 16, 400), (1024, 16, 3000),
    (64, 16, 20000), (3, 1, 70000), (700, 4096, 30000)])
@pytest.mark.parametrize("kind", ["mixed", "same", "end", "one", "turn"])
@pytest.mark.parametrize("inplace", [False, True])
def test_fork(B, P, max_len, kind, inplace):
    length, table, free, count = batch(B + P, B, P, max_len, spare=B + 3)
    assert check_fork(length, table, sources(B, B, kind), free, count, P, inplace)["report"][0] == 0


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("big", [False, True])
def test_fork_all_or_nothing(inplace, big):
    B = 600 if big else 20
    length, table, free, count = batch(3, B, 16, 2500, spare=B, extra=9)
    src = sources(5, B, "mixed")
    need = op.fork(table, length, src, free, count, 16)["report"][2]
    back = op.fork(table, length, src, free, count, 16)["report"][1]
    # fewer than are wanted; exactly as many
    for spare in (max(0, need - back - 1), max(0, need - back)):
        want = check_fork(length, table, src, free, spare, 16, inplace)
        assert want["report"][0] == (3 if spare < need - back else 0)
    one = np.full(B, int(np.argmax(length % 16)))
    assert check_fork(length, table, one, np.full(len(free), -1, np.int32), 0, 16, inplace)["report"][0] in (0, 3)
    # a stack that says that it has more than the pool
    assert check_fork(length, table, np.full(B, -1), free, len(free), 16, inplace)["report"][0] == 3
    # a source that is not there; a length beyond the table
    bad = src.copy()
    bad[-1] = B
    assert check_fork(length, table, bad, free, count, 16, inplace)["report"][0] == 1
    far = length.copy()
    far[1] = table.shape[1] * 16 + 1
    assert check_fork(far, table, src, free, count, 16, inplace)["report"][0] == 3


def test_fork_lengths_below_zero_and_foreign_pages():
    length, table, free, count = batch(11, 12, 16, 500, spare=20)
    length[3] = -7
    table[5, 0], table[6, 1] = len(free) + 5, -9
    length[5], length[6] = 30, 40
    for src in (np.arange(12), np.full(12, -1), np.full(12, 5), np.roll(np.arange(12), 3)):
        check_fork(length, table, src, free, count, 16)


def run_compact(length, table, pages, P, inplace=False, moves=None):
    m = pages // 2 if moves is None else moves
    d = dict(table=i32(table), lengths=i32(length), out=i32(np.full_like(table, 77)), free=i32(np.full(pages, 77)),
             left=i32([77]), moves=i32(np.full((m, 2), 77)), report=i32([77] * 4))
    if inplace:
        d["out"] = d["table"]
    dkv.dkv_pages_compact(d["table"], d["lengths"], P, d["out"], d["free"], d["left"], d["moves"], d["report"])
    return host(d)


def check_compact(length, table, pages, P, inplace=False, moves=None):
    want = op.compact(table, length, pages, P, pages // 2 if moves is None else moves,
                      table if inplace else np.full_like(table, 77), np.full(pages, 77, np.int32))
    got = run_compact(length, table, pages, P, inplace, moves)
    for a, b in (("report", "report"), ("moves", "moves"), ("out", "table"), ("free", "free")):
        assert np.array_equal(got[a], want[b]), (a, got[a], want[b])
    assert got["left"][0] == (77 if want["free_left"] is None else want["free_left"])
    return want


@pytest.mark.parametrize("B,P,max_len,spare,extra", [
    (1, 16, 40, 0, 0), (1, 16, 40, 5, 0), (2, 1, 9, 1, 3), (5, 16, 700, 30, 40), (31, 4, 300, 1, 0), (33, 64, 5000, 0, 900),
    (257, 16, 900, 70, 7), (1024, 16, 400, 20000, 17), (1024, 16, 3000, 50000, 5), (64, 16, 20000, 7, 200000), (3, 1, 70000, 99999, 1)])
@pytest.mark.parametrize("inplace", [False, True])
def test_compact(B, P, max_len, spare, extra, inplace):
    length, table, free, _ = batch(B + P, B, P, max_len, spare, extra=extra)
    assert check_compact(length, table, len(free), P, inplace)["report"][0] == 0


def test_compact_edges():
    # nothing held; all held; a pool of one page; held in front already; more room for moves than needed
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    check_compact([0, 0, 0], table, 12, 16)
    check_compact([64, 64, 64], table, 12, 16)
    check_compact([0, 0, 1], table[:, :1] * 0, 1, 16)
    check_compact([16, 0, 0], table, 40, 16, moves=33)
    check_compact([0, 0, 64], table, 12, 16)
    check_compact([0, -3, 50], table, 12, 16)
    # foreign indices stay; a length beyond the table moves nothing
    odd = table.copy()
    odd[0, 0], odd[2, 3] = 12, -5
    check_compact([64, 0, 64], odd, 12, 16)
    for inplace in (False, True):
        assert check_compact([64, 0, 65], table, 12, 16, inplace)["report"][0] == 3


# ---- copy ---------------------------------------------------------------------------------

@pytest.mark.parametrize("size", [64, 127, 4096, 1 << 15, 1 << 17, 1 << 18])
@pytest.mark.parametrize("off", [-1, 0, 1, 37])
def test_pools_of_all_sizes(size, off):
    """A few sequences in pools around powers of two, with those that just fit one launch and just do not among them."""
    B, P, max_len = 4, 16, 120
    used = len(batch(5, B, P, max_len, spare=0)[2])
    entries = B * (-(-max_len // P) + 1)
    length, table, free, count = batch(5, B, P, max_len, spare=max(8, size - entries - used + off))
    for kind in ("mixed", "end", "one"):
        assert check_fork(length, table, sources(6, B, kind), free, count, P)["report"][0] == 0
    check_compact(length, table, len(free), P, inplace=bool(off & 1))


def pools_of(seed, pages, shapes, pin=False):
    g = torch.Generator().manual_seed(seed)
    made = []
    for shape, dt in shapes:
        t = torch.randint(-100, 100, (pages, *shape), generator=g, dtype=torch.int16 if dt.itemsize == 2 else torch.int8
                          if dt.itemsize == 1 else torch.int32).view(dt)
        made.append(t.pin_memory() if pin else t.cuda())
    return made


SHAPES = [((8, 16, 128), torch.uint8), ((8, 1), torch.float32), ((3, 7, 4), torch.bfloat16), ((1, 4), torch.int8),
          ((2, 16 * 36), torch.uint8), ((5000,), torch.float32), ((16387,), torch.int32)]


@pytest.mark.parametrize("n,pages,apart", [(1, 2, False), (7, 40, False), (300, 700, True), (40, 100, True)])
@pytest.mark.parametrize("where", ["device", "out", "in"])
def test_copy(n, pages, apart, where):
    rng = np.random.default_rng(n)
    order = rng.permutation(pages)
    pairs = np.stack([order[:n], order[n:2 * n] if pages >= 2 * n else order[:n]], -1).astype(np.int32)
    pairs[rng.random(n) < 0.2] = -1
    if n > 20:  # outside one of the pools
        pairs[3], pairs[5], pairs[11] = (pages, pairs[3, 1]), (pairs[5, 0], pages + 900), (-4, 2)
        pairs[0] = -1, 5
    src = pools_of(1, pages, SHAPES, pin=where == "in")
    into = src if not apart and where == "device" else pools_of(2, pages + 3, SHAPES, pin=where == "out")
    byte = lambda t: t.cpu().contiguous().view(torch.uint8).numpy().copy() if t.dim() else None  # noqa: E731
    a, b = [byte(t) for t in src], [byte(t) for t in into]
    dkv.dkv_pages_copy(i32(pairs), src, None if into is src else into)
    torch.cuda.synchronize()
    for x, y, s, t in zip(a, b, src, into):
        want = y.copy()
        for f, to in pairs:
            if 0 <= f < len(x) and 0 <= to < len(y):
                want[to] = x[f]
        assert np.array_equal(byte(t), want)
        if t is not s:
            assert np.array_equal(byte(s), x)


def test_copy_many_pools_and_offsets():
    # more pools than one launch takes; views whose pages have only 4-byte alignment; a page count past 2^31 bytes
    pairs = i32([[0, 3], [1, 2]])
    flat = [torch.arange(1 + 4 * (5 + i % 3), dtype=torch.int32, device="cuda") + 1000 * i for i in range(150)]
    pools = [f[1:].view(4, -1) for f in flat]
    want = [p.clone() for p in pools]
    for w in want:
        w[3], w[2] = w[0].clone(), w[1].clone()
    dkv.dkv_pages_copy(pairs, pools)
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
    big = torch.zeros((70000, 65536), dtype=torch.uint8, device="cuda")
    big[69999] = 7
    big[5] = 9
    dkv.dkv_pages_copy(i32([[69999, 4], [5, 69998]]), [big])
    assert int(big[4].min()) == 7 and int(big[69998].min()) == 9 and int(big[69997].max()) == 0


# ---- together -----------------------------------------------------------------------------

def test_captured_and_replayed_in_place():
    """Beams that go on as one another at every step, sequences that end, in one graph; compaction with its copies in another."""
    B, P, pages = 12, 16, 400
    rng = np.random.default_rng(0)
    lengths = rng.integers(1, 200, B).astype(np.int32)
    table = np.full((B, 32), -1, np.int32)
    order, at = rng.permutation(pages), 0
    for b in range(B):
        n = op.held(lengths[b], P)
        table[b, :n] = order[at:at + n]
        at += n
    free = np.full(pages, -1, np.int32)
    free[:pages - at] = order[at:]
    count = pages - at
    d = dict(table=i32(table), len=i32(lengths), src=i32(np.arange(B)), free=i32(free), count=i32([count]),
             copies=i32(np.zeros((B, 2))), report=i32([0] * 4), moves=i32(np.zeros((pages // 2, 2))))
    pool = torch.randint(0, 255, (pages, 2, P, 8), dtype=torch.uint8, device="cuda")
    ws = torch.empty(dkv.dkv_pages_workspace(B, 32, pages), dtype=torch.uint8, device="cuda")

    def fork():
        dkv.dkv_pages_fork(d["table"], d["len"], d["src"], d["free"], d["count"], P, d["table"], d["len"], d["count"],
                           d["copies"], d["report"], workspace=ws)
        dkv.dkv_pages_copy(d["copies"], [pool])

    def compact():
        dkv.dkv_pages_compact(d["table"], d["len"], P, d["table"], d["free"], d["count"], d["moves"], d["report"])
        dkv.dkv_pages_copy(d["moves"], [pool])

    def rows(b, t, n):
        return pool.cpu().numpy()[t[b, :op.held(n[b], P)]]

    graphs = []
    side = torch.cuda.Stream()
    for f in (fork, compact):
        state = {k: v.clone() for k, v in d.items()}
        keep = pool.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            f()
        for k in d:
            d[k].copy_(state[k])
        pool.copy_(keep)
        graphs.append(g)
    for step in range(8):
        src = np.where(rng.random(B) < 0.15, -1, rng.integers(0, B, B)).astype(np.int32)
        had = [rows(b, table, lengths) for b in range(B)]
        d["src"].copy_(i32(src))
        graphs[0].replay()
        want = op.fork(table, lengths, src, free, count, P, table)
        got = host(d)
        assert np.array_equal(got["table"], want["table"]) and np.array_equal(got["report"], want["report"])
        assert np.array_equal(got["free"], want["free"]) and np.array_equal(got["len"], want["lengths"])
        table, lengths, free, count = got["table"], got["len"], got["free"], int(got["count"][0])
        for b in range(B):
            if src[b] >= 0:
                assert np.array_equal(rows(b, table, lengths), had[src[b]])
        if step % 3 == 2:
            had = [rows(b, table, lengths) for b in range(B)]
            graphs[1].replay()
            got = host(d)
            want = op.compact(table, lengths, pages, P, pages // 2, table, free)
            assert np.array_equal(got["table"], want["table"]) and np.array_equal(got["free"], want["free"])
            table, lengths, free, count = got["table"], got["len"], got["free"], int(got["count"][0])
            assert all(np.array_equal(rows(b, table, lengths), had[b]) for b in range(B))


@pytest.mark.parametrize("op_name", ["fork", "compact"])
def test_large_tables_in_a_graph(op_name):
    """The launches of a large table captured, and replayed on inputs that change, workspace from the allocator."""
    B, P, pages = 300, 16, 120_000
    cases = [batch(s, B, P, 12_000, spare=400) for s in range(3)]
    max_pages = cases[0][1].shape[1]
    d = dict(table=i32(np.zeros((B, max_pages))), len=i32(np.zeros(B)), src=i32(np.zeros(B)), free=i32(np.full(pages, -1)),
             count=i32([0]), out=i32(np.zeros((B, max_pages))), lo=i32(np.zeros(B)), left=i32([0]), copies=i32(np.zeros((B, 2))),
             moves=i32(np.zeros((pages // 2, 2))), report=i32([0] * 4))

    def call():
        if op_name == "fork":
            dkv.dkv_pages_fork(d["table"], d["len"], d["src"], d["free"], d["count"], P, d["out"], d["lo"], d["left"],
                               d["copies"], d["report"])
        else:
            dkv.dkv_pages_compact(d["table"], d["len"], P, d["out"], d["free"], d["left"], d["moves"], d["report"])
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for s in (0, 1, 2, 0):
        length, table, free, count = cases[s]
        assert len(free) <= pages
        src = sources(s, B, "mixed")
        stack = np.full(pages, -1, np.int32)
        stack[:count] = free[:count]
        for k, v in (("table", table), ("len", length), ("src", src), ("free", stack), ("count", [count]), ("out", np.full_like(table, 77))):
            d[k].copy_(i32(v))
        graph.replay()
        got = host(d)
        if op_name == "fork":
            want = op.fork(table, length, src, stack, count, P, np.full_like(table, 77))
            assert np.array_equal(got["lo"], want["lengths"]) and np.array_equal(got["copies"], want["copies"])
        else:
            want = op.compact(table, length, pages, P, pages // 2, np.full_like(table, 77), stack)
            assert np.array_equal(got["moves"], want["moves"])
        assert np.array_equal(got["out"], want["table"]) and np.array_equal(got["free"], want["free"])
        assert np.array_equal(got["report"], want["report"]) and got["left"][0] == want["free_left"]


def test_streams_and_workspaces_from_the_allocator():
    """Many calls at once on two streams, workspaces from torch's allocator: each gives what it gives alone."""
    cases = [batch(s, 200, 16, 4000, spare=300) for s in range(4)]
    src = [sources(s, 200, "mixed") for s in range(4)]
    want = [op.fork(t, n, src[i], f, c, 16, np.full_like(t, 77)) for i, (n, t, f, c) in enumerate(cases)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for rep in range(3):
        for i, (n, t, f, c) in enumerate(cases):
            d = dict(table=i32(t), len=i32(n), src=i32(src[i]), free=i32(f), count=i32([c]), out=i32(np.full_like(t, 77)),
                     lo=i32([0] * 200), left=i32([0]), copies=i32(np.zeros((200, 2))), report=i32([0] * 4))
            torch.cuda.synchronize()
            dkv.dkv_pages_fork(d["table"], d["len"], d["src"], d["free"], d["count"], 16, d["out"], d["lo"], d["left"],
                               d["copies"], d["report"], stream=streams[i % 2])
            got.append((i, d))
    torch.cuda.synchronize()
    for i, d in got:
        assert np.array_equal(d["out"].cpu().numpy(), want[i]["table"])
        assert np.array_equal(d["free"].cpu().numpy(), want[i]["free"])
