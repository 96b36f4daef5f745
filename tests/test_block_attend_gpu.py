"""Attention over an 8-bit cache with block scales on the GPU against the fp64 oracle."""
import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from oracle import block_step as bs
from oracle import paged_step as step
from tests.step_tiles import CASES, TILE, P, Tiles

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step of the type, relative


def tdt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float16


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def i32(x):
    return dev(np.asarray(x, np.int32))


def host(t):
    return t.detach().cpu().double().numpy()


def case(seed, lens, rows, Hq, Hkv, D, dtype, P, spread=1.0, levels=1.0, extra_pages=2):
    """levels: blocks' sizes are spread by up to 2^levels either way."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    max_pages = max(1, max(-(-int(n) // P) for n in lens))
    pages = B * max_pages + extra_pages
    pools = []
    for s in (spread, 1.0):
        y = rng.standard_normal((pages, Hkv, P, D)) * s
        y *= np.repeat(np.exp2(np.round(rng.uniform(-levels, levels, (pages, Hkv, P // 16)))), 16, -1)[..., None]
        pools.append(bs.make_pool(y))
    table = rng.permutation(pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    N = int(start[-1]) + 2  # two rows of no sequence
    q = torch.from_numpy(rng.standard_normal((N, Hq, D)).astype(np.float32)).to(tdt(dtype))
    return dict(q=q, pools=pools, table=table, lens=np.asarray(lens, np.int32), start=start, D=D, dtype=dtype)


def on_device(pools):
    (k, ks), (v, vs) = pools
    return [dev(k).view(torch.float8_e4m3fn), dev(v).view(torch.float8_e4m3fn), dev(ks), dev(vs)]


def run(c, scale=None, pools=None, with_start=True, max_rows=None, **more):
    q = c["q"].cuda()
    if not with_start:
        q = q[:len(c["lens"])].contiguous()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    rows = np.diff(c["start"])
    dkv.dkv_block_attend(q, *(pools or on_device(c["pools"])), i32(c["table"]), i32(c["lens"]), out,
                         row_start=i32(c["start"]) if with_start else None,
                         max_rows=max_rows or max(1, int(rows.max())), scale=scale, lse=lse, **more)
    return out, lse


def check(c, out, lse, scale=None):
    """Bounds, per output: half a step of the type on |o|.  Weights times V's scale (what they add to the outputs) rounded
    to fp16: 2^-11 of each, and half a subnormal step, 2^-25, where the largest is 2^7 and more: 2^-32 of that, which is at
    most the largest scale, for every |code|.  A score's fp32 sum of D products and its scaling, (D + 8) 2^-23
    of sum |q k|, and the sum with log2 of V's scale, 2^-23 of that, move weights by that exponent, twice
    (weight and sum); 2^-20 for the exponential, the logarithm and the inverse of a scale (2^-22 each); fp32 sums over the
    keys, 2^-23 each."""
    n = out.shape[0]
    D, half = c["D"], HALF[c["dtype"]]
    sc = D ** -0.5 if scale is None else scale
    (k, ks), (v, vs) = c["pools"]
    ref = step.attend(c["q"][:n].double().numpy(), bs.values(k, ks), bs.values(v, vs), c["table"], c["lens"],
                      c["start"], sc)
    most = vs[np.isfinite(vs)].max()
    codes = step.attend(c["q"][:n].double().numpy(), bs.values(k, ks), bs.values(v, np.full_like(vs, most)), c["table"],
                        c["lens"], c["start"], sc)["vabs"]
    got, low = host(out), host(lse)
    live = ref["live"]
    lv = np.abs(np.log2(vs[np.isfinite(vs)])).max()
    ds = (D + 8) * 2.0 ** -23 * ref["smax"] + 2.0 ** -20 + (ref["keys"] + lv) * 2.0 ** -23
    tol = half * np.abs(ref["out"]) + ref["wabs"] * (2.0 ** -11 + 2 * ds[..., None]) + 2.0 ** -32 * codes + 2.0 ** -24
    err = np.abs(got - ref["out"])
    assert np.all(err[live] <= tol[live]), (np.nanmax((err / tol)[live]), np.argwhere(err > tol)[:5])
    none = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(low[live]), none[live])
    ok = live[:, None] & ~none
    tol = ds + 2.0 ** -22 * np.abs(ref["lse"], where=ok, out=np.zeros_like(ref["lse"]))
    assert np.all(np.abs(low[ok] - ref["lse"][ok]) <= tol[ok])
    assert np.all(got[~live] == 7) and np.all(low[~live] == 7)
    return ref


LENS = [0, 1, 2, 15, 16, 17, 33, 127, 128, 129, 255, 300, 1000]


@pytest.mark.parametrize("Hq,Hkv,D,dtype,P", [
    (8, 2, 64, "bf16", 16), (4, 1, 128, "bf16", 16), (32, 8, 128, "fp16", 32), (2, 2, 64, "fp16", 64),
    (3, 3, 128, "bf16", 16), (6, 2, 128, "fp16", 256), (16, 2, 64, "bf16", 16), (40, 2, 128, "bf16", 32),
    (33, 1, 64, "fp16", 16), (24, 1, 128, "fp16", 16), (24, 1, 64, "bf16", 16), (12, 1, 128, "bf16", 4096)])
def test_single_rows(Hq, Hkv, D, dtype, P):
    c = case(Hq + D, LENS, [1] * len(LENS), Hq, Hkv, D, dtype, P)
    out, lse = run(c)
    check(c, out, lse)
    alone, low = run(c, with_start=False)
    assert torch.equal(alone, out[:len(LENS)]) and torch.equal(low, lse[:len(LENS)])


@pytest.mark.parametrize("Hq,Hkv,D,dtype,P,rows", [
    (8, 2, 64, "bf16", 16, [2, 3, 1, 5]), (4, 1, 128, "fp16", 16, [4, 7, 0, 9]), (8, 8, 128, "bf16", 32, [17, 1, 33, 2]),
    (6, 2, 64, "fp16", 16, [40, 0, 11, 1]), (5, 1, 128, "bf16", 64, [100, 37, 3, 0]), (8, 2, 128, "bf16", 16, [200, 129, 64, 1])])
@pytest.mark.parametrize("cached", [0, 1, 130])
def test_chunks(Hq, Hkv, D, dtype, P, rows, cached):
    c = case(D + cached, [r + cached for r in rows], rows, Hq, Hkv, D, dtype, P)
    check(c, *run(c))


def test_more_rows_than_keys():
    for rows, lens in (([5, 2, 30], [3, 0, 20]), ([60, 50, 300], [3, 0, 200])):
        c = case(2, lens, rows, 4, 2, 128, "bf16", 16)
        ref = check(c, *run(c))
        assert np.isneginf(ref["lse"][:2]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_long_and_split(D):
    c = case(4, [20000, 7, 4097], [1, 1, 3], 8, 2, D, "bf16", 64)
    check(c, *run(c))


@pytest.mark.parametrize("Hq,D,rows,keys", [
    (2, 64, 1, 320_011), (4, 128, 1, 60_001), (2, 128, 16, 40_003), (2, 64, 10, 60_001), (2, 128, 20, 20_003),
    (1, 64, 200, 1_500), (1, 128, 129, 700)])
def test_one_item_over_all_ctas(Hq, D, rows, keys):
    check(c := case(keys, [keys], [rows], Hq, 1, D, "fp16", 64), *run(c))


@pytest.mark.parametrize("rows", [1, 4, 40])
@pytest.mark.parametrize("spread", [0.01, 20.0])
def test_flat_and_peaked(rows, spread):
    c = case(5, [700, 64, 1000], [rows, rows, 2], 8, 2, 128, "bf16", 16, spread=spread)
    check(c, *run(c))


@pytest.mark.parametrize("rows", [1, 50])
@pytest.mark.parametrize("slope", [0.02, 0.5, 4.0, -1.0])
def test_rising_scores(rows, slope):
    """The maximum rises key by key in steps below and above what moves a row's reference."""
    c = case(6, [900], [rows], 4, 1, 128, "bf16", 16)
    vals = np.zeros((c["pools"][0][0].shape[0], 1, 16, 128))
    for p, page in enumerate(c["table"][0]):
        vals[page, 0] = (np.arange(p * 16, p * 16 + 16) * slope / 8)[:, None]
    c["pools"][0] = bs.make_pool(vals)
    c["q"] = torch.ones_like(c["q"]) * 0.5
    check(c, *run(c))


@pytest.mark.parametrize("rows", [1, 3, 60])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_all_sizes(rows, D):
    """Blocks 2^20 apart either way, in order and not, blocks of zeros, and scales that are no powers of two."""
    c = case(7, [500, 900, 40], [rows, rows, 1], 4, 2, D, "bf16", 16, levels=20.0)
    (k, ks), (v, vs) = c["pools"]
    ks[:] = 2.0 ** -7  # (scores of ordinary size: it is V's scales that the weights carry)
    check(c, *run(c))
    for order in (np.sort(vs, 0), np.sort(vs, 0)[::-1]):
        d = dict(c, pools=[(k, ks), (v, np.ascontiguousarray(order))])
        check(d, *run(d))
    rng = np.random.default_rng(1)
    odd = [(k, (ks * rng.uniform(0.3, 3, ks.shape)).astype(np.float32)), (v, rng.uniform(0.001, 100, vs.shape).astype(np.float32))]
    d = dict(c, pools=odd)
    check(d, *run(d))
    z = v.copy()
    z[::2] = 0
    zs = vs.copy()
    zs[::2] = 2.0 ** -64  # what the append gives a block of zeros
    zs[1::2] = 2.0 ** -5
    d = dict(c, pools=[(k, ks), (z, zs)])
    check(d, *run(d))
    z[:], zs[:] = 0, 2.0 ** -64
    out, _ = run(dict(c, pools=[(k, ks), (z, zs)]))
    assert torch.all(out[:2 * rows + 1] == 0)


@pytest.mark.parametrize("rows", [1, 90])
def test_query_range_and_scale(rows):
    c = case(8, [200, 300], [rows, rows + 1], 4, 2, 128, "bf16", 16)
    for mul, scale in ((1e30, 1e-31), (1e-30, 1e29), (1.0, -0.3), (1.0, 0.0)):
        d = dict(c, q=(c["q"].float() * mul).to(torch.bfloat16))
        check(d, *run(d, scale=scale), scale=scale)
    d = dict(c, q=torch.zeros_like(c["q"]))
    check(d, *run(d))


@pytest.mark.parametrize("rows", [1, 6, 60])
@pytest.mark.parametrize("D", [64, 128])
def test_masked_nan_does_not_leak(rows, D):
    """Everything behind a sequence's length, its last page and pages of no sequence, holds NaN codes; blocks without any
    visible key NaN and infinite scales."""
    lens = [1, 15, 16, 40, 129, 0, 200]
    n = [min(rows, x) for x in lens]
    c = case(9, lens, n, 4, 2, D, "bf16", 16)
    clean = check(c, *run(c))
    used = {(int(c["table"][b, t // 16]), t % 16) for b, x in enumerate(lens) for t in range(x)}
    for code, sc in c["pools"]:
        for p in range(len(code)):
            for r in range(16):
                if (p, r) not in used:
                    code[p, :, r] = 0x7F if r % 2 else 0xFF
            if (p, 0) not in used:
                sc[p] = np.nan if p % 2 else np.inf
    out, lse = run(c)
    assert np.isfinite(host(out)[clean["live"]]).all()
    for i, (code, sc) in enumerate(c["pools"]):  # the reference reads what is visible
        code[(code & 0x7F) == 0x7F] = 0
        sc[~np.isfinite(sc)] = 1
    check(c, out, lse)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -1.0, 0.0])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("rows,G,D", [(20, 1, 64), (12, 2, 128), (100, 2, 64), (70, 1, 128)])
def test_scales_of_later_tokens_do_not_leak(rows, G, D, which, bad):
    """Blocks that the later rows of a chunk see and the earlier ones do not: the earlier ones take nothing from their
    scales, and a NaN reaches all the later ones.  (More than 32 packed rows: a tile with such a scale adds its weights up
    block by block, so fp32 sums of at most 200 weights in another order, 200 * 2^-23 of lse; an output's quotient then
    rounds to the same fp16 number or the one beside it, a step of 2^-10.)"""
    c = case(12, [200], [rows], G, 1, D, "fp16", 16)
    clean, low = run(c)
    c["pools"][which][1][c["table"][0, 12]] = bad  # tokens 192 .. 199
    got, lse = run(c)
    first = 192 - (200 - rows)  # the first row that sees one
    if np.isnan(bad):
        assert torch.isnan(got[first:rows].float()).all()
    if rows * G <= 32:
        assert torch.equal(got[:first], clean[:first]) and torch.equal(lse[:first], low[:first])
    else:
        a, b = host(got)[:first], host(clean)[:first]
        assert np.all(np.abs(a - b) <= 2.0 ** -10 * np.abs(b) + 2.0 ** -24)
        assert np.all(np.abs(host(lse)[:first] - host(low)[:first]) <= 200 * 2.0 ** -23)


@pytest.mark.parametrize("which,dim", [(0, 5), (1, 0), (1, 63), (1, 101)])
@pytest.mark.parametrize("rows,at", [(6, 0), (6, 30), (6, 36), (6, 39), (100, 0), (100, 100), (100, 180), (100, 199)])
def test_visible_nan_reaches_its_rows_and_dims_only(which, dim, rows, at):
    keys = 40 if rows == 6 else 200
    c = case(10, [keys, keys], [rows, rows], 4, 2, 128, "fp16", 16)
    clean = host(run(c)[0])
    c["pools"][which][0][c["table"][1, at // 16], :, at % 16, dim] = 0x7F if dim else 0xFF
    got = host(run(c)[0])
    assert np.array_equal(got[:rows], clean[:rows])  # the other sequence
    for i in range(rows):
        row = got[rows + i]
        if at > keys - rows + i:
            assert np.array_equal(row, clean[rows + i])
        elif which == 0:
            assert np.isnan(row).all()
        else:
            assert np.isnan(row[:, dim]).all() and np.isfinite(np.delete(row, dim, 1)).all()


def test_bad_tables_and_lengths():
    for k in (1, 90):
        c = case(11, [300, 400, 200], [k, k + 1, k], 4, 2, 64, "bf16", 16)
        c["table"][0, 1], c["table"][1, 0], c["table"][1, 13] = -1, 1 << 30, -(1 << 31)
        c["table"][2, :12] = c["pools"][0][0].shape[0]
        check(c, *run(c))
        d = dict(c, lens=np.array([300, 1 << 30, -5], np.int32))
        out, lse = run(d)
        check(dict(c, lens=np.array([300, 400, 0], np.int32)), out, lse)
        run(dict(c, start=np.array([0, 500, -3, 2], np.int32)), max_rows=k + 3)  # held inside q
        torch.cuda.synchronize()


@pytest.mark.parametrize("Hq,Hkv,D,dtype,P,rows,cached", [
    (8, 1, 128, "bf16", 16, [300, 1, 0, 40], [2000, 500, 9, 0]), (4, 2, 64, "fp16", 32, [700, 129], [0, 3000]),
    (8, 8, 128, "fp16", 16, [257, 128, 256], [127, 128, 129]), (7, 1, 64, "bf16", 64, [90, 37, 38], [0, 900, 63]),
    (2, 1, 128, "bf16", 128, [33, 65, 1], [5000, 1, 4000])])
def test_tiles(Hq, Hkv, D, dtype, P, rows, cached):
    c = case(D + len(rows), [r + k for r, k in zip(rows, cached)], rows, Hq, Hkv, D, dtype, P, levels=3.0)
    out, lse = run(c)
    check(c, out, lse)
    again, low = run(c)
    assert torch.equal(out, again) and torch.equal(lse, low)


def test_many_sequences():
    rng = np.random.default_rng(21)
    rows = rng.integers(0, 50, 400)
    rows[:200] = 0
    check(c := case(21, rows + rng.integers(0, 300, 400), rows, 2, 1, 64, "bf16", 16), *run(c))
    check(c := case(15, rng.integers(0, 40, 1024), [1] * 1024, 2, 1, 64, "bf16", 16), *run(c))
    check(c := case(15, rng.integers(0, 200, 1024), [1] * 1024, 2, 1, 128, "bf16", 16), *run(c))
    c = case(22, [0, 5], [0, 0], 4, 1, 128, "bf16", 16)
    out, lse = run(c, max_rows=100)
    assert torch.all(out == 7) and torch.all(lse == 7)


@pytest.mark.parametrize("name", CASES)
def test_no_tile_is_lost_doubled_or_misplaced(name):
    t = Tiles(*CASES[name])
    pools = [bs.make_pool(step.read_pool(p, t.D)) for p in t.pools]
    k, v = [bs.values(*p)[::TILE // P, :, 0] for p in pools]
    t.level, t.v = k[..., 0], v  # as this format holds them
    rows, Hq, D = int(t.start[-1]), t.Hq, t.D
    q = dev(np.broadcast_to(t.q[None, :, None], (rows, Hq, D)).astype(np.float32)).to(tdt(t.dtype)).contiguous()
    out = torch.full((rows, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((rows, Hq), 7.0, device="cuda")
    dkv.dkv_block_attend(q, *on_device(pools), i32(t.table), i32(t.lens), out, row_start=i32(t.start),
                         max_rows=max(1, max(t.rows)), scale=t.scale, lse=lse)
    out, lse = host(out), host(lse)
    for b in range(len(t.lens)):
        if t.rows[b]:
            want = t.reference(b)
            at = slice(t.start[b], t.start[b + 1])
            assert t.bad(b, out[at], lse[at], want) == (0, 0), b


def test_strides_shared_pages_pinned_pools_and_streams():
    for rows in (1, 60):
        c = case(12, [577, 900], [rows, rows], 8, 2, 128, "bf16", 16)
        c["table"][1, :3] = c["table"][0, :3]  # a shared prefix
        want, low = run(c)
        check(c, want, low)
        n = c["q"].shape[0]
        wide = torch.zeros((n, 12, 128), dtype=torch.bfloat16, device="cuda")
        wide[:, :8] = c["q"].cuda()
        out = torch.full((n, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        args = (i32(c["table"]), i32(c["lens"]), out)
        more = dict(row_start=i32(c["start"]), max_rows=rows)
        dkv.dkv_block_attend(wide[:, :8], *on_device(c["pools"]), *args, **more)
        assert torch.equal(out, want)
        pinned = [t.cpu().pin_memory() for t in on_device(c["pools"])]
        out.fill_(7.0)
        dkv.dkv_block_attend(wide[:, :8], *pinned, *args, **more)
        assert torch.equal(out, want)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(3):
            got, low2 = run(c, stream=side)
            side.synchronize()
            assert torch.equal(got, want) and torch.equal(low2, low)
        ws = torch.full((dkv.dkv_paged_attend_workspace(2, 8, 2, 128, rows),), 0xFF, dtype=torch.uint8, device="cuda")
        assert torch.equal(run(c, workspace=ws)[0], want)


def test_workspace_shared_in_turn_with_graphs():
    """One workspace for calls of every kernel of both formats' attention, in turn, and for graphs replayed in turn."""
    cases = [case(31, [3000, 40], [1, 1], 8, 2, 128, "bf16", 16), case(32, [2000, 300], [100, 70], 8, 2, 128, "bf16", 16),
             case(33, [2500, 31], [3, 2], 8, 2, 128, "bf16", 16)]
    want = [run(c) for c in cases]
    size = max(dkv.dkv_paged_attend_workspace(2, 8, 2, 128, m) for m in (1, 3, 100))
    ws = torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")
    for i in (0, 1, 0, 2, 1, 2, 0):
        out, lse = run(cases[i], workspace=ws)
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), i
    graphs = []
    for c in cases:
        q, out = c["q"].cuda(), torch.full(c["q"].shape, 7.0, dtype=c["q"].dtype, device="cuda")
        a = (q, *on_device(c["pools"]), i32(c["table"]), i32(c["lens"]), out)
        kw = dict(row_start=i32(c["start"]), max_rows=int(np.diff(c["start"]).max()), workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dkv.dkv_block_attend(*a, **kw)
        graphs.append((g, out, a, kw))
    for i in (0, 1, 2, 2, 0, 1, 0):
        graphs[i][1].fill_(7.0)
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[i][1], want[i][0]), i


def test_offsets_past_32_bits():
    D, P, Hkv = 128, 64, 8
    per = Hkv * P * D
    pages = (46 * 10 ** 8) // per
    for rows in (2, 60):
        c = case(16, [200, 64], [1, rows], 16, Hkv, D, "bf16", P)
        n = c["pools"][0][0].shape[0]
        big = [torch.empty((pages, Hkv, P, D), dtype=torch.uint8, device="cuda") for _ in "kv"]
        scales = [torch.empty((pages, Hkv, P // 16), device="cuda") for _ in "kv"]
        for b, s, (code, sc) in zip(big, scales, c["pools"]):
            b[pages - n:] = dev(code)
            s[pages - n:] = dev(sc)
        moved = dict(c, table=c["table"] + np.int32(pages - n))
        check(c, *run(moved, pools=[*big, *scales]))


@pytest.mark.parametrize("D", [64, 128])
def test_waits_that_run_out(D):
    """Outputs that are never signalled (a test hook): every wait of the many-row kernel ends, the rows and their lse are NaN,
    and the next call is right."""
    c = case(17, [700, 300], [90, 300], 4, 2, D, "bf16", 16)
    want = run(c)
    dkv.dkv_paged_attend_debug_withhold(True)
    try:
        out, lse = run(c)
        torch.cuda.synchronize()
    finally:
        dkv.dkv_paged_attend_debug_withhold(False)
    assert torch.isnan(out[:390].float()).all() and torch.isnan(lse[:390]).all() and (out[390:] == 7).all()
    again = run(c)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
