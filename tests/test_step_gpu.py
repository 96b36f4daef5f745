"""The device-side step on the GPU against the fp64 / numpy oracle: planning, append and
attention one by one, then together, eagerly and as a captured graph."""
import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from oracle import paged_step as step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step of the type, relative


def tdt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float16


def dev(x, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.to(dt) if dt is not None else t).cuda()


def i32(x):
    return dev(np.asarray(x, np.int32))


def host(t):
    return t.detach().cpu().double().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


# ---- planning ---------------------------------------------------------------------------

def plan_case(seed, B, P, max_new, max_len, max_pages, spare, ended=0.1):
    rng = np.random.default_rng(seed)
    length = rng.integers(0, max_len + 1, B)
    new = rng.integers(0, max_new + 1, B)
    new[rng.random(B) < ended] = -1
    held = -(-length // P)
    pool = rng.permutation(int(held.sum()) + spare).astype(np.int32)
    table = np.full((B, max_pages), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = pool[at:at + held[b]]
        at += held[b]
    free = np.full(len(pool), -1, np.int32)
    free[:spare] = pool[at:]
    return length.astype(np.int32), new.astype(np.int32), table, free, spare


def run_plan(length, new, table, free, count, P, max_rows, inplace=False):
    B = len(length)
    d = dict(length=i32(length), new=i32(new), table=i32(table), free=i32(free), count=i32([count]),
             start=i32(np.full(B + 1, 77)), pos=i32(np.full(max_rows, 77)), slot=i32(np.full(max_rows, 77)),
             kv=i32(np.full(B, 77)), left=i32([77]), report=i32([77] * 4))
    if inplace:
        d["kv"], d["left"] = d["length"], d["count"]
    dkv.dkv_step_plan(d["length"], d["new"], d["table"], d["free"], d["count"], P, d["start"], d["pos"],
                      d["slot"], d["kv"], d["left"], d["report"])
    return {k: host(v) for k, v in d.items()}


def check_plan(case, P, max_rows, inplace=False):
    want = step.plan(*case, P, max_rows)
    got = run_plan(*case, P, max_rows, inplace)
    for a, b in (("table", "table"), ("free", "free"), ("start", "row_start"), ("pos", "pos"), ("slot", "slot"),
                 ("kv", "kv_len"), ("report", "report")):
        assert np.array_equal(got[a], want[b]), (a, got[a], want[b])
    assert got["left"][0] == want["free_left"]
    if not inplace:
        assert np.array_equal(got["length"], case[0]) and got["count"][0] == case[4]
    return want


@pytest.mark.parametrize("B,P,max_new,max_rows", [
    (1, 16, 1, 1), (1, 1, 5, 9), (3, 16, 1, 8), (31, 16, 40, 1300), (32, 64, 1, 32), (33, 16, 17, 600),
    (257, 32, 3, 800), (1024, 16, 1, 1024), (1024, 4096, 30, 31000), (64, 16, 100, 6400), (5, 2, 3000, 15001),
    (700, 16, 60, 40001), (1, 16, 20000, 20011)])
@pytest.mark.parametrize("inplace", [False, True])
def test_plan(B, P, max_new, max_rows, inplace):
    max_pages = -(-(2000 + max_new) // P)
    case = plan_case(B + P, B, P, max_new, 2000, max_pages, B * (max_new // P + 2))
    assert check_plan(case, P, max_rows, inplace)["report"][0] == 0


def test_plan_edges():
    # every sequence ended; none has anything to do; lengths at page borders; no page needed
    for new in ([-1] * 4, [0] * 4, [1, 0, -1, 1]):
        case = plan_case(7, 4, 16, 1, 200, 20, 9)
        length = np.array([16, 32, 0, 15], np.int32)
        table = np.arange(80, dtype=np.int32).reshape(4, 20)
        check_plan((length, np.array(new, np.int32), table, np.r_[np.arange(80, 89), [-1] * 91].astype(np.int32), 9), 16, 8)
        check_plan(case, 16, 4)


@pytest.mark.parametrize("why", ["pages", "rows", "table", "length"])
@pytest.mark.parametrize("inplace", [False, True])
def test_plan_all_or_nothing(why, inplace):
    length, new, table, free, count = plan_case(3, 40, 16, 50, 500, 40, 200)
    max_rows = 2000
    if why == "pages":
        new[:] = 50
        count = 5
    elif why == "rows":
        max_rows = int(new[new > 0].sum()) - 1
    elif why == "table":
        new[17] = 40 * 16
    else:
        length[3] = 40 * 16 + 1
        new[3] = 0
    want = check_plan((length, new, table, free, count), 16, max_rows, inplace)
    assert want["report"][0] == 3 and want["slot"].max() == -1
    # exactly enough is enough
    if why == "rows":
        assert check_plan((length, new, table, free, count), 16, max_rows + 1)["report"][0] == 0


def test_plan_pages_suffice_only_with_released_ones():
    length, new = np.array([64, 64], np.int32), np.array([64, -1], np.int32)
    table = np.arange(16, dtype=np.int32).reshape(2, 8)
    free = np.full(16, -1, np.int32)
    assert check_plan((length, new, table, free, 0), 16, 64)["report"] == [0, 64, 4, 128]
    new[0] = 65
    assert check_plan((length, new, table, free, 0), 16, 65)["report"][0] == 3


# ---- append -----------------------------------------------------------------------------

def append_case(seed, N, Hq, Hkv, D, dtype, spread=1.0):
    g = np.random.default_rng(seed)
    qkv = torch.from_numpy((g.standard_normal((N, (Hq + 2 * Hkv), D)) * np.exp(
        spread * g.standard_normal((N, Hq + 2 * Hkv, 1)))).astype(np.float32)).to(tdt(dtype)).cuda()
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]


def check_append(q, k, v, P, slot, pos, table, inter=False, norm=True, k_scale=1.0, v_scale=1.0, eps=2.0 ** -20,
                 pools=None, outs=True, dtype="bf16"):
    N, Hq, D = q.shape
    Hkv, dt = k.shape[1], q.dtype
    rng = np.random.default_rng(9)
    gq, gk = [torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).to(dt).cuda() if norm else None
              for _ in range(2)]
    pages = int(max(slot.max() // P + 1, 2))
    if pools is None:
        pools = [torch.full((pages, Hkv, P * D * 9 // 16), 0xA5, dtype=torch.uint8, device="cuda") for _ in "kv"]
    pages = pools[0].shape[0]
    qo, ko, vo = [torch.full(x.shape, 7.0, dtype=dt, device="cuda") for x in (q, k, v)]
    dkv.dkv_qkv_append(q, k, v, i32(pos), i32(slot), pools[0], pools[1], qo, k_out=ko if outs else None,
                       v_out=vo if outs else None, q_gamma=gq, k_gamma=gk, eps=eps,
                       cos_sin=None if table is None else dev(table), interleaved=inter, k_scale=k_scale, v_scale=v_scale)
    f = lambda t: None if t is None else t.float().cpu().numpy()  # noqa: E731
    live = (slot >= 0) & (slot < pages * P)
    half = HALF[dtype]
    # q: fp32 with the norm's sum in any order, rounded once
    want, mag = step.turn(f(q), f(gq), eps, table, pos, inter)
    err = np.abs(host(qo) - want)
    tol = half * np.abs(want) + (D + 8) * 2.0 ** -24 * mag + 2.0 ** -25 * (dtype == "fp16")
    assert np.all(err[live] <= tol[live]), (err[live] - tol[live]).max()
    assert np.all(host(qo)[~live] == 7)
    # k, v: the same bytes as the oracle's, padding rows and other slots untouched
    for name, pool, x, mul, out in (("k", pools[0], k, k_scale, ko), ("v", pools[1], v, v_scale, vo)):
        y = step.turn(f(x), f(gk), eps, table, pos, inter)[0] if name == "k" else f(x)
        y = (y * np.float32(1 / np.float32(mul))).astype(np.float32)
        code, scale = step.quantise(y)
        want = np.full(tuple(pool.shape), 0xA5, np.uint8)
        raw, sc = step.pool_views(want, D)
        raw, sc = raw.copy(), sc.copy()
        packed = code[..., 0::2] | (code[..., 1::2] << 4)
        raw[slot[live] // P, :, slot[live] % P] = packed[live]
        sc[slot[live] // P, :, slot[live] % P] = scale[live]
        want = np.concatenate([raw.reshape(pages, Hkv, -1), sc.reshape(pages, Hkv, -1)], -1)
        got = pool.cpu().numpy()
        # the sign of a zero code says nothing
        clean = lambda w: np.where((w & 0x7F) == 0, w & 0x7F, w)  # noqa: E731
        cut = P * D // 2
        zero = lambda a: np.where((a & 0x77) == 0, 0, np.where((a & 7) == 0, a & 0xF0, np.where((a & 0x70) == 0, a & 0x0F, a)))  # noqa: E731
        assert np.array_equal(zero(got[..., :cut]), zero(want[..., :cut])), name
        assert np.array_equal(clean(got[..., cut:]), clean(want[..., cut:])), name
        if outs:
            val = step.dequantise(code, scale) * np.float32(mul)
            got = host(out)
            assert np.array_equal(np.isnan(got[live]), np.isnan(val[live]))
            ok = live[:, None, None] & np.isfinite(val)
            assert np.all(np.abs(got - val)[ok] <= half * np.abs(val)[ok] + 2.0 ** -25 * (dtype == "fp16"))
            assert np.all(got[~live] == 7)
    return pools


def slots_for(seed, N, P, pad=0.2):
    rng = np.random.default_rng(seed)
    slot = rng.permutation((N // P + 3) * P)[:N]
    slot[rng.random(N) < pad] = -1
    slot[0] = 5
    return np.where((slot == 5) & (np.arange(N) > 0), -1, slot).astype(np.int32)


@pytest.mark.parametrize("N,Hq,Hkv,D,dtype,P,rot,inter,norm", [
    (1, 1, 1, 64, "bf16", 16, 64, False, True), (1, 32, 8, 128, "bf16", 16, 128, False, True),
    (7, 5, 5, 64, "fp16", 32, 32, True, False), (33, 8, 2, 128, "fp16", 16, 64, False, True),
    (50, 9, 3, 128, "bf16", 64, 16, True, True), (129, 33, 11, 64, "bf16", 16, 48, False, True),
    (500, 32, 32, 64, "fp16", 4096, 64, True, True), (2049, 6, 1, 128, "bf16", 16, 96, True, True),
    (20, 4, 4, 128, "bf16", 16, 0, False, False), (20, 65, 13, 64, "fp16", 16, 0, False, True)])
def test_append(N, Hq, Hkv, D, dtype, P, rot, inter, norm):
    q, k, v = append_case(N, N, Hq, Hkv, D, dtype)
    pos = np.random.default_rng(N).integers(0, 131072, N).astype(np.int32)
    table = dkv.rope_table(131072, rot).cpu().numpy() if rot else None
    check_append(q, k, v, P, slots_for(N, N, P), pos, table, inter, norm, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_scales_and_extremes(dtype):
    N, D, P = 40, 128, 16
    q, k, v = append_case(5, N, 4, 2, D, dtype, spread=4.0)  # blocks below and above the scale's range
    k = k.clone()
    v = v.clone()
    v[0], k[1] = 0, 0                      # zero blocks
    v[2, 0, 17] = float("nan")             # poisons its block alone
    v[3, 1, 40] = float("inf")
    v[4, 0, 100] = float("-inf")
    v[5] = 6.0 * 448 * 2 if dtype == "bf16" else 65504.0  # saturates
    v[6] = 1e-6                            # below half the smallest scale: zero
    v[7, 0, :16] = torch.arange(16) * 0.25  # ties
    pos = np.arange(N, dtype=np.int32)
    check_append(q, k, v, P, slots_for(1, N, P), pos, dkv.rope_table(64, D).cpu().numpy(), norm=False, dtype=dtype)
    check_append(q, k, v, P, slots_for(1, N, P), pos, None, norm=True, k_scale=0.37, v_scale=0.01, dtype=dtype)


def test_append_norm_extremes():
    # rows of zeros, of the largest and of the smallest numbers keep the formula's value
    N, D = 8, 64
    q, k, v = [x.clone() for x in append_case(6, N, 2, 2, D, "bf16")]
    for x in (q, k):
        x[0] = 0
        x[1] *= 1e18
        x[2] *= 1e-18
        x[3, :, 1:] = 0
    check_append(q, k, v, 16, np.arange(N, dtype=np.int32), np.zeros(N, np.int32), None, eps=2.0 ** -20)
    check_append(q[1:], k[1:], v[1:], 16, np.arange(N - 1, dtype=np.int32), np.zeros(N - 1, np.int32), None, eps=0.0)


def test_append_slot_and_position_bounds():
    N, D = 6, 64
    q, k, v = append_case(8, N, 2, 2, D, "bf16")
    slot = np.array([0, 32, -5, 31, 1 << 30, -(1 << 31)], np.int32)  # the pool has 32
    pools = [torch.full((2, 2, 16 * 36), 0xA5, dtype=torch.uint8, device="cuda") for _ in "kv"]
    check_append(q, k, v, 16, slot, np.arange(N, dtype=np.int32), None, pools=pools)
    # a position outside the table: NaN q, a NaN key, the value as it is
    table = dkv.rope_table(16, D)
    qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    pos = i32([0, 15, 16, -1, 1 << 30, 3])
    dkv.dkv_qkv_append(q, k, v, pos, i32(np.arange(N)), pools[0], pools[1], qo.contiguous(), k_out=ko.contiguous(),
                       v_out=vo.contiguous(), cos_sin=table)
    qo, ko, vo = [torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (q, k, v)]
    dkv.dkv_qkv_append(q, k, v, pos, i32(np.arange(N)), pools[0], pools[1], qo, k_out=ko, v_out=vo, cos_sin=table)
    bad = torch.tensor([False, False, True, True, True, False], device="cuda")
    assert torch.equal(qo.isnan().all(-1).all(-1), bad) and torch.equal(ko.isnan().all(-1).all(-1), bad)
    assert not qo[~bad].isnan().any() and not vo.isnan().any()


def test_append_without_pool_and_in_place():
    N, D = 37, 128
    q, k, v = append_case(11, N, 4, 2, D, "bf16")
    pos, table = np.arange(N).astype(np.int32), dkv.rope_table(64, D)
    g = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    want = {n: step.turn(f(x), f(g), 1e-6, table.cpu().numpy(), pos, False) for n, x in (("q", q), ("k", k))}
    a, b, c = q.contiguous(), k.contiguous(), v.contiguous()
    dkv.dkv_qkv_append(a, b, c, i32(pos), q_out=a, k_out=b, v_out=c, q_gamma=g, k_gamma=g, cos_sin=table)
    for n, x in (("q", a), ("k", b)):
        y, mag = want[n]
        assert np.all(np.abs(host(x) - y) <= 2.0 ** -8 * np.abs(y) + (D + 8) * 2.0 ** -24 * mag)
    assert torch.equal(c, v)
    only = torch.empty(q.shape, dtype=q.dtype, device="cuda")  # queries alone, keys and values alone
    dkv.dkv_qkv_append(q, None, None, i32(pos), q_out=only, q_gamma=g, cos_sin=table)
    assert torch.equal(only, a)
    ko, vo = torch.empty_like(b), torch.empty_like(c)
    dkv.dkv_qkv_append(None, k, v, i32(pos), k_out=ko, v_out=vo, k_gamma=g, cos_sin=table)
    assert torch.equal(ko, b) and torch.equal(vo, c)


# ---- attention --------------------------------------------------------------------------

def attend_case(seed, lens, rows, Hq, Hkv, D, dtype, P, spread=1.0, extra_pages=2):
    rng = np.random.default_rng(seed)
    B = len(lens)
    max_pages = max(1, max(-(-int(n) // P) for n in lens))
    pages = B * max_pages + extra_pages
    vals = [rng.standard_normal((pages, Hkv, P, D)).astype(np.float32) for _ in "kv"]
    vals[0] *= spread
    pools = [step.make_pool(v) for v in vals]
    table = rng.permutation(pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    N = int(start[-1]) + 2  # two rows of no sequence
    q = torch.from_numpy(rng.standard_normal((N, Hq, D)).astype(np.float32)).to(tdt(dtype))
    return dict(q=q, pools=pools, table=table, lens=np.asarray(lens, np.int32), start=start, D=D, dtype=dtype)


def run_attend(c, scale=None, v_scale=1.0, pools=None, with_start=True, max_rows=None, **more):
    q = c["q"].cuda()
    if not with_start:
        q = q[:len(c["lens"])].contiguous()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    pools = pools or [dev(p) for p in c["pools"]]
    rows = np.diff(c["start"])
    dkv.dkv_paged_attend(q, pools[0], pools[1], i32(c["table"]), i32(c["lens"]), out,
                         row_start=i32(c["start"]) if with_start else None,
                         max_rows=max_rows or max(1, int(rows.max())), scale=scale, v_scale=v_scale, lse=lse, **more)
    return out, lse


def check_attend(c, out, lse, scale=None, v_scale=1.0):
    """Bounds, per output: half a step of the type on |o|; weights rounded to fp16 (2^-11 of each, and
    2^-25 where fp16 is subnormal: the largest weight of a row is at least 1 and so is their sum); a
    score's fp32 sum of D products and its scaling, (D + 8) 2^-23 of sum |q k|, moves weights by that
    exponent, twice (weight and sum); 2^-21 for the exponential; fp32 sums over the keys, 2^-23 each."""
    n = out.shape[0]
    D, half = c["D"], HALF[c["dtype"]]
    sc = D ** -0.5 if scale is None else scale
    ref = step.attend(c["q"][:n].double().numpy(), step.read_pool(c["pools"][0], D), step.read_pool(c["pools"][1], D),
                      c["table"], c["lens"], c["start"], sc, v_scale)
    got, low = host(out), host(lse)
    live = ref["live"]
    ds = (D + 8) * 2.0 ** -23 * ref["smax"] + 2.0 ** -21 + ref["keys"] * 2.0 ** -23
    tol = (half * np.abs(ref["out"]) + ref["wabs"] * (2.0 ** -11 + 2 * ds[..., None]) + 2.0 ** -25 * ref["vabs"]
           + 2.0 ** -24)
    err = np.abs(got - ref["out"])
    assert np.all(err[live] <= tol[live]), (np.nanmax((err / tol)[live]), np.argwhere(err > tol)[:5])
    none = np.isneginf(ref["lse"])
    assert np.all(np.isneginf(low[live & none.any(1)][none[live & none.any(1)]])) if none.any() else True
    ok = live[:, None] & ~none
    tol = ds + 2.0 ** -22 * np.abs(ref["lse"], where=ok, out=np.zeros_like(ref["lse"]))
    assert np.all(np.abs(low[ok] - ref["lse"][ok]) <= tol[ok])
    assert np.all(got[~live] == 7) and np.all(low[~live] == 7)
    return ref


LENS = [0, 1, 2, 15, 16, 17, 33, 127, 128, 129, 255, 300, 1000]


@pytest.mark.parametrize("Hq,Hkv,D,dtype,P", [
    (8, 2, 64, "bf16", 16), (4, 1, 128, "bf16", 16), (32, 8, 128, "fp16", 32), (2, 2, 64, "fp16", 64),
    (3, 3, 128, "bf16", 16), (6, 2, 128, "fp16", 256), (16, 2, 64, "bf16", 16), (40, 2, 128, "bf16", 32),
    (33, 1, 64, "fp16", 16)])
def test_attend_single_rows(Hq, Hkv, D, dtype, P):
    c = attend_case(Hq + D, LENS, [1] * len(LENS), Hq, Hkv, D, dtype, P)
    out, lse = run_attend(c)
    check_attend(c, out, lse)
    alone, low = run_attend(c, with_start=False)
    assert torch.equal(alone, out[:len(LENS)]) and torch.equal(low, lse[:len(LENS)])


@pytest.mark.parametrize("Hq,Hkv,D,dtype,P,rows", [
    (8, 2, 64, "bf16", 16, [2, 3, 1, 5]), (4, 1, 128, "fp16", 16, [4, 7, 0, 9]), (8, 8, 128, "bf16", 32, [17, 1, 33, 2]),
    (6, 2, 64, "fp16", 16, [40, 0, 11, 1]), (5, 1, 128, "bf16", 64, [100, 37, 3, 0]), (8, 2, 128, "bf16", 16, [200, 129, 64, 1])])
@pytest.mark.parametrize("cached", [0, 1, 130])
def test_attend_chunks(Hq, Hkv, D, dtype, P, rows, cached):
    c = attend_case(D + cached, [r + cached for r in rows], rows, Hq, Hkv, D, dtype, P)
    check_attend(c, *run_attend(c))


def test_attend_more_rows_than_keys():
    # rows before the first key see nothing
    c = attend_case(2, [3, 0, 20], [5, 2, 30], 4, 2, 128, "bf16", 16)
    ref = check_attend(c, *run_attend(c))
    assert np.isneginf(ref["lse"][:2]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_attend_long_and_split(D):
    c = attend_case(4, [20000, 7, 4097], [1, 1, 3], 8, 2, D, "bf16", 64)
    check_attend(c, *run_attend(c))


@pytest.mark.parametrize("Hq,D,rows,keys", [
    (2, 64, 1, 320_011), (4, 128, 1, 60_001), (2, 128, 16, 40_003), (2, 64, 10, 60_001), (2, 128, 20, 20_003),
    (1, 64, 200, 1_500), (1, 128, 129, 700)])
def test_attend_one_item_over_all_ctas(Hq, D, rows, keys):
    # one KV head: its pieces, up to one a CTA, are joined in groups, or by the blocks of several CTAs
    check_attend(c := attend_case(keys, [keys], [rows], Hq, 1, D, "fp16", 64), *run_attend(c))


@pytest.mark.parametrize("spread", [0.01, 20.0])
def test_attend_flat_and_peaked(spread):
    # near-uniform weights, and scores whose running maximum keeps moving by hundreds
    c = attend_case(5, [700, 64, 1000], [1, 4, 2], 8, 2, 128, "bf16", 16, spread=spread)
    check_attend(c, *run_attend(c))


def test_attend_rising_scores():
    # the maximum rises key by key in steps below and above the lazy threshold
    c = attend_case(6, [600], [1], 4, 1, 128, "bf16", 16)
    for slope in (0.02, 0.5, 4.0, -1.0):
        ramp = np.arange(c["pools"][0].shape[0] * 16, dtype=np.float32) * slope
        vals = np.zeros((c["pools"][0].shape[0], 1, 16, 128), np.float32)
        for p, page in enumerate(c["table"][0]):
            vals[page, 0, :, :] = (ramp[p * 16:(p + 1) * 16] / 8)[:, None]
        c["pools"][0] = step.make_pool(vals)
        c["q"] = torch.ones_like(c["q"]) * 0.5
        check_attend(c, *run_attend(c))


def test_attend_query_range():
    # bf16 queries far outside fp16's range, with small elements next to large ones
    c = attend_case(7, [200, 300], [1, 2], 4, 2, 128, "bf16", 16)
    for mul, scale in ((1e30, 1e-31), (1e-30, 1e29)):
        d = dict(c, q=(c["q"].float() * mul).to(torch.bfloat16))
        d["q"][:, :, ::3] *= 2.0 ** -12
        check_attend(d, *run_attend(d, scale=scale), scale=scale)
    d = dict(c, q=torch.zeros_like(c["q"]))
    check_attend(d, *run_attend(d))


def test_attend_scale_and_v_scale():
    c = attend_case(8, [100, 31], [1, 3], 4, 4, 64, "fp16", 16)
    for scale, v_scale in ((0.0, 2.0), (-0.3, -0.5), (0.01, 1e-3)):
        check_attend(c, *run_attend(c, scale=scale, v_scale=v_scale), scale=scale, v_scale=v_scale)


def poison(pool, D, page, row, k=None):
    """NaN scales (all blocks, or block k) in one row of a page, and codes of the largest magnitude."""
    raw, sc = step.pool_views(pool, D)
    cut = raw[0].size
    flat = pool.reshape(pool.shape[0], -1)
    P, heads = raw.shape[2], raw.shape[1]
    for h in range(heads):
        base = h * (P * D * 9 // 16)
        flat[page, base + row * D // 2: base + (row + 1) * D // 2] = 0x77
        s0 = base + P * D // 2 + row * D // 16
        if k is None:
            flat[page, s0: s0 + D // 16] = 0x7F
        else:
            flat[page, s0 + k] = 0xFF
    assert cut


@pytest.mark.parametrize("rows", [1, 6])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_masked_nan_does_not_leak(rows, D):
    # everything behind a sequence's length, its last page and pages of no sequence, holds NaN
    lens = [1, 15, 16, 40, 129, 0]
    n = [min(rows, x) for x in lens]
    c = attend_case(9, lens, n, 4, 2, D, "bf16", 16)
    clean = check_attend(c, *run_attend(c))
    used = {(int(c["table"][b, t // 16]), t % 16) for b, x in enumerate(lens) for t in range(x)}
    for p in range(c["pools"][0].shape[0]):
        for r in range(16):
            if (p, r) not in used:
                poison(c["pools"][0], D, p, r)
                poison(c["pools"][1], D, p, r)
    out, lse = run_attend(c)
    assert np.isfinite(host(out)[clean["live"]]).all()
    check_attend(c, out, lse)


@pytest.mark.parametrize("which,block", [(0, None), (1, None), (1, 2)])
@pytest.mark.parametrize("at", [0, 30, 36, 39])
def test_attend_visible_nan_reaches_its_rows_only(which, block, at):
    D, G = 128, 2
    c = attend_case(10, [40, 40], [6, 6], 2 * G, 2, D, "fp16", 16)
    clean, _ = run_attend(c)
    poison(c["pools"][which], D, int(c["table"][1, at // 16]), at % 16, block)
    out, _ = run_attend(c)
    got, clean = host(out), host(clean)
    assert np.array_equal(got[:6], clean[:6])  # the other sequence
    for i in range(6):
        sees = at <= 40 - 6 + i
        row = got[6 + i]
        if not sees:
            assert np.array_equal(row, clean[6 + i])
        elif block is None:
            assert np.isnan(row).all()
        else:
            assert np.isnan(row[:, 16 * block:16 * block + 16]).all()
            keep = np.r_[0:16 * block, 16 * block + 16:D]
            assert np.isfinite(row[:, keep]).all()


def test_attend_bad_tables_and_lengths():
    # page indices outside the pool count as pages without keys, lengths are cut to the table
    c = attend_case(11, [60, 64, 50], [1, 2, 1], 4, 2, 64, "bf16", 16)
    c["table"][0, 1], c["table"][1, 0], c["table"][1, 3] = -1, 1 << 30, -(1 << 31)
    c["table"][2, :] = c["pools"][0].shape[0]
    check_attend(c, *run_attend(c))
    d = dict(c, lens=np.array([60, 1 << 30, -5], np.int32))
    out, lse = run_attend(d)
    check_attend(dict(c, lens=np.array([60, 64, 0], np.int32)), out, lse)
    # row starts that fall or pass the rows are held inside q
    bad = dict(c, start=np.array([0, 500, -3, 2], np.int32))
    run_attend(bad, max_rows=4)
    torch.cuda.synchronize()


# ---- attention for many rows (tiles of 128 and 256 packed rows) -----------------------------

@pytest.mark.parametrize("Hq,Hkv,D,dtype,P,rows,cached", [
    (8, 1, 128, "bf16", 16, [300, 1, 0, 40], [2000, 500, 9, 0]), (4, 2, 64, "fp16", 32, [700, 129], [0, 3000]),
    (8, 8, 128, "fp16", 16, [257, 128, 256], [127, 128, 129]), (7, 1, 64, "bf16", 64, [90, 37, 38], [0, 900, 63]),
    (2, 1, 128, "bf16", 128, [33, 65, 1], [5000, 1, 4000])])
def test_attend_tiles(Hq, Hkv, D, dtype, P, rows, cached):
    c = attend_case(D + len(rows), [r + k for r, k in zip(rows, cached)], rows, Hq, Hkv, D, dtype, P)
    out, lse = run_attend(c)
    check_attend(c, out, lse)
    again, low = run_attend(c)
    assert torch.equal(out, again) and torch.equal(lse, low)


def test_attend_tiles_many_sequences():
    rng = np.random.default_rng(21)
    rows = rng.integers(0, 50, 400)
    rows[:200] = 0
    c = attend_case(21, rows + rng.integers(0, 300, 400), rows, 2, 1, 64, "bf16", 16)
    check_attend(c, *run_attend(c))


def test_attend_tiles_none_live():
    c = attend_case(22, [0, 5], [0, 0], 4, 1, 128, "bf16", 16)
    out, lse = run_attend(c, max_rows=100)
    assert torch.all(out == 7) and torch.all(lse == 7)


def test_attend_tiles_more_rows_than_keys():
    c = attend_case(23, [3, 0, 200], [60, 50, 300], 4, 2, 128, "bf16", 16)
    check_attend(c, *run_attend(c))


@pytest.mark.parametrize("spread", [0.01, 20.0])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_tiles_flat_and_peaked(spread, D):
    c = attend_case(24, [1500, 400], [60, 300], 4, 2, D, "bf16", 16, spread=spread)
    check_attend(c, *run_attend(c))


@pytest.mark.parametrize("slope", [0.02, 0.5, 4.0, -1.0])
def test_attend_tiles_rising_scores(slope):
    # the maximum rises tile by tile by less and by more than the weights' bound
    c = attend_case(25, [900], [50], 4, 1, 128, "bf16", 16)
    n = c["pools"][0].shape[0]
    ramp = np.arange(n * 16, dtype=np.float32) * slope
    vals = np.zeros((n, 1, 16, 128), np.float32)
    for p, page in enumerate(c["table"][0]):
        vals[page, 0, :, :] = (ramp[p * 16:(p + 1) * 16] / 8)[:, None]
    c["pools"][0] = step.make_pool(vals)
    c["q"] = torch.ones_like(c["q"]) * 0.5
    check_attend(c, *run_attend(c))


def test_attend_tiles_query_range_and_scale():
    c = attend_case(26, [200, 300], [90, 120], 4, 2, 128, "bf16", 16)
    for mul, scale in ((1e30, 1e-31), (1e-30, 1e29), (1.0, -0.3), (1.0, 0.0)):
        d = dict(c, q=(c["q"].float() * mul).to(torch.bfloat16))
        check_attend(d, *run_attend(d, scale=scale, v_scale=-0.5), scale=scale, v_scale=-0.5)


@pytest.mark.parametrize("D", [64, 128])
def test_attend_tiles_masked_nan_does_not_leak(D):
    lens, rows = [150, 129, 64], [60, 129, 40]
    c = attend_case(27, lens, rows, 4, 2, D, "bf16", 16)
    clean = check_attend(c, *run_attend(c))
    used = {(int(c["table"][b, t // 16]), t % 16) for b, x in enumerate(lens) for t in range(x)}
    for p in range(c["pools"][0].shape[0]):
        for r in range(16):
            if (p, r) not in used:
                poison(c["pools"][0], D, p, r)
                poison(c["pools"][1], D, p, r)
    out, lse = run_attend(c)
    assert np.isfinite(host(out)[clean["live"]]).all()
    check_attend(c, out, lse)


@pytest.mark.parametrize("which,block", [(0, None), (1, None), (1, 2)])
@pytest.mark.parametrize("at", [0, 100, 180, 199])
def test_attend_tiles_visible_nan_reaches_its_rows_only(which, block, at):
    D, G, n = 128, 2, 100
    c = attend_case(28, [200, 200, 40], [n, n, 30], 2 * G, 2, D, "fp16", 16)
    clean, _ = run_attend(c)
    poison(c["pools"][which], D, int(c["table"][1, at // 16]), at % 16, block)
    out, _ = run_attend(c)
    got, clean = host(out), host(clean)
    assert np.array_equal(got[:n], clean[:n]) and np.array_equal(got[2 * n:], clean[2 * n:])
    for i in range(n):
        row = got[n + i]
        if at > 200 - n + i:
            assert np.array_equal(row, clean[n + i])
        elif block is None:
            assert np.isnan(row).all()
        else:
            assert np.isnan(row[:, 16 * block:16 * block + 16]).all()
            assert np.isfinite(row[:, np.r_[0:16 * block, 16 * block + 16:D]]).all()


def test_attend_tiles_bad_tables_and_lengths():
    c = attend_case(29, [300, 400, 200], [90, 120, 60], 4, 2, 64, "bf16", 16)
    c["table"][0, 1], c["table"][1, 0], c["table"][1, 13] = -1, 1 << 30, -(1 << 31)
    c["table"][2, :12] = c["pools"][0].shape[0]
    check_attend(c, *run_attend(c))
    run_attend(dict(c, start=np.array([0, 500, -3, 200], np.int32)), max_rows=100)
    torch.cuda.synchronize()


def test_attend_tiles_in_pinned_host_memory():
    c = attend_case(30, [300, 500], [50, 80], 8, 2, 128, "bf16", 16)
    out, lse = run_attend(c, pools=[torch.from_numpy(p).pin_memory() for p in c["pools"]])
    check_attend(c, out, lse)


def test_attend_strided_queries_and_shared_pages():
    c = attend_case(12, [77, 90], [1, 1], 8, 2, 128, "bf16", 16)
    c["table"][1, :3] = c["table"][0, :3]  # a shared prefix
    wide = torch.zeros((4, 12, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = c["q"].cuda()
    out = torch.full((4, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 8), 7.0, device="cuda")
    pools = [dev(p) for p in c["pools"]]
    dkv.dkv_paged_attend(wide[:, :8], pools[0], pools[1], i32(c["table"]), i32(c["lens"]), out, row_start=i32(c["start"]), lse=lse)
    check_attend(c, out, lse)
    assert torch.equal(out, run_attend(c)[0])


def test_attend_in_pinned_host_memory():
    c = attend_case(13, [300, 5, 1000], [1, 1, 2], 8, 2, 128, "bf16", 16)
    pinned = [torch.from_numpy(p).pin_memory() for p in c["pools"]]
    out, lse = run_attend(c, pools=pinned)
    check_attend(c, out, lse)
    assert torch.equal(out, run_attend(c)[0])


def test_attend_repeats_bit_for_bit_and_on_other_streams():
    c = attend_case(14, [3000, 40, 900, 2500], [1, 1, 3, 1], 8, 2, 128, "bf16", 16)
    out, lse = run_attend(c)
    for _ in range(3):
        again, low = run_attend(c)
        assert torch.equal(out, again) and torch.equal(lse, low)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [run_attend(c, stream=s)[0] for _ in range(3)]
    ws = torch.full((dkv.dkv_paged_attend_workspace(4, 8, 2, 128, 3),), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got.append(run_attend(c, workspace=ws)[0])  # whatever the workspace holds
    torch.cuda.synchronize()
    assert all(torch.equal(out, x) for x in got)


def test_attend_workspace_shared_in_turn():
    # one workspace for calls of every kernel, in turn, and for two graphs replayed in turn
    cases = [attend_case(31, [3000, 40], [1, 1], 8, 2, 128, "bf16", 16), attend_case(32, [2000, 300], [100, 70], 8, 2, 128, "bf16", 16),
             attend_case(33, [2500, 31], [3, 2], 8, 2, 128, "bf16", 16)]
    want = [run_attend(c) for c in cases]
    size = max(dkv.dkv_paged_attend_workspace(2, 8, 2, 128, m) for m in (1, 3, 100))
    ws = torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")
    for i in (0, 1, 0, 2, 1, 2, 0):
        out, lse = run_attend(cases[i], workspace=ws)
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), i
    graphs = []
    for c in cases:
        q, out = c["q"].cuda(), torch.full(c["q"].shape, 7.0, dtype=c["q"].dtype, device="cuda")
        a = (q, *[dev(p) for p in c["pools"]], i32(c["table"]), i32(c["lens"]), out)
        kw = dict(row_start=i32(c["start"]), max_rows=int(np.diff(c["start"]).max()), workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dkv.dkv_paged_attend(*a, **kw)
        graphs.append((g, out, a, kw))
    for i in (0, 1, 2, 2, 0, 1, 0):
        graphs[i][1].fill_(7.0)
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[i][1], want[i][0]), i


def test_attend_two_streams_at_once():
    cases = [attend_case(34, [9000, 40, 7000], [1, 1, 1], 8, 2, 128, "bf16", 16),
             attend_case(35, [6000, 300], [100, 70], 8, 2, 128, "bf16", 16)]
    want = [run_attend(c)[0] for c in cases]
    sets = []
    for c in cases:
        out = torch.full(c["q"].shape, 7.0, dtype=c["q"].dtype, device="cuda")
        kw = dict(row_start=i32(c["start"]), max_rows=int(np.diff(c["start"]).max()), stream=torch.cuda.Stream())
        sets.append((c["q"].cuda(), *[dev(p) for p in c["pools"]], i32(c["table"]), i32(c["lens"]), out, kw))
    torch.cuda.synchronize()
    for _ in range(20):
        for a in sets:
            dkv.dkv_paged_attend(*a[:-1], **a[-1])
    torch.cuda.synchronize()
    for a, w in zip(sets, want):
        assert torch.equal(a[5], w)


def test_attend_many_sequences():
    rng = np.random.default_rng(15)
    lens = rng.integers(0, 40, 1024)
    c = attend_case(15, lens, [1] * 1024, 2, 1, 64, "bf16", 16)
    check_attend(c, *run_attend(c))


def test_attend_offsets_past_32_bits():
    # 4.6 GB pools, the sequences' pages at their end
    D, P, Hkv = 128, 64, 8
    per = Hkv * P * D * 9 // 16
    pages = (46 * 10 ** 8) // per
    c = attend_case(16, [200, 64], [1, 2], 16, Hkv, D, "bf16", P)
    n = c["pools"][0].shape[0]
    big = [torch.empty((pages, Hkv, P * D * 9 // 16), dtype=torch.uint8, device="cuda") for _ in "kv"]
    for b, p in zip(big, c["pools"]):
        b[pages - n:] = dev(p)
    moved = dict(c, table=c["table"] + np.int32(pages - n))
    out, lse = run_attend(moved, pools=big)
    check_attend(c, out, lse)
    # and the append reaches them
    q, k, v = append_case(3, 5, 16, Hkv, D, "bf16")
    slot = np.array([pages * P - 1, pages * P - 70, 3, pages * P, pages * P - 2], np.int64).astype(np.int32)
    qo = torch.empty((5, 16, D), dtype=torch.bfloat16, device="cuda")
    dkv.dkv_qkv_append(q, k, v, None, i32(slot), big[0], big[1], qo)
    for i in (0, 1, 2, 4):
        page = big[1][slot[i] // P].cpu().numpy()[None]
        got = step.read_pool(page, D)[0, :, slot[i] % P]
        assert np.array_equal(got, step.dequantise(*step.quantise(v[i].float().cpu().numpy())))


# ---- together ---------------------------------------------------------------------------

class Loop:
    """A decoder layer's cache as a user's program keeps it: everything on the device."""

    def __init__(self, B, Hq, Hkv, D, P, pages, max_pages, max_rows, dtype="bf16", cache=None, table=None):
        self.shape = B, Hq, Hkv, D, P
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.lengths, self.new, self.table = z(B), z(B), z(B, max_pages) - 1
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int().cuda()
        self.count, self.start, self.report = z(1) + pages, z(B + 1), z(4)
        self.pos, self.slot = z(max_rows), z(max_rows)
        if cache is None:
            self.pools = [torch.zeros((pages, Hkv, P * D * 9 // 16), dtype=torch.uint8, device="cuda") for _ in "kv"]
        else:
            self.pools = [cache.k_pool, cache.v_pool]
        self.rope = dkv.rope_table(4096, D, base=1e4)
        g = torch.Generator().manual_seed(2)
        self.gq, self.gk = [(1 + 0.1 * torch.randn(D, generator=g)).to(tdt(dtype)).cuda() for _ in "qk"]
        self.qkv = torch.zeros((max_rows, Hq + 2 * Hkv, D), dtype=tdt(dtype), device="cuda")
        self.q = torch.zeros((max_rows, Hq, D), dtype=tdt(dtype), device="cuda")
        self.out = torch.zeros((max_rows, Hq, D), dtype=tdt(dtype), device="cuda")
        self.lse = torch.zeros((max_rows, Hq), device="cuda")
        self.max_rows = max_rows

    def __call__(self, max_rows):
        B, Hq, Hkv, D, P = self.shape
        dkv.dkv_step_plan(self.lengths, self.new, self.table, self.free, self.count, P, self.start, self.pos,
                          self.slot, self.lengths, self.count, self.report)
        dkv.dkv_qkv_append(self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:], self.pos, self.slot,
                           *self.pools, self.q, q_gamma=self.gq, k_gamma=self.gk, cos_sin=self.rope)
        dkv.dkv_paged_attend(self.q, *self.pools, self.table, self.lengths, self.out, row_start=self.start,
                             max_rows=max_rows, lse=self.lse)


def follow(loop, news, run, dtype="bf16", seed=0):
    """Drives `loop` through steps of new-token counts and checks each against an oracle that keeps
    every sequence's rows as a list."""
    B, Hq, Hkv, D, P = loop.shape
    rng = np.random.default_rng(seed)
    held = [[np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))] for _ in range(B)]
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    for new in news:
        n = int(sum(x for x in new if x > 0))
        x = rng.standard_normal((loop.max_rows, Hq + 2 * Hkv, D)).astype(np.float32)
        loop.qkv.copy_(torch.from_numpy(x))
        loop.new.copy_(torch.tensor(new, dtype=torch.int32))
        loop.out.fill_(7.0)
        run(max(1, max(new)))
        torch.cuda.synchronize()
        x = f(loop.qkv)
        assert loop.report.tolist()[:2] == [0, n]
        out, low = host(loop.out), host(loop.lse)
        assert np.all(out[n:] == 7)
        r = 0
        for b, k in enumerate(new):
            if k < 0:
                held[b] = [np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))]
                continue
            if k == 0:
                continue
            at = len(held[b][0])
            pos = np.arange(at, at + k)
            rope = loop.rope.cpu().numpy()
            y = step.turn(x[r:r + k, Hq:Hq + Hkv], f(loop.gk), 1e-6, rope, pos, False)[0]
            for i, new_rows in enumerate((y, x[r:r + k, Hq + Hkv:])):
                held[b][i] = np.concatenate([held[b][i], step.dequantise(*step.quantise(new_rows))])
            keys, vals = [h.transpose(1, 0, 2)[None] for h in held[b]]  # one page
            q = host(loop.q)[r:r + k]
            ref = step.attend(q, keys, vals, np.array([[0]]), [at + k], [0, k], D ** -0.5)
            ds = (D + 8) * 2.0 ** -23 * ref["smax"] + 2.0 ** -21 + ref["keys"] * 2.0 ** -23
            tol = (HALF[dtype] * np.abs(ref["out"]) + ref["wabs"] * (2.0 ** -11 + 2 * ds[..., None])
                   + 2.0 ** -25 * ref["vabs"] + 2.0 ** -24)
            assert np.all(np.abs(out[r:r + k] - ref["out"]) <= tol), (new, b)
            assert np.all(np.abs(low[r:r + k] - ref["lse"]) <= ds + 2.0 ** -22 * np.abs(ref["lse"]))
            r += k


NEWS = [[40, 1, 130, 0], [1, 1, 1, 1], [1, 0, 1, 17], [1, -1, 1, 1], [3, 20, -1, 1], [1, 1, 33, 1]] + [[1] * 4] * 20


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64)])
def test_steps_together(Hq, Hkv, D):
    loop = Loop(4, Hq, Hkv, D, 16, 64, 32, 256)
    follow(loop, NEWS, loop)


def test_steps_over_a_pinned_cache():
    cache = dkv.PagedKVCache(4, 2, 128, 16, 64, 32, kv_format="e2m1")
    try:
        info = dkv.dkv_cache_info(cache.h)
        assert info["host_pinned_bytes"] == 2 * 64 * 2 * 16 * 72 and info["kv_format"] == 2
        assert cache.k_host.shape == (64, 2, 16 * 72)
        loop = Loop(4, 8, 2, 128, 16, 64, 32, 256, cache=cache)
        follow(loop, NEWS[:8], loop)
        x = torch.zeros((4, 1, 128), dtype=torch.bfloat16, device="cuda")
        w = torch.zeros((128, 1024), dtype=torch.bfloat16, device="cuda")
        for call in (cache.decode, cache.prefill):
            with pytest.raises(dkv.DkvError) as ei:
                call(x, w, w, w, 8, torch.zeros((4, 1, 8, 128), dtype=torch.bfloat16, device="cuda"))
            assert ei.value.name == "DKV_ERR_UNSUPPORTED"
        q = torch.zeros((4, 8, 128), dtype=torch.bfloat16, device="cuda")
        cache.attend(loop.q[:4], loop.table, loop.lengths, q)
        k = torch.zeros((4, 2, 128), dtype=torch.bfloat16, device="cuda")
        cache.append(loop.q[:4], k, k, None, i32([-1] * 4), q)
        torch.cuda.synchronize()
    finally:
        cache.free()


def test_steps_as_a_captured_graph():
    loop = Loop(4, 8, 2, 128, 16, 64, 32, 8)
    loop.new.fill_(0)
    loop(2)  # nothing new: loads the kernels before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop(2)
    follow(loop, [[1, 2, 0, 1]] * 12 + [[1, -1, 2, 1]] + [[2, 2, 2, 2]] * 3, lambda rows: graph.replay())
    # out of pages: the step is refused as a whole, on the device
    loop.count.fill_(0)
    loop.lengths.fill_(16)
    loop.new.fill_(1)
    loop.out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert loop.report.tolist()[0] == 3 and loop.lengths.tolist() == [16] * 4
    assert torch.all(loop.out == 7) and loop.slot.max().item() == -1
