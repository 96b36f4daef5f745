"""The append to an 8-bit cache with block scales on the GPU: the oracle's bytes and scales, equal."""
import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from oracle import block_step as bs
from oracle import paged_step as step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step of the type, relative


def tdt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float16


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def i32(x):
    return dev(np.asarray(x, np.int32))


def rows_of(seed, N, Hq, Hkv, D, dtype, spread=1.0):
    g = np.random.default_rng(seed)
    x = g.standard_normal((N, Hq + 2 * Hkv, D)) * np.exp(spread * g.standard_normal((N, Hq + 2 * Hkv, 1)))
    qkv = torch.from_numpy(x.astype(np.float32)).to(tdt(dtype)).cuda()
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]


def slots_of(seed, lens, P, pad=3):
    """Slots of sequences that each append `len` rows from somewhere inside a page on, in pages of their own; padding between
    some and behind."""
    rng = np.random.default_rng(seed)
    per = [-(-(n + P) // P) for n in lens]
    pages = rng.permutation(sum(per) + 2)
    slot, at = [], 0
    for n, k in zip(lens, per):
        pos = int(rng.integers(0, P)) + np.arange(n)
        slot += list(pages[at + pos // P] * P + pos % P)
        at += k
        if rng.random() < 0.2:
            slot.append(-1)
    return np.array(slot + [-1] * pad, np.int32), sum(per) + 2


def filled(seed, pages, Hkv, P, D, level=1.0):
    rng = np.random.default_rng(seed + 50)
    return [bs.make_pool(rng.standard_normal((pages, Hkv, P, D)) * level) for _ in "kv"]


def check(q, k, v, slot, pos, table, pools, inter=False, norm=True, eps=2.0 ** -20, dtype="bf16", outs=True, pin=False):
    N, Hkv, D = k.shape
    dt = k.dtype
    rng = np.random.default_rng(9)
    gq, gk = [torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).to(dt).cuda() if norm else None
              for _ in range(2)]
    pages, _, P, _ = pools[0][0].shape
    put = (lambda x: torch.from_numpy(x.copy()).pin_memory()) if pin else dev
    d = [(put(c), put(s)) for c, s in pools]
    qo = None if q is None else torch.full(q.shape, 7.0, dtype=dt, device="cuda")
    ko, vo = [torch.full(k.shape, 7.0, dtype=dt, device="cuda") for _ in "kv"]
    dkv.dkv_block_append(q, k, v, i32(pos), i32(slot), d[0][0], d[1][0].view(torch.float8_e4m3fn), d[0][1], d[1][1], qo,
                         k_out=ko if outs else None, v_out=vo if outs else None, q_gamma=None if q is None else gq,
                         k_gamma=gk, eps=eps, cos_sin=None if table is None else dev(table), interleaved=inter)
    torch.cuda.synchronize()
    f = lambda t: None if t is None else t.float().cpu().numpy()  # noqa: E731
    live = (slot >= 0) & (slot < pages * P)
    half = HALF[dtype]
    if q is not None:  # fp32 with the norm's sum in any order, rounded once
        want, mag = step.turn(f(q), f(gq), eps, table, pos, inter)
        got = qo.double().cpu().numpy()
        tol = half * np.abs(want) + (D + 8) * 2.0 ** -24 * mag + 2.0 ** -25 * (dtype == "fp16")
        assert np.all(np.abs(got - want)[live] <= tol[live]) and np.all(got[~live] == 7)
    for name, (code, sc), was, x, out in (("k", d[0], pools[0], k, ko), ("v", d[1], pools[1], v, vo)):
        y = step.turn(f(x), f(gk), eps, table, pos, inter)[0] if name == "k" else f(x)
        code2, sc2, held = bs.append(y, slot, *was)
        got = code.view(torch.uint8).cpu().numpy()
        assert np.array_equal(sc.cpu().numpy().view(np.uint32), sc2.view(np.uint32)), name  # NaN that nobody touched too
        nan = lambda c: np.where((c & 0x7F) == 0x7F, 0x7F, c)  # noqa: E731
        assert np.array_equal(nan(got), nan(code2)), name
        if outs:
            o = out.double().cpu().numpy()
            assert np.array_equal(np.isnan(o[live]), np.isnan(held[live])) and np.all(o[~live] == 7)
            # E4M3 may round the type's largest numbers up to a power of two that it does not hold: an infinity there
            past = np.abs(held) >= (2.0 ** 128 if dtype == "bf16" else 65520.0)
            assert np.array_equal(o[live & past.any((1, 2))][past[live & past.any((1, 2))]],
                                  np.copysign(np.inf, held[past & live[:, None, None]]))
            ok = live[:, None, None] & np.isfinite(held) & ~past
            assert np.all(np.abs(o - held)[ok] <= half * np.abs(held)[ok] + 2.0 ** -25 * (dtype == "fp16"))
    return d


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype,P,rot,inter,norm", [
    ([1], 1, 1, 64, "bf16", 16, 64, False, True), ([1] * 9, 32, 8, 128, "bf16", 16, 128, False, True),
    ([7, 1, 16, 33], 5, 5, 64, "fp16", 32, 32, True, False), ([100], 8, 2, 128, "fp16", 16, 64, False, True),
    ([5] * 12, 9, 3, 128, "bf16", 64, 16, True, True), ([129, 3], 33, 11, 64, "bf16", 16, 48, False, True),
    ([200], 4, 1, 64, "fp16", 128, 0, False, False), ([1, 0, 2, 4000], 3, 1, 128, "bf16", 64, 128, True, True),
    ([1] * 3000, 2, 2, 64, "fp16", 16, 64, True, True), ([17, 2, 3, 900] * 3, 8, 8, 64, "bf16", 4096, 64, False, False)])
def test_append(lens, Hq, Hkv, D, dtype, P, rot, inter, norm):
    slot, pages = slots_of(1, lens, P)
    N = len(slot)
    q, k, v = rows_of(2, N, Hq, Hkv, D, dtype)
    pos = np.random.default_rng(3).integers(0, 500, N).astype(np.int32)
    table = dkv.rope_table(500, rot, device="cpu").numpy() if rot else None
    check(q, k, v, slot, pos, table, filled(4, pages, Hkv, P, D), inter, norm, dtype=dtype)


@pytest.mark.parametrize("Hkv,D,dtype,norm", [(1, 128, "bf16", True), (3, 128, "fp16", True), (3, 64, "bf16", False)])
@pytest.mark.parametrize("mix", ["single", "few", "all"])
def test_long_calls_of_short_blocks(mix, Hkv, D, dtype, norm):
    """4096 rows and more, in blocks of one row, of a few, of all counts beside one another."""
    rng = np.random.default_rng(21)
    lens = {"single": [1] * 4200, "few": list(rng.integers(1, 9, 1000)),
            "all": list(rng.permutation([1] * 600 + [5, 6, 7, 8] * 90 + [16, 17, 40] * 9 + [900]))}[mix]
    slot, pages = slots_of(22, [int(n) for n in lens], 16)
    N = len(slot)
    assert N >= 4096
    _, k, v = rows_of(23, N, 1, Hkv, D, dtype)
    pos = rng.integers(0, 500, N).astype(np.int32)
    table = dkv.rope_table(500, 32, device="cpu").numpy()
    check(None, k, v, slot, pos, table, filled(24, pages, Hkv, 16, D), norm=norm, dtype=dtype, outs=mix == "all")


@pytest.mark.parametrize("D,dtype,norm", [(64, "bf16", False), (64, "fp16", True), (128, "bf16", True)])
def test_every_operation_rounds_once(D, dtype, norm):
    """Millions of keys, each row a block of its own: one rounding more or less on the way moves some code across a border."""
    N, Hkv = 4200, 33
    _, k, v = rows_of(25, N, 1, Hkv, D, dtype, spread=0.3)
    pos = np.random.default_rng(26).integers(0, 500, N).astype(np.int32)
    table = dkv.rope_table(500, D, device="cpu").numpy()
    gk = torch.from_numpy((1 + 0.2 * np.random.default_rng(9).standard_normal(D)).astype(np.float32)).to(k.dtype).cuda() if norm else None
    code = [torch.zeros((N, Hkv, 16, D), dtype=torch.uint8, device="cuda") for _ in "kv"]
    sc = [torch.zeros((N, Hkv, 1), device="cuda") for _ in "kv"]
    slot = 16 * np.arange(N, dtype=np.int32)
    dkv.dkv_block_append(None, k, v, i32(pos), i32(slot), *code, *sc, k_gamma=gk, eps=2.0 ** -20, cos_sin=dev(table))
    f = lambda t: None if t is None else t.float().cpu().numpy()  # noqa: E731
    for c, s, y in zip(code, sc, (step.turn(f(k), f(gk), 2.0 ** -20, table, pos, False)[0], f(v))):
        want = bs.scale_for(np.abs(y).max(-1))
        assert np.array_equal(s.cpu().numpy()[..., 0], want.astype(np.float32))
        assert np.array_equal(c[:, :, 0].cpu().numpy(), bs.encode(y / want[..., None]))


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16")])
def test_token_by_token_is_the_chunk(D, dtype):
    """40 tokens one call each, into blocks that grow: with powers of two the same bytes as the oracle's at every call, and
    what the chunk's call writes up to E4M3's subnormals."""
    q, k, v = rows_of(5, 40, 2, 2, D, dtype, spread=2.0)
    slot = (np.arange(40) + 32 + 5).astype(np.int32)
    empty = [(np.full((8, 2, 16, D), 0x55, np.uint8), np.full((8, 2, 1), 2.0 ** -40, np.float32)) for _ in "kv"]
    pools = empty
    for i in range(40):
        d = check(q[i:i + 1], k[i:i + 1], v[i:i + 1], slot[i:i + 1], np.array([i], np.int32), None, pools, norm=False, dtype=dtype)
        pools = [(c.view(torch.uint8).cpu().numpy(), s.cpu().numpy()) for c, s in d]
    d = check(q, k, v, slot, np.arange(40, dtype=np.int32), None, empty, norm=False, dtype=dtype)
    for (c, s), (c2, s2) in zip(pools, d):
        assert np.array_equal(s, s2.cpu().numpy())
        # slots 48 .. 76 are appended rows of blocks that begin anew (what lies behind them is nobody's)
        a, b = (bs.values(x, s)[3:5].swapaxes(1, 2).reshape(32, -1)[:29] for x in (c, c2.view(torch.uint8).cpu().numpy()))
        # growing scales round subnormals again, half a step of ever larger steps each time: a step of the last in all
        step_of = 2.0 ** -9 * np.repeat(np.repeat(s[3:5], 16, -1)[..., None], D, -1).swapaxes(1, 2).reshape(32, -1)[:29]
        assert np.all(np.abs(a - b) <= step_of)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_extremes(dtype):
    """Zeros, the type's largest and smallest numbers, borders of scales and codes, infinities and NaN."""
    top = float(torch.finfo(tdt(dtype)).max)
    tiny = float(torch.finfo(tdt(dtype)).tiny)
    N, D = 64, 64
    _, k, v = rows_of(6, N, 1, 2, D, dtype, spread=3.0)
    k, v = k.clone(), v.clone()
    k[0:16] = 0
    k[16, 0, 3], k[17, 1, 5] = top, -top
    k[20, 0, 1], k[21, 1, 2] = float("inf"), float("nan")
    k[32:48] = tiny
    v[0:16] = 3.5  # 448 * 2^-7, the border of a scale
    v[3, 0, 0] = 3.515625
    v[16:32] = torch.linspace(-448, 448, 16 * 2 * D).reshape(16, 2, D).to(v.dtype)
    v[32:48] = float("nan")
    v[48:64] = float("-inf")
    slot = np.arange(N).astype(np.int32)
    for order in (slot, slot + 5):
        check(None, k, v, order, slot, None, filled(7, 5, 2, 16, D), norm=False, dtype=dtype)
    # one by one beside what is there, infinities first
    for i in (20, 21, 16, 35, 3):
        check(None, k[i:i + 1], v[i:i + 1], np.array([37], np.int32), slot[:1], None, filled(8, 5, 2, 16, D, 100.0), norm=False, dtype=dtype)


def test_foreign_scales():
    """Scales that something else has written: not a power of two, none at all."""
    _, k, v = rows_of(8, 3, 1, 2, 64, "bf16")
    for s in (0.013, 3.0, 0.0, -1.0, np.inf, np.nan, 1e-42, 1e30):
        pools = [(c, np.full_like(x, s)) for c, x in filled(9, 4, 2, 16, 64)]
        check(None, k, v, np.array([20, 21, 22], np.int32), np.zeros(3, np.int32), None, pools, norm=False)


def test_positions_outside_the_table_and_slots_outside_the_pool():
    slot, pages = slots_of(3, [20, 5], 16)
    N = len(slot)
    q, k, v = rows_of(4, N, 3, 1, 128, "bf16")
    slot[4:6] = pages * 16, 1 << 30
    pos = np.arange(N).astype(np.int32)
    table = dkv.rope_table(8, 128, device="cpu").numpy()
    pools = filled(5, pages, 1, 16, 128)
    qo = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    d = [(dev(c), dev(s)) for c, s in pools]
    pos[7] = -3
    dkv.dkv_block_append(q, k, v, i32(pos), i32(slot), d[0][0], d[1][0], d[0][1], d[1][1], qo, cos_sin=dev(table))
    got = d[0][0].cpu().numpy()
    for i in range(N):
        if 0 <= slot[i] < pages * 16:
            far = pos[i] >= 8 or pos[i] < 0
            assert bool(torch.isnan(qo[i].float()).all()) == far
            assert np.isnan(bs.decode(got[slot[i] // 16, 0, slot[i] % 16])).all() == far
        else:
            assert (qo[i] == 7).all()


def test_pinned_pools_views_and_streams():
    """Pools and scales in pinned host memory; queries left out; another stream; rows of a wider projection."""
    slot, pages = slots_of(11, [3, 40, 1], 32)
    N = len(slot)
    wide = torch.randn((N, 1000), device="cuda").to(torch.float16)
    k, v = wide[:, 8:8 + 256].unflatten(-1, (2, 128)), wide[:, 512:768].unflatten(-1, (2, 128))
    check(None, k, v, slot, np.arange(N, dtype=np.int32), None, filled(12, pages, 2, 32, 128), norm=False, dtype="fp16", pin=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        check(None, k, v, slot, np.arange(N, dtype=np.int32), None, filled(12, pages, 2, 32, 128), dtype="fp16", outs=False)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes, rows at its end."""
    P, Hkv, D = 4096, 32, 128
    pages = 280
    kp = torch.zeros((pages, Hkv, P, D), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((pages, Hkv, P // 16), dtype=torch.float32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((20, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    slot = i32(pages * P - 20 + np.arange(20))
    vp, vs = kp.clone(), sc.clone()
    dkv.dkv_block_append(None, k, -k, slot, slot, kp, vp, sc, vs)
    tail = np.zeros((1, Hkv, 32, D), np.uint8), np.zeros((1, Hkv, 2), np.float32)
    code, s, _ = bs.append(k.float().cpu().numpy(), np.arange(12, 32), *tail)
    assert np.array_equal(kp[-1, :, -32:].cpu().numpy(), code[0]) and np.array_equal(sc[-1, :, -2:].cpu().numpy(), s[0])
    assert np.array_equal(vp[-1, :, -32:].cpu().numpy(), np.where(code[0] & 0x7F, code[0] ^ 0x80, vp[-1, :, -32:].cpu().numpy()))
    assert int(kp[:-1].max()) == 0 and int(kp[-1, :, :-32].max()) == 0
