"""The device-side step where sums, ranges and waits have little room: peaked softmaxes, items in many
pieces, scales, waits that run out."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from oracle import paged_step as step

from .step_tiles import CASES, Tiles
from .test_step_gpu import HALF, check_plan, dev, host, i32, tdt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# ---- one key far above the others ------------------------------------------------------------

def sink_case(keys, Hkv, D, at, P=64):
    """Pools of one sequence: key `at` is a row of ones (as the format holds them) with value 0, every other
    key is 0, its value one of the format's positive numbers times 32, another one for each head and dim."""
    pages = keys // P
    t = np.arange(keys)
    k = np.zeros((keys, D), np.float32)
    k[at] = 1.0
    h, d = np.arange(Hkv)[:, None, None], np.arange(D)
    v = 32.0 * step.E2M1[1 + (3 * t[:, None] + t[:, None] // 64 + h + d // 16) % 7]  # [Hkv, keys, D]
    v[:, at] = 0.0
    pool = lambda x: step.make_pool(np.ascontiguousarray(  # noqa: E731
        np.broadcast_to(x, (Hkv, keys, D)).reshape(Hkv, pages, P, D).transpose(1, 0, 2, 3)).astype(np.float32))
    pools = pool(k), pool(v)
    one = step.read_pool(pools[0][at // P][None], D)[0, 0, at % P, 0]
    held = step.read_pool(pools[1], D).transpose(1, 0, 2, 3).reshape(Hkv, keys, D)
    return pools, one, held


@pytest.mark.parametrize("bits", [16.6, 20.6, 24.4, 26.3])
@pytest.mark.parametrize("at", [0, 77, 2049])
@pytest.mark.parametrize("rows,Hkv,D,dtype,keys,B", [
    (1, 32, 64, "fp16", 4096, 16), (1, 8, 128, "bf16", 8192, 64), (3, 32, 128, "fp16", 4096, 16), (8, 32, 64, "bf16", 4096, 16),
    (40, 8, 128, "bf16", 8192, 20), (64, 8, 64, "fp16", 8192, 20)])
def test_small_weights_beside_a_large_one(rows, Hkv, D, dtype, keys, B, at, bits):
    """Each of thousands of keys weighs 2^-bits of one whose value is 0, so the output is theirs alone.

    A row's weights are rounded to fp16 with the largest at 2^7 or above: 2^-11 of a weight that fp16 holds
    as a normal number, 2^(-25 - 7) of the largest below that, which is 2^(bits - 32) of the weight.  All
    values are positive, so the output is off by no more than that, relative.  2^-12 covers the
    rest: the scores (one fp32 sum of D products and the scale, |score| <= 26.3: 2^-18), the exponential
    2^-21, and the fp32 sums of 2 x 4096 equal terms and fewer, 2^-13 for numerator and denominator each."""
    G = 4 if rows == 3 else 1
    pools, one, v = sink_case(keys, Hkv, D, at)
    scale = bits * np.log(2) / (D * one)
    table = np.broadcast_to(np.arange(keys // 64, dtype=np.int32), (B, keys // 64))
    q = torch.ones((B * rows, Hkv * G, D), dtype=tdt(dtype), device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    dkv.dkv_paged_attend(q, dev(pools[0]), dev(pools[1]), i32(table), i32([keys] * B), out,
                         row_start=i32(np.arange(B + 1) * rows), max_rows=rows, scale=scale, lse=lse)
    seen = keys - rows + 1 + np.arange(rows)
    w = 2.0 ** -bits
    total = 1 + (seen - 1) * w  # of the largest weight
    want = w * np.cumsum(v, 1)[:, seen - 1] / total[:, None]  # [Hkv, rows, D]
    want = np.tile(np.repeat(want.transpose(1, 0, 2), G, 1), (B, 1, 1))
    r = max(2.0 ** -11, 2.0 ** (bits - 32)) + 2.0 ** -12
    err = np.abs(host(out) - want)
    tol = (HALF[dtype] + r) * want + 2.0 ** -25 * (dtype == "fp16")
    assert np.all(err <= tol), (err / want).max()
    low = np.tile(bits * np.log(2) + np.log(total), B)[:, None]
    assert np.all(np.abs(host(lse) - low) <= 2.0 ** -12)


@pytest.mark.parametrize("rows,dtype,sign", [(1, "fp16", 1), (5, "bf16", 1), (1, "bf16", -1), (40, "fp16", 1), (70, "bf16", -1)])
@pytest.mark.parametrize("step_up", [0.3, 3.0, 20.0])
def test_scores_of_two_million(rows, dtype, sign, step_up):
    """Scores of 2^21, which fp32 resolves to 1/4 and no better, that rise from key to key.  A row stays a
    weighted mean of the values, and its lse its largest score: both bounds hold whatever the rounding of
    the scores, which is (D + 8) 2^-23 of 2^21, 35 at most, plus log(keys)."""
    D, keys, P = 128, 600, 16
    pages = -(-keys // P)
    t = np.arange(pages * P, dtype=np.float32)
    k = np.empty((1, pages * P, D), np.float32)
    k[..., :112] = 6.0
    k[..., 112:] = (t * step_up / 16)[:, None]
    v = np.random.default_rng(1).uniform(1, 3, (1, pages * P, D)).astype(np.float32)
    pools = [step.make_pool(x.reshape(1, pages, P, D).transpose(1, 0, 2, 3).copy()) for x in (k, v)]
    kd, vd = [step.read_pool(x, D)[:, 0].reshape(-1, D) for x in pools]
    q = torch.full((rows, 2, D), 1024.0, device="cuda")
    q[..., 112:] = 1.0
    scale = sign * 2.0 ** 21 / (1024.0 * 112 * kd[0, 0])
    q *= sign
    q[..., 112:] /= abs(scale)
    q = q.to(tdt(dtype))
    out, lse = torch.empty_like(q), torch.empty((rows, 2), device="cuda")
    dkv.dkv_paged_attend(q, dev(pools[0]), dev(pools[1]), i32(np.arange(pages)[None]), i32([keys]), out,
                         row_start=i32([0, rows]), max_rows=rows, scale=scale, lse=lse)
    got, low = host(out), host(lse)
    half = HALF[dtype]
    for i in range(rows):
        n = keys - rows + 1 + i
        assert np.all(got[i] >= vd[:n].min(0) * (1 - 2 * half - 2.0 ** -10)), (i, got[i].min())
        assert np.all(got[i] <= vd[:n].max(0) * (1 + 2 * half + 2.0 ** -10)), (i, got[i].max())
        s = scale * (kd[:n] @ host(q)[i].T)
        assert np.all(np.abs(low[i] - s.max(0)) <= 36 + np.log(n))


# ---- a wait that runs out ------------------------------------------------------------------------

@pytest.mark.parametrize("keys,B", [(100, 3), (3000, 2)])
def test_withheld_outputs_time_out_then_recover(keys, B):
    """The many-row kernel's waits for its outputs run out: out and lse of every row are NaN, whether a CTA holds
    a whole item or a piece of one, and the next call is right."""
    rows, Hkv, D, P = 40, 2, 128, 16
    rng = np.random.default_rng(3)
    pages = -(-keys // P)
    pools = [dev(step.make_pool(rng.standard_normal((pages, Hkv, P, D)).astype(np.float32))) for _ in "kv"]
    q = torch.from_numpy(rng.standard_normal((B * rows, 4, D)).astype(np.float32)).bfloat16().cuda()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    args = (q, *pools, i32(np.broadcast_to(np.arange(pages, dtype=np.int32), (B, pages))), i32([keys] * B))
    kw = dict(row_start=i32(np.arange(B + 1) * rows), max_rows=rows)
    dkv.dkv_paged_attend(*args, out, lse=lse, **kw)
    torch.cuda.synchronize()
    late, low = torch.zeros_like(out), torch.zeros_like(lse)
    dkv.dkv_paged_attend_debug_withhold(True)
    try:
        dkv.dkv_paged_attend(*args, late, lse=low, **kw)
        torch.cuda.synchronize()
    finally:
        dkv.dkv_paged_attend_debug_withhold(False)
    assert late.float().isnan().all()
    assert low.isnan().all()
    dkv.dkv_paged_attend(*args, late, lse=low, **kw)
    torch.cuda.synchronize()
    assert out.float().isfinite().all() and torch.equal(late, out) and torch.equal(low, lse)


# ---- scales of the append --------------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [41.0, 47.0, 0.37, 1e-30, 2.0 ** 127])
def test_append_divides_by_the_scales(D, scale):
    """The pools hold k / scale and v / scale, rounded once: 41 times a number half way between two codes is
    that number again when divided by 41, and lies below it when multiplied by the rounded 1 / 41."""
    Hkv, P, N = 2, 16, 32
    tie = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 2, np.float32)
    x = np.tile(tie, D // 16) * np.float32(41) * (1 + np.arange(N * Hkv, dtype=np.float32).reshape(N, Hkv, 1) % 8 / 8)
    k = torch.from_numpy(x.astype(np.float16)).cuda()
    v = torch.from_numpy(x[::-1].astype(np.float16)).cuda()
    pools = [torch.zeros((N // P, Hkv, P * D * 9 // 16), dtype=torch.uint8, device="cuda") for _ in "kv"]
    dkv.dkv_qkv_append(None, k, v, None, i32(np.arange(N)), *pools, k_scale=scale, v_scale=scale)
    s = np.float32(scale)
    moved = 0
    for pool, t in zip(pools, (k, v)):
        y = t.float().cpu().numpy()
        code, sc = step.quantise(y / s)
        other = step.quantise(y * (np.float32(1) / s))
        moved += int((code != other[0]).sum() + (sc != other[1]).sum())
        raw, got = step.pool_views(pool.cpu().numpy(), D)
        rows = lambda a: a.transpose(0, 2, 1, 3).reshape(N, Hkv, -1)  # noqa: E731
        assert np.array_equal(rows(got), sc)
        assert np.array_equal(rows(raw), code[..., 0::2] | (code[..., 1::2] << 4))
    assert moved > 0 or scale != 41.0  # the two differ here


# ---- a capture that torch does not know ------------------------------------------------------------

@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("given", [False, True])
def test_foreign_capture_needs_a_workspace(rows, given):
    """A workspace of torch's allocator is free again behind the call: fine in a graph whose memory pool torch
    keeps, not in one that it does not know.  Such a capture is refused without a workspace, and replays
    with one."""
    try:
        rt = ctypes.CDLL("libcudart.so.13")
    except OSError:
        pytest.skip("no shared CUDA runtime")
    ok = lambda e: pytest.fail(f"CUDA error {e}") if e else None  # noqa: E731
    rng = np.random.default_rng(3)
    pools = [dev(step.make_pool(rng.standard_normal((32, 2, 16, 64)).astype(np.float32))) for _ in "kv"]
    q = torch.from_numpy(rng.standard_normal((rows, 4, 64)).astype(np.float32)).half().cuda()
    want, out = torch.zeros_like(q), torch.zeros_like(q)
    args = (q, *pools, i32(np.arange(32)[None]), i32([500]))
    kw = dict(row_start=i32([0, rows]), max_rows=rows)
    dkv.dkv_paged_attend(*args, want, **kw)
    ws = torch.empty(dkv.dkv_paged_attend_workspace(1, 4, 2, 64, rows), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    if given:  # the call's own stream, another one than the current
        kw["stream"] = s
    torch.cuda.synchronize()
    raw, graph, ex = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p(), ctypes.c_void_p()
    with torch.cuda.stream(torch.cuda.current_stream() if given else s):
        ok(rt.cudaStreamBeginCapture(raw, 2))  # relaxed
        try:
            with pytest.raises(ValueError, match="needs a workspace"):
                dkv.dkv_paged_attend(*args, out, **kw)
            dkv.dkv_paged_attend(*args, out, workspace=ws, **kw)
        finally:
            ended = rt.cudaStreamEndCapture(raw, ctypes.byref(graph))
    ok(ended)
    ok(rt.cudaGraphInstantiate(ctypes.byref(ex), graph, ctypes.c_ulonglong(0)))
    ok(rt.cudaGraphLaunch(ex, raw))
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    ok(rt.cudaGraphExecDestroy(ex))
    ok(rt.cudaGraphDestroy(graph))
    # one of torch's needs none, on the capturing stream or on one that joined the capture
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        dkv.dkv_paged_attend(*args, out, **kw)
        torch.cuda.current_stream().wait_stream(s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ---- pages that are none -----------------------------------------------------------------------------

@pytest.mark.parametrize("P", [16, 256])
def test_plan_pages_outside_the_pool_are_padding(P):
    """A page index whose slots pass 2^32 must not come back as a slot of another page."""
    pages = 64
    bad = [-1, pages, (1 << 32) // P // 2 + 3, (1 << 31) - 1, -(1 << 31), -((1 << 31) // P) + 5, (1 << 28) + 1]
    B = len(bad) + 1
    table = np.full((B, 4), -1, np.int32)
    table[:-1, 0] = bad
    table[-1, 0] = 5
    free = np.full(pages, -1, np.int32)
    free[:4] = [9, 1 << 28, -7, pages - 1]  # two sequences take pages, one of them no page of the pool
    length, new = np.full(B, P - 2, np.int32), np.full(B, 2, np.int32)
    new[[0, 1, 2]] = 4
    case = (length, new, table, free, 4)
    want = check_plan(case, P, 40)
    assert want["report"][0] == 0
    live = want["slot"][:want["report"][1]]
    assert sorted(live[live >= 0]) == sorted([5 * P + P - 2, 5 * P + P - 1, (pages - 1) * P, (pages - 1) * P + 1])


# ---- every tile of every item counts once ------------------------------------------------------------

def run_tiles(case):
    N = int(case.start[-1]) + 3  # three rows of no sequence
    q = dev(np.broadcast_to(case.q[None, :, None], (N, case.Hq, case.D)), tdt(case.dtype))
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    dkv.dkv_paged_attend(q, *[dev(p) for p in case.pools], i32(case.table), i32(case.lens), out,
                         row_start=i32(case.start), max_rows=max(1, max(case.rows)), scale=case.scale, lse=lse)
    return host(out), host(lse)


@pytest.mark.parametrize("name", CASES)
def test_every_tile_counts_once(name):
    case = Tiles(*CASES[name])
    out, lse = run_tiles(case)
    for b, n in enumerate(case.rows):
        at = slice(case.start[b], case.start[b] + n)
        if n:
            assert case.bad(b, out[at], lse[at], case.reference(b)) == (0, 0), b
    assert np.all(out[case.start[-1]:] == 7) and np.all(lse[case.start[-1]:] == 7)


def test_many_rows_with_offsets_past_32_bits():
    # 4.6 GB pools, the pages at their end and one at their start
    case = Tiles([1000, 300], [90, 40], 16, 8, 128, "bf16")
    n, Hkv, nbytes = case.pools[0].shape
    pages = 46 * 10 ** 8 // (Hkv * nbytes)
    big = [torch.empty((pages, Hkv, nbytes), dtype=torch.uint8, device="cuda") for _ in "kv"]
    assert big[0].numel() > 1 << 32
    for b, p in zip(big, case.pools):
        b[0] = dev(p[:1])[0]
        b[pages - n:] = dev(p)
    table = np.where(case.table == 0, 0, case.table + pages - n)
    assert (table == 0).any() and table.max() > (1 << 32) // (Hkv * nbytes)
    N = int(case.start[-1])
    q = dev(np.broadcast_to(case.q[None, :, None], (N, 16, 128)), torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    dkv.dkv_paged_attend(q, *big, i32(table), i32(case.lens), out, row_start=i32(case.start), max_rows=90,
                         scale=case.scale, lse=lse)
    for b in range(2):
        at = slice(case.start[b], case.start[b + 1])
        assert case.bad(b, host(out)[at], host(lse)[at], case.reference(b)) == (0, 0), b


def test_public_calls_of_torch_do(monkeypatch):
    # a torch without the inner calls that the binding prefers
    rng = np.random.default_rng(3)
    pools = [dev(step.make_pool(rng.standard_normal((32, 2, 16, 64)).astype(np.float32))) for _ in "kv"]
    q = torch.from_numpy(rng.standard_normal((2, 4, 64)).astype(np.float32)).half().cuda()
    args = (q, *pools, i32(np.arange(32).reshape(2, 16)), i32([200, 100]))
    want, out, side = [torch.zeros_like(q) for _ in range(3)]
    dkv.dkv_paged_attend(*args, want)
    had = {n: getattr(torch._C, n) for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream", "_cuda_cudaCachingAllocator_raw_alloc",
                                            "_cuda_cudaCachingAllocator_raw_delete") if hasattr(torch._C, n)}
    dkv._torch_calls.cache_clear()
    try:
        with monkeypatch.context() as m:  # torch's public calls use some of them themselves
            for n in had:
                m.delattr(torch._C, n)
            public = dkv._torch_calls()
        assert not any(f in had.values() for f in public)
        dkv.dkv_paged_attend(*args, out)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        dkv.dkv_paged_attend(*args, side, stream=s)
        torch.cuda.synchronize()
        assert dkv._torch_calls() is public
    finally:
        dkv._torch_calls.cache_clear()
    assert torch.equal(out, want) and torch.equal(side, want)


ASYNC = """
import numpy as np, torch
import zero_copy_offloaded_gb300 as dkv
from oracle import paged_step as step
assert torch.cuda.get_allocator_backend() == "cudaMallocAsync"
rng = np.random.default_rng(3)
pools = [torch.from_numpy(step.make_pool(rng.standard_normal((32, 2, 16, 64)).astype(np.float32))).cuda() for _ in "kv"]
q = torch.from_numpy(rng.standard_normal((2, 4, 64)).astype(np.float32)).half().cuda()
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
args = (q, *pools, i(list(range(32))).view(2, 16), i([200, 100]))
want, out = torch.zeros_like(q), torch.zeros_like(q)
dkv.dkv_paged_attend(*args, want)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    dkv.dkv_paged_attend(*args, out)
g.replay()
torch.cuda.synchronize()
assert torch.equal(out, want)
print("as without a graph")
"""


def test_capture_with_another_allocator():
    # torch's cudaMallocAsync backend makes the workspace a node of the graph
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, PYTORCH_CUDA_ALLOC_CONF="backend:cudaMallocAsync", PYTHONPATH=root)
    r = subprocess.run([sys.executable, "-c", ASYNC], env=env, cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as without a graph" in r.stdout, r.stderr[-2000:]
