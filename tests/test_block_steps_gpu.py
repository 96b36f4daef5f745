"""The 8-bit step and the life of its pages together, as a serving program uses them: plan, append, attend, sequences
forked, reordered and ended, pages compacted, moved to the host and back, eagerly and as graphs.  The oracle keeps the
same table, stack, pools and scales; all of it has to be equal after every step."""
import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from oracle import block_step as bs
from oracle import pages as op
from oracle import paged_step as step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def tdt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float16


class Server:
    """A decoder layer's cache on the device, and the same by the oracle."""

    def __init__(self, B, Hq, Hkv, D, P, pages, max_pages, max_rows, dtype="bf16", cache=None):
        self.B, self.Hq, self.Hkv, self.D, self.P, self.pages, self.max_rows, self.dtype = B, Hq, Hkv, D, P, pages, max_rows, dtype
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.lengths, self.new, self.table = z(B), z(B), z(B, max_pages) - 1
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int().cuda()
        self.count, self.start, self.report = z(1) + pages, z(B + 1), z(4)
        self.pos, self.slot = z(max_rows), z(max_rows)
        self.sources, self.copies, self.moves, self.life = z(B), z(B, 2), z(pages // 2, 2), z(4)
        if cache is None:
            codes = [torch.full((pages, Hkv, P, D), 0x33, dtype=torch.uint8, device="cuda") for _ in "kv"]
            self.pools = [t.view(torch.float8_e4m3fn) for t in codes] + [torch.ones((pages, Hkv, P // 16), device="cuda") for _ in "kv"]
        else:
            cache.k_host[:] = cache.v_host[:] = 0x33
            self.pools = cache.pools
        self.rope = dkv.rope_table(2048, D, base=1e4)
        g = torch.Generator().manual_seed(2)
        self.gq, self.gk = [(1 + 0.1 * torch.randn(D, generator=g)).to(tdt(dtype)).cuda() for _ in "qk"]
        f = lambda *s: torch.zeros(s, dtype=tdt(dtype), device="cuda")  # noqa: E731
        self.qkv, self.q, self.out = f(max_rows, Hq + 2 * Hkv, D), f(max_rows, Hq, D), f(max_rows, Hq, D)
        self.lse = torch.zeros((max_rows, Hq), device="cuda")
        # the oracle's
        self.o = dict(lengths=np.zeros(B, np.int32), table=self.table.cpu().numpy(), free=self.free.cpu().numpy(), count=pages,
                      pools=[(np.full((pages, Hkv, P, D), 0x33, np.uint8), np.ones((pages, Hkv, P // 16), np.float32)) for _ in "kv"])
        self.rng = np.random.default_rng(5)

    # ---- on the device
    def device_step(self, max_rows):
        Hq, Hkv = self.Hq, self.Hkv
        dkv.dkv_step_plan(self.lengths, self.new, self.table, self.free, self.count, self.P, self.start, self.pos,
                          self.slot, self.lengths, self.count, self.report)
        dkv.dkv_block_append(self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:], self.pos, self.slot,
                             *self.pools, self.q, q_gamma=self.gq, k_gamma=self.gk, cos_sin=self.rope)
        dkv.dkv_block_attend(self.q, *self.pools, self.table, self.lengths, self.out, row_start=self.start,
                             max_rows=max_rows, lse=self.lse)

    def device_fork(self):
        dkv.dkv_pages_fork(self.table, self.lengths, self.sources, self.free, self.count, self.P, self.table, self.lengths,
                           self.count, self.copies, self.life)
        dkv.dkv_pages_copy(self.copies, self.pools)

    def device_compact(self):
        dkv.dkv_pages_compact(self.table, self.lengths, self.P, self.table, self.free, self.count, self.moves, self.life)
        dkv.dkv_pages_copy(self.moves, self.pools)

    # ---- both, and compared
    def same(self):
        torch.cuda.synchronize()
        o = self.o
        assert np.array_equal(self.lengths.cpu().numpy(), o["lengths"]) and int(self.count) == o["count"]
        assert np.array_equal(self.table.cpu().numpy(), o["table"]) and np.array_equal(self.free.cpu().numpy(), o["free"])
        for i, (code, scale) in enumerate(o["pools"]):
            assert np.array_equal(self.pools[2 + i].cpu().numpy(), scale)
            assert np.array_equal(self.pools[i].view(torch.uint8).cpu().numpy(), code)

    def step(self, new, run=None):
        o, n = self.o, int(sum(x for x in new if x > 0))
        size = np.exp(self.rng.standard_normal((self.max_rows, 1, 1)))  # some tokens are larger: scales grow
        x = self.rng.standard_normal((self.max_rows, self.Hq + 2 * self.Hkv, self.D)) * size
        self.qkv.copy_(torch.from_numpy(x.astype(np.float32)))
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.out.fill_(7.0)
        (run or self.device_step)(max(1, max(new)))
        plan = step.plan(o["lengths"], np.array(new, np.int32), o["table"], o["free"], o["count"], self.P, self.max_rows)
        assert plan["report"][0] == 0
        o.update(table=plan["table"], free=plan["free"], lengths=plan["kv_len"], count=plan["free_left"])
        f = lambda t: t.float().cpu().numpy()  # noqa: E731
        x, slot = f(self.qkv), plan["slot"]
        y = step.turn(x[:, self.Hq:self.Hq + self.Hkv], f(self.gk), 1e-6, self.rope.cpu().numpy(), plan["pos"], False)[0]
        o["pools"] = [bs.append(rows, slot, *pool)[:2] for rows, pool in zip((y, x[:, self.Hq + self.Hkv:]), o["pools"])]
        self.same()
        k, v = [bs.values(*pool) for pool in o["pools"]]
        ref = step.attend(self.q.double().cpu().numpy()[:n], k, v, o["table"], o["lengths"], plan["row_start"], self.D ** -0.5)
        out, low = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        assert np.all(out[n:] == 7)
        most = o["pools"][1][1].max()  # see test_block_attend_gpu.py for the bound
        codes = np.abs(bs.decode(o["pools"][1][0])).max() * most * ref["keys"][..., None]
        lv = np.abs(np.log2(o["pools"][1][1])).max()
        ds = (self.D + 8) * 2.0 ** -23 * ref["smax"] + 2.0 ** -20 + (ref["keys"] + lv) * 2.0 ** -23
        tol = HALF[self.dtype] * np.abs(ref["out"]) + ref["wabs"] * (2.0 ** -11 + 2 * ds[..., None]) + 2.0 ** -32 * codes + 2.0 ** -24
        assert np.all(np.abs(out[:n] - ref["out"]) <= tol), new
        assert np.all(np.abs(low[:n] - ref["lse"]) <= ds + 2.0 ** -22 * np.abs(ref["lse"]))

    def fork(self, sources, run=None):
        o = self.o
        self.sources.copy_(torch.tensor(sources, dtype=torch.int32))
        (run or self.device_fork)()
        r = op.fork(o["table"], o["lengths"], sources, o["free"], o["count"], self.P, o["table"])
        assert self.life.tolist() == r["report"] and r["report"][0] == 0
        o.update(table=r["table"], lengths=r["lengths"], free=r["free"], count=r["free_left"])
        self.move(r["copies"])
        self.same()

    def compact(self, run=None):
        o = self.o
        (run or self.device_compact)()
        r = op.compact(o["table"], o["lengths"], self.pages, self.P, self.pages // 2, o["table"], o["free"])
        assert self.life.tolist() == r["report"]
        o.update(table=r["table"], free=r["free"], count=r["free_left"])
        self.move(r["moves"])
        self.same()

    def move(self, pairs):
        for code, scale in self.o["pools"]:
            was = code.copy(), scale.copy()
            for a, b in pairs:
                if a >= 0:
                    code[b], scale[b] = was[0][a], was[1][a]


FIRST = [40, 0, 130, 0, 7, 0]
STORY = [  # each step, and what the sequences become after it
    ([1, 0, 1, 0, 3, 0], [0, 0, 2, 2, 4, 4]), ([1] * 6, [1, 1, 3, 2, 4, 5]), ([1, 5, 1, 17, 1, 1], None), ([1] * 6, [0, 0, -1, 3, 3, 3]),
    ([33, 1, 0, 1, 1, 1], [5, 1, 3, 0, -1, 3]), ([1, 1, 1, 1, 20, 1], "compact"), ([1] * 6, [0, 0, 0, 0, 0, 0]), ([1, 2, 3, 4, 5, 6], [3, 1, 2, 0, -1, -1]),
    ([1, 1, 1, 1, 0, 0], "compact"), ([1, -1, 1, 1, 9, 0], [0, 2, 2, 0, 4, 4])]


@pytest.mark.parametrize("Hq,Hkv,D,P,dtype", [(8, 2, 128, 16, "bf16"), (4, 4, 64, 32, "fp16"), (12, 1, 64, 64, "bf16")])
def test_a_story(Hq, Hkv, D, P, dtype):
    s = Server(6, Hq, Hkv, D, P, 96, 24, 256, dtype)
    s.step(FIRST)
    for new, then in STORY:
        if -1 in new:  # a sequence that shares pages ends by a fork: alone it may end by the plan
            s.fork([b if n >= 0 else -1 for b, n in enumerate(new)])
            new = [max(n, 0) for n in new]
        s.step(new)
        if then == "compact":
            s.compact()
        elif then:
            s.fork(then)


def test_a_story_in_pinned_memory():
    cache = dkv.PagedKVCache(6, 2, 128, 16, 96, 24, kv_format="e4m3_block")
    try:
        assert cache.k_host.shape == (96, 2, 16, 128) and [tuple(t.shape) for t in cache.pools[2:]] == [(96, 2, 1)] * 2
        s = Server(6, 8, 2, 128, 16, 96, 24, 256, cache=cache)
        s.step(FIRST)
        for new, then in STORY[:6]:
            s.step(new)
            s.compact() if then == "compact" else s.fork(then) if then else None
        x = torch.zeros((6, 1, 128), dtype=torch.bfloat16, device="cuda")
        w = torch.zeros((128, 1024), dtype=torch.bfloat16, device="cuda")
        for call in (cache.decode, cache.prefill):
            with pytest.raises(dkv.DkvError, match="block scales"):
                call(x, w, w, w, 8, torch.zeros((6, 1, 8, 128), dtype=torch.bfloat16, device="cuda"))
        want, low = s.out.clone(), s.lse.clone()
        n = int(s.start[-1])
        s.out.fill_(0)
        if then != "compact":
            n = 0
        cache.attend(s.q, s.table, s.lengths, s.out, row_start=s.start, max_rows=20, lse=s.lse)
        assert torch.equal(s.out[:n], want[:n]) and torch.equal(s.lse[:n], low[:n])
        k = torch.zeros((6, 2, 128), dtype=torch.bfloat16, device="cuda")
        cache.append(s.q[:6], k, k, None, torch.full((6,), -1, dtype=torch.int32, device="cuda"), s.q[:6].clone())
        torch.cuda.synchronize()
        s.same()
    finally:
        cache.free()


def test_a_story_as_graphs():
    """The step, the fork and the compaction captured once and replayed, the copies of a fork in its graph."""
    s = Server(6, 8, 2, 128, 16, 96, 24, 64)
    kept = [s.lengths, s.table, s.free, s.count, *s.pools]
    saved = [t.clone() for t in kept]
    graphs = {}
    for name, f in (("step", lambda: s.device_step(4)), ("fork", s.device_fork), ("compact", s.device_compact)):
        f()  # loads the kernels
        torch.cuda.synchronize()
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            f()
    for t, v in zip(kept, saved):
        t.copy_(v)
    s.step([40, 0, 16, 0, 7, 0])  # a prompt, outside the graph
    for i, (new, then) in enumerate(STORY):
        s.step([min(max(n, 0), 4) for n in new], lambda rows: graphs["step"].replay())
        if then == "compact":
            s.compact(graphs["compact"].replay)
        elif then:
            s.fork(then, graphs["fork"].replay)


def test_pages_leave_for_the_host_and_come_back():
    """A sequence's pages to pinned memory, its places given away, then back to other pages: it goes on as if nothing had been."""
    s = Server(3, 8, 2, 128, 16, 64, 16, 256)
    s.step([70, 33, 5])
    s.step([1, 1, 1])
    host = [torch.empty((8, *t.shape[1:]), dtype=t.dtype, pin_memory=True) for t in s.pools]
    held = s.table[0, :5].clone()
    out = torch.stack((held, torch.arange(5, dtype=torch.int32, device="cuda")), -1).contiguous()
    dkv.dkv_pages_copy(out, s.pools, host)
    s.fork([-1, 1, 2])
    s.step([0, 40, 3])  # others take the pages
    # back: 71 rows on pages from the stack
    take = s.free[int(s.count) - 5:int(s.count)].clone()
    back = torch.stack((out[:, 1], take), -1).contiguous()
    dkv.dkv_pages_copy(back, host, s.pools)
    s.table[0, :5] = take
    s.lengths[0] = 71
    s.count -= 5
    torch.cuda.synchronize()
    o = s.o
    o["table"][0, :5], o["lengths"][0], o["count"] = take.cpu().numpy(), 71, o["count"] - 5
    for i, (code, scale) in enumerate(o["pools"]):
        code[take.cpu().numpy()], scale[take.cpu().numpy()] = host[i][:5].view(torch.uint8).numpy(), host[2 + i][:5].numpy()
    s.same()
    s.step([1, 1, 1])
