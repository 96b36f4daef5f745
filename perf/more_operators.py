"""A paged cache held in 8 bits, and the life of its pages, operator by operator, with their plain forms.

Five operators serve a decoder over a cache of E4M3 codes with one scale for each block of 16 tokens of a KV head:

* ``append``: queries and keys are normalised per head and rotated to their positions, keys and values go to their
  slots; a block's scale is the smallest power of two that holds its largest value, and grows with it;
* ``attend``: softmax attention of ragged query rows over that cache;
* ``fork``: sequences go on as copies of others, or end: full pages are shared, a partly filled one is copied,
  pages that nobody holds any more go back to the free stack;
* ``copy``: pages of some pools to other pages of them, or of other pools;
* ``compact``: the pages in use move to the front of the pool.

A pool is [pages, KV heads, page_tokens, D] of E4M3 codes, its scales [pages, KV heads, page_tokens / 16] in 32 bits.
"""
import math

import torch

own = False

F32, I32 = torch.float32, torch.int32
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 16
EPS = 2.0 ** -20
ROPE_BASE = 500000.0


def listed():
    return [
        # the eight fresh tokens of the Llama-3-8B-shaped decode, each somewhere inside a block of its sequence
        dict(name="append_decode_8", op="append", rows=8, seqs=8, hq=32, hkv=8, d=128, dtype="bf16", norm=True,
             rot=128, inter=False, page=16, far=131072),
        # its 4096-token prefill chunk
        dict(name="append_prefill_4096", op="append", rows=4096, seqs=1, hq=32, hkv=8, d=128, dtype="bf16",
             norm=True, rot=128, inter=False, page=16, far=32768),
        # the smallest decode: one sequence, 2 KV heads, where latency counts
        dict(name="attend_tiny", op="attend", batch=1, new=1, hq=8, hkv=2, d=64, dtype="bf16", keys=2049,
             ragged=False, page=16, host=False),
        # the Llama-3-8B-shaped decode, pool in HBM
        dict(name="attend_8x32k", op="attend", batch=8, new=1, hq=32, hkv=8, d=128, dtype="bf16", keys=32769,
             ragged=False, page=16, host=False),
        # many sequences of any length (none for some), a few drafted tokens each, fp16, heads of 64
        dict(name="attend_ragged_48", op="attend", batch=48, new=5, hq=32, hkv=8, d=64, dtype="fp16",
             keys=8193, ragged=True, page=32, host=False),
        # the 4096-token prefill chunk over 28 672 cached tokens
        dict(name="attend_prefill_4096", op="attend", batch=1, new=4096, hq=32, hkv=8, d=128, dtype="bf16",
             keys=32768, ragged=False, page=16, host=False),
        # one step of four beams for each of 16 prompts: each beam goes on as one of its prompt's four
        dict(name="fork_beams_64", op="fork", batch=64, group=4, ended=0.0, page=16, max_len=4096),
        # a scheduler's round over 512 places: some sequences have ended, some are sampled several times
        dict(name="fork_mixed_512", op="fork", batch=512, group=8, ended=0.25, page=16, max_len=32768),
        # the partly filled pages of 64 forks, codes and scales of keys and values
        dict(name="copy_forks_64", op="copy", pairs=64, live=0.75, pages=4096, hkv=8, d=128, page=16, host=False),
        # what a compaction moves
        dict(name="copy_moves_8192", op="copy", pairs=8192, live=1.0, pages=20480, hkv=8, d=128, page=32, host=False),
        # a pool of 64 sequences of any length, less than half of it in use
        dict(name="compact_64", op="compact", batch=64, group=4, page=16, max_len=4096, spare=1.0),
        # a pool of 512 long sequences, pages shared by the samples of a prompt
        dict(name="compact_512", op="compact", batch=512, group=4, page=16, max_len=32768, spare=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "append", "attend", "attend", "attend", "fork", "copy", "compact"))
    page = rng.choice((16, 32, 64, 128))
    hkv = rng.choice((1, 2, 4, 8, 8, 32))
    d = rng.choice((64, 128))
    if op == "fork":
        return dict(op=op, batch=_log(rng, 1, 512), group=rng.choice((1, 2, 3, 4, 8)),
                    ended=rng.choice((0.0, 0.1, 0.5)), page=page, max_len=_log(rng, 64, 32768))
    if op == "compact":
        return dict(op=op, batch=_log(rng, 1, 512), group=rng.choice((1, 2, 4)), page=page, max_len=_log(rng, 64, 32768),
                    spare=rng.choice((1.0, 1.25, 2.0)))
    if op == "copy":
        most = 8192 * 8 * 128 * 32 // (hkv * d * page)
        pairs = _log(rng, 1, max(2, min(16384, most)))
        host = rng.random() < 0.2
        pairs = max(1, pairs // 16) if host else pairs
        return dict(op=op, pairs=pairs, live=rng.choice((0.5, 1.0)), hkv=hkv, d=d, page=page, host=host,
                    pages=2 * pairs + rng.randint(1, 4096 if most > 16384 else 64))
    group = 1 if hkv == 32 else rng.choice((1, 2, 3, 4, 4, 5, 7, 8))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "append":
        rows = min(_log(rng, 1, 16384), 4096 * 48 * 128 // ((hkv * group + 2 * hkv) * d))
        return dict(op=op, rows=rows, seqs=min(rows, rng.choice((1, 2, 7, 64, 1024))), hq=hkv * group, hkv=hkv, d=d,
                    dtype=dtype, norm=rng.random() < 0.6, rot=rng.choice((0, 32, d, d)), inter=rng.random() < 0.4,
                    page=page, far=_log(rng, 64, 131072))
    new = rng.choice((1, 1, 1, _log(rng, 2, 8), _log(rng, 9, 700)))
    batch = _log(rng, 1, 48 if new <= 8 else 6)
    most = 8 * 32769 * 8 * 128 // (batch * hkv * d)
    if new > 8:
        most = min(most, 600_000_000 // (batch * new * hkv * group))
    keys = max(new, min(_log(rng, 1, 131073), most))
    host = new == 1 and rng.random() < 0.15
    return dict(op=op, batch=batch, new=new, hq=hkv * group, hkv=hkv, d=d, dtype=dtype,
                keys=min(keys, 32769) if host else keys, ragged=rng.random() < 0.5, page=page, host=host)


# ---- inputs -------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 29)


def _need(top):
    """The smallest power of two that brings `top` to at most 448, from 2^-64 on."""
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    k = torch.where(top > 0, e - 9 + (m > 0.875), -64).clamp(-64, 120)
    return torch.ldexp(torch.ones_like(top), k)


def _random_pool(pages, hkv, page, d, g):
    """Codes and scales of rows that are normal but for one channel in 32 that is eight times as large."""
    pool = torch.empty((pages, hkv, page, d), dtype=F8, device="cuda")
    scales = torch.empty((pages, hkv, page // BLOCK), dtype=F32, device="cuda")
    wide = torch.where(torch.rand((hkv, 1, d), generator=g, device="cuda") < 1 / 32, 8.0, 1.0)
    step = max(1, (1 << 26) // (hkv * page * d))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        y = torch.randn((n, hkv, page, d), generator=g, device="cuda") * wide
        s = _need(y.abs().unflatten(2, (-1, BLOCK)).amax((-1, -2)))
        scales[at:at + n] = s
        pool[at:at + n] = (y / s.repeat_interleave(BLOCK, 2)[..., None]).to(F8)
    return pool, scales


def _rope_table(n, rot):
    freq = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), -1).to(F32)


def _prepare_append(c, seed):
    g = _gen(seed)
    n, seqs, hq, hkv, d, page, dt = c["rows"], c["seqs"], c["hq"], c["hkv"], c["d"], c["page"], TYPES[c["dtype"]]
    qkv = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device="cuda")  # one projection's output
    qkv = (qkv * (0.25 + 2 * torch.rand((n, 1), generator=g, device="cuda"))).to(dt)
    q, k, v = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
    gamma = [(1 + 0.1 * torch.randn((d,), generator=g, device="cuda")).to(dt) if c["norm"] else None for _ in "qk"]
    # the rows of a sequence follow one another from a position of its own on, in pages of its own
    row = torch.arange(n, device="cuda")
    seq = row * seqs // n
    start = (torch.arange(seqs, device="cuda") * n + seqs - 1) // seqs
    first = torch.randint(0, max(1, c["far"] - n // seqs - 1), (seqs,), generator=g, device="cuda")
    pos = first[seq] + row - start[seq]
    per = (n // seqs + 1) // page + 2  # pages that a sequence's rows can touch
    pages = seqs * per + 3
    order = torch.randperm(pages, generator=g, device="cuda")
    slot = order[seq * per + pos // page - first[seq] // page] * page + pos % page
    pools = [_random_pool(pages, hkv, page, d, g) for _ in "kv"]
    return dict(c=c, q=q.unflatten(-1, (hq, d)), k=k.unflatten(-1, (hkv, d)), v=v.unflatten(-1, (hkv, d)),
                q_gamma=gamma[0], k_gamma=gamma[1], pos=pos.to(I32), slot=slot.to(I32),
                cos_sin=_rope_table(c["far"] + n, c["rot"]) if c["rot"] else None,
                k_pool=pools[0][0], v_pool=pools[1][0], k_scales=pools[0][1], v_scales=pools[1][1],
                q_out=torch.empty((n, hq, d), dtype=dt, device="cuda"))


def _prepare_attend(c, seed):
    g = _gen(seed)
    b, hq, hkv, d, page, dt = c["batch"], c["hq"], c["hkv"], c["d"], c["page"], TYPES[c["dtype"]]
    kv = torch.full((b,), c["keys"], dtype=I32, device="cuda")
    rows = torch.full((b,), c["new"], dtype=I32, device="cuda")
    if c["ragged"]:  # the last is the longest; lengths down to none
        kv = torch.randint(0, c["keys"] + 1, (b,), generator=g, device="cuda", dtype=I32)
        kv[b - 1] = c["keys"]
        if c["new"] > 1:
            rows = torch.randint(1, c["new"] + 1, (b,), generator=g, device="cuda", dtype=I32)
            rows = torch.minimum(rows, kv)
    start = torch.zeros((b + 1,), dtype=I32, device="cuda")
    start[1:] = torch.cumsum(rows, 0)
    n = b * c["new"]  # the rows behind the last sequence are padding
    max_pages = -(-c["keys"] // page)
    pages = b * max_pages
    table = torch.randperm(pages, generator=g, device="cuda").to(I32).view(b, max_pages)
    (kp, ks), (vp, vs) = (_random_pool(pages, hkv, page, d, g) for _ in "kv")
    if c["host"]:  # codes in pinned host memory, read across the link; scales stay on the device
        kp, vp = (torch.empty(p.shape, dtype=F8, pin_memory=True).copy_(p) for p in (kp, vp))
    q = torch.randn((n, hq, d), generator=g, device="cuda").to(dt)
    return dict(c=c, q=q, k_pool=kp, v_pool=vp, k_scales=ks, v_scales=vs, table=table, kv_len=kv,
                start=start if c["new"] > 1 else None,  # a row each needs no starts
                out=torch.zeros((n, hq, d), dtype=dt, device="cuda"),
                lse=torch.zeros((n, hq), dtype=F32, device="cuda"))


def _sequences(c, g, pool):
    """Lengths and table of a batch whose places come in groups that share the full pages of a prompt."""
    b, page = c["batch"], c["page"]
    max_pages = -(-c["max_len"] // page)
    lengths = torch.randint(0, c["max_len"] + 1, (b,), generator=g, device="cuda")
    lead = torch.arange(b, device="cuda") // c["group"] * c["group"]
    prompt = lengths[lead] // (2 * page)  # pages that the group shares
    lengths = torch.maximum(lengths, prompt * page)
    held = (lengths + page - 1) // page
    col = torch.arange(max_pages, device="cuda")
    alone = (col < held[:, None]) & ((col >= prompt[:, None]) | (lead == torch.arange(b, device="cuda"))[:, None])
    at = torch.cumsum(alone.flatten(), 0).view(b, max_pages) - 1
    used = int(at[-1, -1]) + 1
    pages = int(b * max_pages * pool) + b + 1
    order = torch.randperm(pages, generator=g, device="cuda")
    table = torch.where(alone, order[at.clamp(min=0)], -1)
    table = torch.where((col < prompt[:, None]) & (col < held[:, None]), table[lead], table)
    return lengths.to(I32), table.to(I32).contiguous(), order[used:].to(I32), pages


def _prepare_fork(c, seed):
    g = _gen(seed)
    b, group = c["batch"], c["group"]
    lengths, table, spare, pages = _sequences(c, g, 1.0)
    place = torch.arange(b, device="cuda")
    lead = place // group * group
    sources = lead + torch.randint(0, group, (b,), generator=g, device="cuda")
    sources = torch.where(torch.rand((b,), generator=g, device="cuda") < 0.5, place, sources).clamp(max=b - 1)
    sources = torch.where(torch.rand((b,), generator=g, device="cuda") < c["ended"], -1, sources)
    free = torch.full((pages,), -1, dtype=I32, device="cuda")
    free[:len(spare)] = spare
    return dict(c=c, lengths=lengths, table=table, sources=sources.to(I32), free=free,
                free_count=torch.tensor([len(spare)], dtype=I32, device="cuda"),
                table_out=torch.full_like(table, -1), len_out=torch.zeros_like(lengths),
                free_left=torch.zeros((1,), dtype=I32, device="cuda"),
                copies=torch.zeros((b, 2), dtype=I32, device="cuda"), report=torch.zeros((4,), dtype=I32, device="cuda"))


def _prepare_compact(c, seed):
    g = _gen(seed)
    lengths, table, spare, pages = _sequences(c, g, c["spare"])
    return dict(c=c, lengths=lengths, table=table, pages=pages, table_out=torch.full_like(table, -1),
                free=torch.full((pages,), -1, dtype=I32, device="cuda"),
                free_left=torch.zeros((1,), dtype=I32, device="cuda"),
                moves=torch.zeros((pages // 2, 2), dtype=I32, device="cuda"),
                report=torch.zeros((4,), dtype=I32, device="cuda"))


def _prepare_copy(c, seed):
    g = _gen(seed)
    n, pages, hkv, d, page = c["pairs"], c["pages"], c["hkv"], c["d"], c["page"]
    order = torch.randperm(pages, generator=g, device="cuda")
    pairs = torch.stack((order[:n], order[n:2 * n]), -1).to(I32)
    live = torch.rand((n, 1), generator=g, device="cuda") < c["live"]
    pairs = torch.where(live, pairs, -1).to(I32).contiguous()
    pools = []
    for _ in "kv":
        codes = torch.randint(0, 256, (pages, hkv, page, d), generator=g, device="cuda", dtype=torch.uint8) & 0x77
        pools += [codes.view(F8), torch.rand((pages, hkv, page // BLOCK), generator=g, device="cuda")]
    into = pools
    if c["host"]:  # pages leave for pinned host memory
        into = [torch.zeros(p.shape, dtype=p.dtype, pin_memory=True) for p in pools]
    return dict(c=c, pairs=pairs, pools=pools, into=into)


def prepare(case, seed):
    return {"append": _prepare_append, "attend": _prepare_attend, "fork": _prepare_fork, "copy": _prepare_copy,
            "compact": _prepare_compact}[case["op"]](case, seed)


# ---- plain forms --------------------------------------------------------------------------------------

def _plain_rows(x, gamma, eps, table, inter):
    """Norm (if gamma) and rotation (if a table's rows) of x [N, H, D], in 32 bits with the norm's sum in 64."""
    y = x.to(F32)
    if gamma is not None:
        mean = x.to(torch.float64).square().mean(-1, keepdim=True)
        y = y * (1.0 / torch.sqrt(mean + eps)).to(F32) * gamma.to(F32)
    if table is None:
        return y
    half = table.shape[-1] // 2
    cos, sin = table[:, None, :half], table[:, None, half:]
    if inter:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
    else:
        a, b = y[..., :half], y[..., half:2 * half]
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((turned, y[..., 2 * half:]), -1)


def _plain_store(y, slot, pool, scales, page):
    h, d = y.shape[1:]
    block, at = torch.unique(slot // BLOCK, return_inverse=True)
    top = torch.zeros((len(block), h), device=y.device)
    top = top.scatter_reduce(0, at[:, None].expand(-1, h), y.abs().amax(-1), "amax")
    first = torch.zeros((len(block),), dtype=torch.bool, device=y.device)
    first[at[slot % BLOCK == 0]] = True
    pg, sub = block * BLOCK // page, block % (page // BLOCK)
    old = torch.where(first[:, None], 0.0, scales[pg, :, sub])
    new = torch.maximum(old, _need(top))
    scales[pg, :, sub] = new
    head, row = torch.arange(h, device=y.device), torch.arange(BLOCK, device=y.device)
    where = (pg[:, None, None], head[:, None], (sub * BLOCK)[:, None, None] + row)
    code = pool.view(torch.uint8)
    held = code[where].view(F8)  # [blocks, H, 16, D]
    grown = (held.to(F32) * torch.where(old > 0, old / new, 1.0)[..., None, None]).to(F8)
    code[where] = torch.where(((new > old) & (old > 0))[..., None, None], grown.view(torch.uint8), held.view(torch.uint8))
    put = (y / new[at][..., None]).to(F8)
    code[(slot // page)[:, None], head, (slot % page)[:, None]] = put.view(torch.uint8)


def _plain_append(s):
    c = s["c"]
    table = s["cos_sin"][s["pos"].long()] if s["cos_sin"] is not None else None
    q = _plain_rows(s["q"], s["q_gamma"], EPS, table, c["inter"]).to(s["q_out"].dtype)
    k = _plain_rows(s["k"], s["k_gamma"], EPS, table, c["inter"])
    slot = s["slot"].long()
    _plain_store(k, slot, s["k_pool"], s["k_scales"], c["page"])
    _plain_store(s["v"].to(F32), slot, s["v_pool"], s["v_scales"], c["page"])
    return {"q": q, "k": s["k_pool"], "v": s["v_pool"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _plain_read(pool, scales, table):
    """[B, KV heads, max_pages * page, D] in 32 bits."""
    at = table.long()
    code = pool.cuda().view(torch.uint8)[at].view(F8).to(F32)  # [B, pages, Hkv, page, D]
    return (code * scales[at].repeat_interleave(BLOCK, -1)[..., None]).transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    c = s["c"]
    b, hkv, d, new = c["batch"], c["hkv"], c["d"], c["new"]
    n, hq, _ = s["q"].shape
    group = hq // hkv
    dev = s["q"].device
    k, v = (_plain_read(s[x + "_pool"], s[x + "_scales"], s["table"]) for x in "kv")
    start = s["start"].long() if s["start"] is not None else torch.arange(b + 1, device=dev)
    rows = start[1:] - start[:-1]
    t = torch.arange(new, device=dev)
    live = t < rows[:, None]  # [B, new]
    row = torch.where(live, start[:-1, None] + t, 0)
    q = s["q"].to(F32)[row].unflatten(2, (hkv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, Hkv, new*G, D]
    score = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(d))
    at = s["kv_len"].long()[:, None] - rows[:, None] + t  # the row's own position
    seen = torch.arange(k.shape[2], device=dev) <= at[..., None]  # [B, new, S]
    seen = (seen & live[..., None]).repeat_interleave(group, 1)[:, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    score = torch.exp(score - top)
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score, torch.where(seen.any(2)[..., None], v, 0.0))
    o = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0)
    lse = (torch.log(total) + top)[..., 0]
    back = lambda x: x.unflatten(2, (new, group)).transpose(1, 2).flatten(2, 3)[live]  # noqa: E731
    out, low = torch.zeros_like(s["out"]), torch.zeros_like(s["lse"])
    out[:int(live.sum())] = back(o).to(out.dtype)
    low[:int(live.sum())] = back(lse)
    return {"out": out, "lse": low}


def _marks(table, held, pages):
    """Which pages of the pool the first `held` entries of each row name."""
    on = torch.arange(table.shape[1], device=table.device) < held[:, None]
    mark = torch.zeros((pages + 1,), dtype=torch.int64, device=table.device)
    mark[torch.where(on, table.long(), pages)] = 1
    return mark[:pages]


def _plain_fork(s):
    c = s["c"]
    page, dev = c["page"], s["table"].device
    b, max_pages = s["table"].shape
    pages = len(s["free"])
    place, col = torch.arange(b, device=dev), torch.arange(max_pages, device=dev)
    src = s["sources"].long()
    on = src >= 0
    at = src.clamp(min=0)
    length = s["lengths"].long()
    new_len = torch.where(on, length[at], 0)
    held, old_held = (new_len + page - 1) // page, (length + page - 1) // page
    # the heir of a source's last, partly filled page: itself, or the lowest place that goes on as it
    heir = torch.full((b + 1,), b, device=dev).scatter_reduce(0, torch.where(on, src, b), place, "amin")[:b]
    heir = torch.where(src == place, place, heir)
    need = (on & (new_len % page != 0) & (heir[at] != place)).long()
    table = s["table"].long()[at]
    shared = held - need  # the entries that are the source's own
    freed = _marks(s["table"], old_held, pages) & ~_marks(table, shared, pages)
    count = s["free_count"].long()
    rank = torch.cumsum(freed, 0)
    stack = count + rank[-1]
    ok = (need.sum() <= stack[0]) & (stack[0] <= pages) & (src < b).all()
    free = torch.cat((s["free"], s["free"][:1]))
    free[torch.where((freed > 0) & ok, count + rank - 1, pages)] = torch.arange(pages, dtype=I32, device=dev)
    free = free[:pages]
    taken = free[(stack - torch.cumsum(need, 0)).clamp(0, pages - 1)].long()
    last = table.gather(1, (held - 1).clamp(min=0)[:, None])[:, 0]
    pair = torch.where((need > 0)[:, None] & ok, torch.stack((last, taken), -1), -1)
    table = torch.where((need > 0)[:, None] & (col == held[:, None] - 1), taken[:, None], table)
    keep = torch.where(ok, held, old_held)
    table = torch.where(ok, table, s["table"].long())
    s["free"].copy_(free)
    s["table_out"].copy_(torch.where(col < keep[:, None], table, s["table_out"]))
    new_len = torch.where(ok, new_len, length)
    left = torch.where(ok, stack - need.sum(), count)
    zero = torch.zeros_like(rank[-1])
    report = torch.stack((torch.where(ok, zero, zero + 3), torch.where(ok, rank[-1], zero),
                          torch.where(ok, need.sum(), zero), new_len.max()))
    return {"table": s["table_out"], "lengths": new_len.to(I32), "free": free, "free_left": left.to(I32),
            "copies": pair.to(I32), "report": report.to(I32)}


def _plain_compact(s):
    c = s["c"]
    page, pages, dev = c["page"], s["pages"], s["table"].device
    held = (s["lengths"].long() + page - 1) // page
    live = _marks(s["table"], held, pages)
    count = live.sum()
    index = torch.arange(pages, device=dev)
    high = (live > 0) & (index >= count)
    hole = (live == 0) & (index < count)
    moved = high.sum()
    n = len(s["moves"])
    place = lambda m: torch.where(m, torch.cumsum(m.long(), 0) - 1, n)  # noqa: E731
    moves = torch.full((n + 1, 2), -1, device=dev)
    moves[place(high).clamp(max=n), 0] = index
    moves[place(hole).clamp(max=n), 1] = index
    moves = moves[:n]
    goes = torch.where(high, moves[place(high).clamp(max=n - 1), 1], index)
    on = torch.arange(s["table"].shape[1], device=dev) < held[:, None]
    table = goes[torch.where(on, s["table"].long(), 0)]
    s["table_out"].copy_(torch.where(on, table, s["table_out"]))
    s["free"].copy_(torch.where(index < pages - count, pages - 1 - index, s["free"].long()))
    report = torch.stack((torch.zeros_like(count), moved, count, s["lengths"].max().long()))
    return {"table": s["table_out"], "free": s["free"], "free_left": (pages - count).to(I32)[None],
            "moves": moves.to(I32), "report": report.to(I32)}


def _plain_copy(s):
    pairs = s["pairs"][s["pairs"][:, 0] >= 0].long()
    a, b = pairs[:, 0], pairs[:, 1]
    byte = lambda p: p.view(torch.uint8) if p.dtype == F8 else p  # noqa: E731
    if s["c"]["host"]:
        b = b.cpu()
        for x, y in zip(s["pools"], s["into"]):
            byte(y)[b] = byte(x)[a].cpu()
    else:
        for x, y in zip(s["pools"], s["into"]):
            byte(y)[b] = byte(x)[a]
    return {"pools": s["into"]}


def run(s):
    op = s["c"]["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "fork": _plain_fork, "copy": _plain_copy,
                "compact": _plain_compact}[op](s)
    import zero_copy_offloaded_gb300 as dkv
    c = s["c"]
    if op == "append":
        dkv.dkv_block_append(s["q"], s["k"], s["v"], s["pos"], s["slot"], s["k_pool"], s["v_pool"], s["k_scales"],
                             s["v_scales"], s["q_out"], q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=EPS,
                             cos_sin=s["cos_sin"], interleaved=c["inter"])
        return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"], "k_scales": s["k_scales"],
                "v_scales": s["v_scales"]}
    if op == "attend":
        dkv.dkv_block_attend(s["q"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"], s["table"], s["kv_len"],
                             s["out"], row_start=s["start"], max_rows=c["new"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "fork":
        dkv.dkv_pages_fork(s["table"], s["lengths"], s["sources"], s["free"], s["free_count"], c["page"],
                           s["table_out"], s["len_out"], s["free_left"], s["copies"], s["report"])
        return {"table": s["table_out"], "lengths": s["len_out"], "free": s["free"], "free_left": s["free_left"],
                "copies": s["copies"], "report": s["report"]}
    if op == "compact":
        dkv.dkv_pages_compact(s["table"], s["lengths"], c["page"], s["table_out"], s["free"], s["free_left"],
                              s["moves"], s["report"])
        return {"table": s["table_out"], "free": s["free"], "free_left": s["free_left"], "moves": s["moves"],
                "report": s["report"]}
    dkv.dkv_pages_copy(s["pairs"], s["pools"], s["into"])
    return {"pools": s["into"]}


# ---- what a pass cannot do without ----------------------------------------------------------------------

def work(c):
    op = c["op"]
    if op in ("fork", "compact"):
        # the entries of pages in use read and written, lengths, sources and pairs; a compaction also writes its stack
        most = c["batch"] * c["max_len"] // c["page"]
        more = 4 * int(most * c["spare"]) - 2 * most + 8 * most // 4 if op == "compact" else 0
        return {"bytes": 4 * most + 24 * c["batch"] + more, "flops": 0}
    d, hkv = c["d"], c["hkv"]
    if op == "copy":
        return {"bytes": 8 * c["pairs"] + 4 * c["pairs"] * c["live"] * hkv * c["page"] * (d + 4 / BLOCK), "flops": 0}
    hq, n = c["hq"], c.get("rows")
    if op == "append":
        per = 2 * (hq + 2 * hkv) * d + 2 * hq * d + 2 * hkv * d + 8  # read; q; codes; position and slot
        return {"bytes": n * (per + 4 * c["rot"]) + 8 * hkv * max(c["seqs"], n // BLOCK),
                "flops": n * (hq + hkv) * d * (4 * c["norm"] + 3 * (c["rot"] > 0))}
    share = 0.5 if c["ragged"] and c["batch"] > 1 else 1.0
    cached = c["batch"] * c["keys"] * share
    rows = c["batch"] * c["new"] * (share if c["new"] > 1 else 1.0)
    seen = rows * max(1.0, c["keys"] * share - (c["new"] - 1) / 2)
    return {"bytes": 2 * cached * hkv * (d + 4 / BLOCK) + rows * hq * (4 * d + 4), "flops": 4 * d * hq * seen}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------

def _exact_turn(x, gamma, table, inter):
    y = x.to(torch.float64)
    if gamma is not None:
        y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS).pow(0.5) * gamma.to(torch.float64)
    if table is not None:
        half = table.shape[-1] // 2
        turn = torch.complex(table[:, :half].double(), table[:, half:].double())[:, None]
        first = slice(0, 2 * half, 2) if inter else slice(0, half)
        second = slice(1, 2 * half, 2) if inter else slice(half, 2 * half)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """The nearest E4M3 number (a tie: the even one) of x, at most 448 in size."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.pow(torch.full_like(x, 2.0), e - 3)
    return torch.round(x / step) * step  # torch.round: halves to even


def _exact_store(y, slot, pool, scales, page):
    """Codes and scales of the whole pool, block by block of the rows' own."""
    code, scale = pool.double(), scales.double()
    order = sorted(range(len(slot)), key=slot.__getitem__)
    at = 0
    while at < len(order):
        block, rows = slot[order[at]] // BLOCK, []
        while at < len(order) and slot[order[at]] // BLOCK == block:
            rows.append(order[at])
            at += 1
        pg, lo = block * BLOCK // page, block * BLOCK % page
        fresh = y[rows]  # [rows, H, D]
        top = fresh.abs().amax((0, 2))
        need = torch.pow(torch.full_like(top, 2.0), torch.floor(torch.log2((top / 448).clamp(min=2.0 ** -64))))
        need = torch.where(need * 448 < top, 2 * need, need)
        need = torch.where(need * 224 >= top.clamp(min=448 * 2.0 ** -64), need / 2, need)
        old = scale[pg, :, lo // BLOCK].clone()
        if slot[rows[0]] % BLOCK == 0:
            old.zero_()
        new = torch.maximum(old, need)
        scale[pg, :, lo // BLOCK] = new
        ratio = torch.where((new > old) & (old > 0), old / new, 1.0)
        code[pg, :, lo:lo + BLOCK] = _exact_e4m3(code[pg, :, lo:lo + BLOCK] * ratio[:, None, None])
        inside = [slot[r] % page for r in rows]
        code[pg, :, inside] = _exact_e4m3(fresh / new[:, None]).transpose(0, 1)
    return code, scale


def _exact_append(s, c):
    slot = s["slot"].tolist()
    table = s["cos_sin"][s["pos"].long()] if c["rot"] else None
    k, ks = _exact_store(_exact_turn(s["k"], s["k_gamma"], table, c["inter"]), slot, s["k_pool"], s["k_scales"], c["page"])
    v, vs = _exact_store(s["v"].double(), slot, s["v_pool"], s["v_scales"], c["page"])
    return {"q": _exact_turn(s["q"], s["q_gamma"], table, c["inter"]), "k": k, "v": v, "k_scales": ks, "v_scales": vs}


def _exact_rows(pool, scales, pages, head, keys):
    """Rows 0..keys-1 of one sequence's KV head, in 64 bits."""
    code = pool.view(torch.uint8)[pages, head].view(F8).double().flatten(0, 1)[:keys]
    scale = scales[pages, head].double().flatten()
    return code * scale[torch.arange(keys, device=code.device) // BLOCK, None]


def _exact_attend(s, c):
    hkv = c["hkv"]
    group = c["hq"] // hkv
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    pools = (s["k_pool"].cuda(), s["k_scales"]), (s["v_pool"].cuda(), s["v_scales"])
    start = s["start"].tolist() if s["start"] is not None else list(range(c["batch"] + 1))
    for b, keys in enumerate(s["kv_len"].tolist()):
        n = start[b + 1] - start[b]
        if n and not keys:
            lse[start[b]:start[b + 1]] = -math.inf
        if not n or not keys:
            continue
        pages = s["table"][b, :-(-keys // c["page"])].long()
        for h in range(hkv):
            k, v = (_exact_rows(p, sc, pages, h, keys) for p, sc in pools)
            for i in range(0, n, 512):
                j = slice(start[b] + i, start[b] + min(n, i + 512))
                q = s["q"][j, h * group:(h + 1) * group].double()
                score = torch.einsum("tgd,sd->tgs", q, k) / c["d"] ** 0.5
                at = keys - n + i + torch.arange(q.shape[0], device="cuda")
                score[(torch.arange(keys, device="cuda") > at[:, None])[:, None].expand_as(score)] = -math.inf
                lse[j, h * group:(h + 1) * group] = torch.logsumexp(score, -1)
                out[j, h * group:(h + 1) * group] = torch.einsum("tgs,sd->tgd", torch.softmax(score, -1), v)
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] not in ("append", "attend"):
        return None  # whole numbers, and bytes as they are
    s = prepare(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_attend)(s, case)
