"""The paged 4-bit cache and the attention of drafted rows over it: what is measured.

Plain forms (``own`` false) are elementary torch operations in 32 bits; with
``own`` true the same passes go through the package's entry points.

The cache.  ``pool`` is uint8 [layers, pages, kv heads, block] (one layer:
[pages, kv heads, block]).  A block holds one page of P tokens of one kv head:

    K codes [P][D/2] | K scales bf16 [P][D/32] | V codes [P][D/2] | V scales bf16 [P][D/32]

Element d of a row is the low (even d) or high (odd d) half of byte d/2 and
stands for (code - 8) * scale[d // 32].
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attend(name, **kw):
    c = dict(op="attend", B=1, n=1, T=512, hq=32, hkv=8, d=128, page=64, tree=False, window=0, sinks=0)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, one token, a short context: the latency of a call
        _attend("attend one token", B=1, n=1, T=517),
        # a chain of 3 drafted tokens and the root for a batch of requests of mixed lengths
        _attend("attend chain of 4", B=64, n=4, T=2048),
        # a block draft of 8 and the root, a large batch
        _attend("attend chain of 9", B=256, n=9, T=4096),
        # the verification of 64-node draft trees under ancestor masks
        _attend("attend tree of 64", B=32, n=64, T=8192, tree=True),
        # a model with a sliding window and 4 sinks, narrow heads, small pages, long contexts
        _attend("attend window and sinks", B=64, n=4, T=16384, hq=64, hkv=8, d=64, page=32, window=2048, sinks=4),
        # few users with very long contexts, single tokens
        _attend("attend long", B=4, n=1, T=131072),
        # one decoding step's rows written into the cache and read back
        dict(name="append one step", op="append", B=64, n=4, T=2048, hkv=8, d=128, page=64),
        # prompts written into the cache
        dict(name="append prompts", op="append", B=8, n=8192, T=100, hkv=8, d=128, page=64),
        # the accepted paths of a few small trees, a shallow model
        dict(name="compact few", op="compact", B=4, n=5, T=100, layers=4, hkv=8, d=128, page=64),
        # the accepted paths of a large batch of 64-node trees, 32 layers
        dict(name="compact batch", op="compact", B=128, n=64, T=70, layers=32, hkv=8, d=128, page=64),
        # four requests forked once, with room for a step, and the children freed
        dict(name="pages few", op="pages", B=4, kids=1, n=5, T=300, layers=4, hkv=8, d=128, page=64),
        # parallel sampling: 64 prompts forked twice, 32 layers
        dict(name="pages batch", op="pages", B=64, kids=2, n=9, T=500, layers=32, hkv=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend"] * 5 + ["append", "append", "compact", "pages"])
    hkv, d, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64])
    if op == "attend":
        tree = rng.random() < 0.3
        n = _log(rng, 2, 128) if tree else _log(rng, 1, 16)
        hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
        B = _log(rng, 1, 256)
        T = _log(rng, 1, 131072)
        T = max(1, min(T, 500_000_000 // (B * hkv * d), 60_000_000_000 // (B * hq * n * d)))
        window = _log(rng, 16, 4096) if rng.random() < 0.4 else 0
        sinks = rng.choice([0, 1, 4, 5, 70]) if window else 0
        return _attend(None, B=B, n=n, T=T, hq=hq, hkv=hkv, d=d, page=page, tree=tree, window=window, sinks=sinks)
    if op == "append":
        B = _log(rng, 1, 256)
        n = max(1, min(_log(rng, 1, 8192), 60_000_000 // (B * hkv * d)))
        return dict(op=op, B=B, n=n, T=_log(rng, 1, 2000), hkv=hkv, d=d, page=page)
    layers = rng.choice([1, 2, 8, 24, 32])
    if op == "compact":
        return dict(op=op, B=_log(rng, 1, 128), n=_log(rng, 2, 64), T=_log(rng, 1, 130), layers=layers, hkv=hkv, d=d, page=page)
    return dict(op=op, B=_log(rng, 1, 64), kids=rng.choice([1, 2]), n=_log(rng, 1, 64), T=_log(rng, 1, 500), layers=layers, hkv=hkv, d=d, page=page)


# ---------------------------------------------------------------------------
# the cache in plain operations
# ---------------------------------------------------------------------------
def _sections(pool, d):
    """Views of a pool's four arrays: K codes, K scales, V codes, V scales, each [..., P, width]."""
    p = pool.shape[-1] * 8 // (d * 9)
    a, b = p * d // 2, p * d // 16
    cut = [pool[..., :a], pool[..., a:a + b].view(torch.bfloat16),
           pool[..., a + b:2 * a + b], pool[..., 2 * a + b:].view(torch.bfloat16)]
    return [x.unflatten(-1, (p, -1)) for x in cut]


def _codes_of(x, dtype=torch.float32):
    """[..., D] -> packed codes uint8 [..., D/2] and bf16 scales [..., D/32]."""
    g = x.to(dtype).unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(-1) / 7).to(torch.float32)
    u = s.view(torch.int32)
    s = ((u + 0x3FFFF + ((u >> 19) & 1)) & -0x80000).view(torch.float32)      # five significant bits, ties to even
    s = torch.where(s < 2.0 ** -120, 0.0, s)
    c = torch.where(s[..., None] > 0, torch.round(g / s[..., None].to(dtype)), 0.0).clamp(-7, 7).flatten(-2)
    c = (c + 8).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.to(torch.bfloat16)


def _values_of(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    return (c.unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def _rows_of(table, pos, page):
    """Page and slot of positions [B, n] under a table [B, M]."""
    return table.gather(1, (pos // page).clamp(0, table.shape[1] - 1)).long(), pos % page


def _append_plain(s):
    n, page = s["k"].shape[1], s["page"]
    pos = s["start"].long()[:, None] + torch.arange(n, device=DEV)
    b, i = torch.nonzero(torch.arange(n, device=DEV) < s["count"][:, None], as_tuple=True)
    pages, slots = _rows_of(s["table"], pos, page)
    pages, slots = pages[b, i], slots[b, i]
    kc, ks, vc, vs = _sections(s["pool"], s["d"])
    kc[pages, :, slots], ks[pages, :, slots] = _codes_of(s["k"][b, i])
    vc[pages, :, slots], vs[pages, :, slots] = _codes_of(s["v"][b, i])


def _read_plain(s):
    n, page = s["k"].shape[1], s["page"]
    pos = s["start"].long()[:, None] + torch.arange(n, device=DEV)
    live = (torch.arange(n, device=DEV) < s["count"][:, None])[..., None, None]
    pages, slots = _rows_of(s["table"], pos, page)
    kc, ks, vc, vs = [x[pages, :, slots] for x in _sections(s["pool"], s["d"])]
    return [torch.where(live, _values_of(c, f), 0.0).to(torch.bfloat16) for c, f in ((kc, ks), (vc, vs))]


def _visible(ctx, rows, depth, seen, n, T, window, sinks):
    """Which of the T cache positions each of the n rows sees: [B, n, T]."""
    t = torch.arange(T, device=DEV)
    j = t - ctx.long()[:, None]                                              # drafted row held at t
    drafted = (j >= 0) & (j < rows[:, None])
    jj = j.clamp(0, n - 1)
    vis = torch.where(drafted[:, None], seen.gather(2, jj[:, None].expand(-1, n, -1)), (j < 0)[:, None])
    vis &= torch.arange(n, device=DEV)[:, None] < rows[:, None, None]
    key = torch.where(drafted, ctx.long()[:, None] + depth.long().gather(1, jj), t)
    row = ctx.long()[:, None] + depth.long()
    if window:
        vis &= (row[:, :, None] - key[:, None] < window) | (key[:, None] < sinks)
    return vis


def _seen(s):
    """The drafted rows that each drafted row sees, [B, n, n], and the rows' depths."""
    B, n = s["q"].shape[:2]
    i = torch.arange(n, device=DEV)
    if s["mask"] is None:
        return (i[:, None] >= i).expand(B, n, n), i.expand(B, n)
    return (s["mask"][:, :, i // 64] >> (i % 64)) & 1 > 0, s["depth"]


def _attend_plain(s):
    B, n, hq, d = s["q"].shape
    kc, ks, vc, vs = _sections(s["pool"], d)
    hkv, page = kc.shape[1], kc.shape[2]
    T = s["table"].shape[1] * page
    at = s["table"].clamp(min=0).long()
    k = _values_of(kc[at], ks[at]).permute(0, 2, 1, 3, 4).reshape(B, hkv, T, d)
    v = _values_of(vc[at], vs[at]).permute(0, 2, 1, 3, 4).reshape(B, hkv, T, d)
    held = torch.arange(T, device=DEV) < (s["ctx"] + s["rows"]).long()[:, None]
    v = torch.where(held[:, None, :, None], v, 0.0)                          # what lies past the end may be anything
    seen, depth = _seen(s)
    vis = _visible(s["ctx"], s["rows"], depth, seen, n, T, s["window"], s["sinks"])
    q = s["q"].float().unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)        # [B, hkv, n, G, d]
    x = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (n, -1)) * (1 / math.sqrt(d))
    x = torch.where(vis[:, None, :, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    empty = m == -math.inf
    p = torch.exp(x - torch.where(empty, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (n, -1)) / torch.where(empty, 1.0, total)
    lse = torch.where(empty, -math.inf, m + torch.log(total))[..., 0]
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, hq, d).to(torch.bfloat16), lse.permute(0, 2, 1, 3).reshape(B, n, hq)


def _compact_plain(s):
    page = s["page"]
    j = torch.arange(s["path"].shape[1], device=DEV)
    b, i = torch.nonzero((j <= s["acc"][:, None]) & (s["path"] != j), as_tuple=True)
    ctx = s["ctx"].long()[:, None]
    fp, fs = [x[b, i] for x in _rows_of(s["table"], ctx + s["path"].clamp(min=0), page)]
    tp, ts = [x[b, i] for x in _rows_of(s["table"], ctx + j, page)]
    kc, ks, vc, vs = _sections(s["pool"], s["d"])
    kc[:, tp, :, ts] = kc[:, fp, :, fs]
    ks[:, tp, :, ts] = ks[:, fp, :, fs]
    vc[:, tp, :, ts] = vc[:, fp, :, fs]
    vs[:, tp, :, ts] = vs[:, fp, :, fs]


def _reserve_plain(s, length):
    table, held, ref, free, left = s["table"], s["held"], s["ref"], s["free"], s["left"]
    need = (-(-length.clamp(min=0) // s["page"]) - held).clamp(min=0)
    off = need.cumsum(0) - need
    need = torch.where(off + need <= left, need, 0)
    j = torch.arange(table.shape[1], device=DEV) - held[:, None]
    take = (j >= 0) & (j < need[:, None])
    new = free[(left - 1 - off[:, None] - j)[take].long()]
    table[take] = new
    ref[new.long()] = 1
    held += need.to(held.dtype)
    left -= need.sum().to(left.dtype)


def _fork_plain(s):
    table, held, ref, free, left = s["table"], s["held"], s["ref"], s["free"], s["left"]
    src, dst, page = s["src"].long(), s["dst"].long(), s["page"]
    full, tail = s["length"][src] // page, s["length"][src] % page
    own_page = (tail > 0).to(torch.int32)
    off = own_page.cumsum(0) - own_page
    f = torch.nonzero(own_page, as_tuple=True)[0]
    new = free[(left - 1 - off[f]).long()]
    col = torch.arange(table.shape[1], device=DEV)
    old = table[src]
    share = col < full[:, None]
    table[dst] = torch.where(share, old, -1)
    ref.index_add_(0, old[share].long(), torch.ones_like(old[share]))
    table[dst[f], full[f].long()] = new
    ref[new.long()] = 1
    held[dst] = (full + own_page).to(held.dtype)
    left -= own_page.sum().to(left.dtype)
    slot = torch.arange(page, device=DEV)[None] < tail[f][:, None]           # the rows that the child has
    d = s["d"]
    slot = torch.cat([slot.repeat_interleave(w, 1) for w in (d // 2, d // 16, d // 2, d // 16)], 1)[None, :, None]
    a, b = old[f, full[f].long()].long(), new.long()
    s["pool"][:, b] = torch.where(slot, s["pool"][:, a], s["pool"][:, b])


def _release_plain(s, length):
    table, held, ref, free, left = s["table"], s["held"], s["ref"], s["free"], s["left"]
    keep = torch.minimum(-(-length.clamp(min=0) // s["page"]), held)
    col = torch.arange(table.shape[1], device=DEV)
    gone = (col >= keep[:, None]) & (col < held[:, None])
    ids = table[gone].long()
    ref.index_add_(0, ids, torch.full_like(table[gone], -1))
    touched = torch.zeros_like(ref).index_fill_(0, ids, 1)
    freed = torch.nonzero((touched > 0) & (ref == 0), as_tuple=True)[0].to(free.dtype)
    free[(left + torch.arange(freed.shape[0], device=DEV)).long()] = freed
    left += freed.shape[0]
    table[gone] = -1
    held.copy_(keep)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _spread(top, B, low=0.25):
    """B lengths from top down to a share of it: their sum does not depend on the seed."""
    return [max(1, int(top - (top * (1 - low)) * b // B)) for b in range(B)]


def _ints(v, gen):
    """The values in an order drawn from the seed."""
    v = torch.tensor(v, dtype=torch.int32, device=DEV)
    return v[torch.randperm(len(v), device=DEV, generator=gen)]


def _fill(pool, d, gen):
    """Codes of normal rows, with channels of different size, in every block."""
    kc, ks, vc, vs = _sections(pool.flatten(0, -3), d)
    step = max(1, 64_000_000 // (kc.shape[1] * kc.shape[2] * d))
    size = torch.exp(0.5 * torch.randn(kc.shape[1], 1, d, device=DEV, generator=gen))
    for a in range(0, kc.shape[0], step):
        for codes, scales, by in ((kc, ks, size), (vc, vs, 1.0)):
            x = torch.randn((min(step, kc.shape[0] - a),) + tuple(kc.shape[1:3]) + (d,), device=DEV, generator=gen) * by
            codes[a:a + step], scales[a:a + step] = _codes_of(x.to(torch.bfloat16))


def _pages(lengths, page, width, spare, gen):
    """A table [B, width] of the pages that hold these lengths, drawn without order, and the pages in all."""
    held = -(-lengths // page)
    count = int(held.sum())
    ids = torch.randperm(count + spare, device=DEV, generator=gen).to(torch.int32)
    has = torch.arange(width, device=DEV) < held[:, None]
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device=DEV)
    table[has] = ids[:count]
    return table, held.to(torch.int32), ids[count:].clone(), count + spare


def _trees(B, n, gen):
    """Random draft trees, parents first: ancestor masks as 64-bit words and depths of at most 16."""
    up = torch.randint(1, 9, (B, n), device=DEV, generator=gen)
    mask = torch.zeros((B, n, (n + 63) // 64), dtype=torch.int64, device=DEV)
    depth = torch.zeros((B, n), dtype=torch.int32, device=DEV)
    b = torch.arange(B, device=DEV)
    for i in range(n):
        if i:
            p = (i - up[:, i]).clamp(min=0)
            p = torch.where(depth[b, p] >= 16, 0, p)
            mask[:, i] = mask[b, p]
            depth[:, i] = depth[b, p] + 1
        bit = 1 << (i % 64)
        mask[:, i, i // 64] |= bit if bit < 1 << 63 else bit - (1 << 64)
    return mask, depth


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)
    c, B, d, page, hkv, n = case, case["B"], case["d"], case["page"], case["hkv"], case["n"]
    width = -(-(c["T"] + n + page) // page)
    block = page * d * 9 // 8
    s = {"op": c["op"], "d": d, "page": page}
    ctx = _ints(_spread(c["T"], B), gen)
    if c["op"] == "attend":
        rows = _ints([n - (b * n // 2) // B for b in range(B)] if c["tree"] else [n] * B, gen)
        table, held, _, count = _pages(ctx + rows, page, width, 3, gen)
        pool = torch.empty((count, hkv, block), dtype=torch.uint8, device=DEV)
        _fill(pool, d, gen)
        # the last page's slots past the end were never written: whatever they hold must not matter
        last = table.gather(1, (held - 1).long()[:, None])[:, 0].long()
        past = torch.arange(page, device=DEV) >= ((ctx + rows - 1) % page)[:, None] + 1
        for f in _sections(pool, d)[1::2]:
            f[last] = torch.where(past[:, None, :, None], math.nan, f[last])
        mask, depth = _trees(B, n, gen) if c["tree"] else (None, None)
        q = 2 * torch.randn((B, n, c["hq"], d), device=DEV, generator=gen)
        s.update(q=q.to(torch.bfloat16), pool=pool, table=table, ctx=ctx, rows=rows, mask=mask, depth=depth,
                 window=c["window"], sinks=c["sinks"], out=torch.empty_like(q, dtype=torch.bfloat16),
                 lse=torch.empty(q.shape[:3], device=DEV))
    elif c["op"] == "append":
        table, _, _, count = _pages(ctx + n, page, width, 3, gen)
        kv = [torch.randn((B, n, hkv, d), device=DEV, generator=gen).to(torch.bfloat16) for _ in range(2)]
        rows = _ints([max(1, n - (b * n // 2) // B) for b in range(B)], gen)
        pool = torch.zeros((count, hkv, block), dtype=torch.uint8, device=DEV)
        s.update(k=kv[0], v=kv[1], pool=pool, table=table, start=ctx, count=rows)
    elif c["op"] == "compact":
        table, _, _, count = _pages(ctx + n, page, width, 3, gen)
        pool = torch.empty((c["layers"], count, hkv, block), dtype=torch.uint8, device=DEV)
        _fill(pool, d, gen)
        deep = min(n, 17)
        step = torch.rand((B, deep - 1), device=DEV, generator=gen) if deep > 1 else torch.zeros((B, 0), device=DEV)
        room = (n - 1) // max(1, deep - 1)
        path = torch.cat([torch.zeros((B, 1), device=DEV), (1 + torch.floor(step * room)).cumsum(1)], 1).to(torch.int32)
        acc = _ints([_kept(b, deep) for b in range(B)], gen)
        path = torch.where(torch.arange(deep, device=DEV) <= acc[:, None], path, -1).to(torch.int32)
        s.update(pool=pool, table=table, ctx=ctx, path=path, acc=acc)
    else:
        kids = B * c["kids"]
        table, held, free, count = _pages(ctx, page, width, (B + kids) * (-(-n // page) + 1) + 5, gen)
        more = torch.zeros(kids, dtype=torch.int32, device=DEV)
        pool = torch.empty((c["layers"], count, hkv, block), dtype=torch.uint8, device=DEV)
        _fill(pool, d, gen)
        ref = torch.zeros(count, dtype=torch.int32, device=DEV)
        ref[table[table >= 0].long()] = 1
        stack = torch.full((count,), -1, dtype=torch.int32, device=DEV)
        stack[:len(free)] = free
        src = torch.arange(B, dtype=torch.int32, device=DEV).repeat(c["kids"])
        length = torch.cat([ctx, more])
        both = torch.cat([ctx, ctx[src.long()]])
        s.update(pool=pool, table=torch.cat([table, torch.full((kids, width), -1, dtype=torch.int32, device=DEV)]),
                 held=torch.cat([held, more]), ref=ref, free=stack,
                 left=torch.tensor([len(free)], dtype=torch.int32, device=DEV), src=src,
                 dst=torch.arange(B, B + kids, dtype=torch.int32, device=DEV), length=length, grown=both + n)
    return s


def _kept(b, deep):
    """Accepted rows after the root: most walks are short."""
    return min(deep - 1, (b * 7 % 11) * (b % 3 > 0))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "attend":
        o, lse = _attend_plain(s)
        return {"out": o, "lse": lse}
    if s["op"] == "append":
        _append_plain(s)
        k, v = _read_plain(s)
        return {"k": k, "v": v}
    if s["op"] == "compact":
        _compact_plain(s)
        return {"pool": s["pool"]}                   # bytes that were moved: no numbers are computed
    _fork_plain(s)
    _reserve_plain(s, s["grown"])
    grown = s["table"].clone()
    _release_plain(s, s["length"])
    return {"pool": s["pool"], "grown": grown, "table": s["table"], "held": s["held"], "ref": s["ref"],
            "free": s["free"], "left": s["left"]}


def _run_own(s):
    import speculative_decoding_draft_sampling_gb300 as sv
    if s["op"] == "attend":
        r = sv.cache_attend(s["q"], s["pool"], s["table"], s["ctx"], s["rows"], anc_mask=s["mask"], depth=s["depth"],
                            window=s["window"], sinks=s["sinks"], out=s["out"], lse=s["lse"])
        return {"out": r.out, "lse": r.lse}
    if s["op"] == "append":
        sv.cache_append(s["k"], s["v"], s["pool"], s["table"], s["start"], s["count"])
        k, v = sv.cache_read(s["pool"], s["table"], s["start"], s["k"].shape[1], s["d"], s["count"])
        return {"k": k, "v": v}
    if s["op"] == "compact":
        sv.cache_compact(s["pool"], s["table"], s["ctx"], s["path"], s["acc"], s["d"])
        return {"pool": s["pool"]}
    pages = sv.PageState(s["table"], s["held"], s["ref"], s["free"], s["left"])
    sv.cache_fork(s["pool"], pages, s["src"], s["dst"], s["length"], s["d"])
    sv.cache_reserve(pages, s["grown"], s["page"])
    grown = s["table"].clone()
    sv.cache_release(pages, s["length"], s["page"])
    return {"pool": s["pool"], "grown": grown, "table": s["table"], "held": s["held"], "ref": s["ref"],
            "free": s["free"], "left": s["left"]}


def work(case):
    """What a pass cannot do without: the visible part of the cache, the rows in and out."""
    c, B, d, hkv, n = case, case["B"], case["d"], case["hkv"], case["n"]
    row = hkv * d * 9 // 8                                                   # a token's K and V in the cache
    ctx = _spread(c["T"], B)
    if c["op"] == "attend":
        rows = [n - (b * n // 2) // B for b in range(B)] if c["tree"] else [n] * B
        r = sum(rows) / B
        keep = sum(min(t, c["window"] + c["sinks"]) if c["window"] else t for t in ctx) / B
        return {"bytes": B * (keep + r) * row + B * n * c["hq"] * (4 * d + 4),
                "flops": 4 * d * c["hq"] * sum(rows) * (keep + r / 2)}
    if c["op"] == "append":
        rows = sum(max(1, n - (b * n // 2) // B) for b in range(B))
        return {"bytes": rows * hkv * d * 4 + 2 * rows * row + B * n * hkv * d * 4, "flops": 2 * rows * hkv * d * 4}
    if c["op"] == "compact":
        deep = min(n, 17)
        moved = sum(_kept(b, deep) for b in range(B))
        return {"bytes": 2 * moved * row * c["layers"] + 4 * B * deep, "flops": 0}
    tails = sum(t % c["page"] for t in ctx) * c["kids"]
    width = -(-(c["T"] + n + c["page"]) // c["page"])
    return {"bytes": 2 * tails * row * c["layers"] + 12 * B * (1 + c["kids"]) * width, "flops": 0}


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------
def _exact_values(codes, scales):
    lo, hi = (codes.long() % 16).double() - 8, (codes.long() // 16).double() - 8
    return torch.stack([lo, hi], -1).flatten(-2) * scales.double().repeat_interleave(GROUP, -1)


def _exact_attend(s):
    B, n, hq, d = s["q"].shape
    kc, ks, vc, vs = _sections(s["pool"], d)
    hkv, page = kc.shape[1], kc.shape[2]
    o = torch.zeros((B, n, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((B, n, hq), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        ctx, rows = int(s["ctx"][b]), int(s["rows"][b])
        held = ctx + rows
        at = s["table"][b, :-(-held // page)].long()
        k, v = [_exact_values(x[at], y[at]).transpose(0, 1).flatten(1, 2)[:, :held] for x, y in ((kc, ks), (vc, vs))]
        see = torch.ones((rows, held), dtype=torch.bool, device=DEV)
        here = torch.arange(held, device=DEV)
        if s["mask"] is None:
            see[:, ctx:] = torch.ones((rows, rows), device=DEV).tril() > 0
            row = ctx + torch.arange(rows, device=DEV)
        else:
            for j in range(rows):
                see[:, ctx + j] = (s["mask"][b, :rows, j // 64] >> (j % 64)) % 2 != 0
            row = ctx + s["depth"][b, :rows].long()
            here = torch.cat([here[:ctx], row])
        if s["window"]:
            see &= (here[None] > row[:, None] - s["window"]) | (here < s["sinks"])[None]
        for h in range(hq):
            g = h // (hq // hkv)
            x = s["q"][b, :rows, h].double() @ k[g].T / math.sqrt(d)
            x[~see] = -math.inf
            lse[b, :rows, h] = torch.logsumexp(x, 1)
            some = see.any(1)
            o[b, :rows, h][some] = torch.softmax(x[some], 1) @ v[g]
    return {"out": o, "lse": lse}


def _exact_held(x):
    """What the cache stands for after x was written, by the definition."""
    g = x.double().unflatten(-1, (-1, GROUP))
    m, e = torch.frexp(g.abs().amax(-1, keepdim=True) / 7)
    s = torch.ldexp(torch.round(m * 32) / 32, e)
    return torch.where(s > 0, torch.round(g / s) * s, 0.0).flatten(-2)


def exact(case, seed):
    if case["op"] not in ("attend", "append"):
        return None                                                          # bytes and page numbers
    s = prepare(case, seed)
    if s["op"] == "attend":
        return _exact_attend(s)
    live = (torch.arange(s["k"].shape[1], device=DEV) < s["count"][:, None])[..., None, None]
    return {"k": torch.where(live, _exact_held(s["k"]), 0.0), "v": torch.where(live, _exact_held(s["v"]), 0.0)}
