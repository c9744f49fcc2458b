"""The paged 4-bit cache in plain 64-bit torch on the CPU: the definitions the
GPU tests compare against.  Shares no code with the library."""
import math

import numpy as np
import torch


def round5(x):
    """Five significant bits, ties to even; 0 below 2^-120."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)
    return np.where(x < 2.0 ** -120, 0.0, np.ldexp(np.rint(m * 32), e - 5))


def quantise(x):
    """[..., D] float64 -> codes (int) [..., D], scales [..., D/32]; NaN -> 0, inf -> +-7 steps."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    fin = np.isfinite(g)
    a = np.where(fin, np.abs(g), 0.0)
    top = a.max(-1, keepdims=True)
    s = round5(top / 7)
    g = np.where(np.isnan(g), 0.0, np.where(np.isinf(g), np.sign(g) * top, g))
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s > 0, np.rint(g / np.where(s > 0, s, 1.0)), 0.0)
    return (c + 8).astype(np.int64).reshape(x.shape), s[..., 0]


def held(x):
    """What the cache stands for after x was written."""
    c, s = quantise(x)
    return (c - 8) * np.repeat(s, 32, -1)


class Pool:
    """A CPU copy of one layer's pool [pages, heads, block], read and written row by row."""

    def __init__(self, raw, D):
        self.raw = raw.detach().cpu().numpy().copy()
        self.D = D
        self.P = self.raw.shape[-1] * 8 // (9 * D)
        r, s = D // 2, D // 16
        self.off = {"k": (0, self.P * r), "v": (self.P * (r + s), self.P * (r + s) + self.P * r)}

    def bytes_of(self, page, head, slot, which):
        D = self.D
        a, b = self.off[which]
        blk = self.raw[page, head]
        return blk[a + slot * D // 2:][:D // 2], blk[b + slot * D // 16:][:D // 16]

    def row(self, page, head, slot, which):
        codes, scales = self.bytes_of(page, head, slot, which)
        c = np.empty(self.D, dtype=np.float64)
        c[0::2] = codes & 15
        c[1::2] = codes >> 4
        s = (scales.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        return (c - 8) * np.repeat(s, 32)

    def put(self, page, head, slot, which, x):
        codes, scales = self.bytes_of(page, head, slot, which)
        c, s = quantise(x)
        codes[:] = (c[0::2] | (c[1::2] << 4)).astype(np.uint8)
        scales[:] = (s.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16).view(np.uint8)

    def rows(self, table, count, head, which):
        """Values of positions 0 .. count-1, [count, D]; absent pages as NaN."""
        out = np.full((count, self.D), np.nan)
        for t in range(count):
            page = int(table[t // self.P]) if t // self.P < len(table) else -1
            if 0 <= page < self.raw.shape[0]:
                out[t] = self.row(page, head, t % self.P, which)
        return out


def seen_by(ctx, rows, n, mask, depth, window, sinks):
    """[n, ctx + rows] bool and nothing else: which keys each row sees."""
    vis = np.zeros((n, ctx + rows), dtype=bool)
    for i in range(rows):
        p = ctx + (int(depth[i]) if depth is not None else i)
        for t in range(ctx + rows):
            key, j = t, t - ctx
            if j >= 0:
                if mask is None:
                    ok = j <= i
                else:
                    ok = bool((int(mask[i, j // 64]) >> (j % 64)) & 1)
                key = ctx + (int(depth[j]) if depth is not None else j)
            else:
                ok = True
            if ok and window > 0:
                ok = p - key < window or key < sinks
            vis[i, t] = ok
    return vis


def attend(q, pool, table, ctx, rows, mask=None, depth=None, window=0, sinks=0, scale=None):
    """float64 attention of q [B, n, hq, D].  Returns out, lse, the weighted
    mean of |v| (what the rounding errors of out scale with) and the largest
    scale * sum |q k| of a row."""
    q = q.detach().double().cpu().numpy()
    B, n, hq, D = q.shape
    H = pool.raw.shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, absv = np.zeros((B, n, hq, D)), np.zeros((B, n, hq, D))
    lse, size = np.full((B, n, hq), -np.inf), np.zeros((B, n, hq))
    for b in range(B):
        c = max(0, min(int(ctx[b]), table.shape[1] * pool.P))
        r = n if rows is None else max(0, min(int(rows[b]), n))
        vis = seen_by(c, r, n, None if mask is None else mask[b], None if depth is None else depth[b], window, sinks)
        for h in range(H):
            k, v = pool.rows(table[b], c + r, h, "k"), pool.rows(table[b], c + r, h, "v")
            there = ~np.isnan(k).all(-1) if c + r else np.zeros(0, dtype=bool)
            for i in range(n):
                sel = np.nonzero(vis[i] & there)[0]
                if not len(sel):
                    continue
                for g in range(hq // H):
                    x = (k[sel] @ q[b, i, h * (hq // H) + g]) * scale
                    m = x.max()
                    e = np.exp(x - m)
                    at = (b, i, h * (hq // H) + g)
                    out[at] = (e @ v[sel]) / e.sum()
                    absv[at] = (e @ np.abs(v[sel])) / e.sum()
                    lse[at] = m + np.log(e.sum())
                    size[at] = scale * (np.abs(k[sel]) @ np.abs(q[at])).max()
    return out, lse, absv, size


def values(pool, which):
    """All of a pool at once: [pages, heads, P, D] float64."""
    D, P = pool.D, pool.P
    a, b = pool.off[which]
    codes = pool.raw[..., a:a + P * D // 2].reshape(pool.raw.shape[:2] + (P, D // 2))
    c = np.empty(pool.raw.shape[:2] + (P, D), dtype=np.float64)
    c[..., 0::2] = codes & 15
    c[..., 1::2] = codes >> 4
    s = np.ascontiguousarray(pool.raw[..., b:b + P * D // 16]).view(np.uint16).astype(np.uint32) << 16
    with np.errstate(invalid="ignore"):           # unwritten scales may be any NaN
        s = s.view(np.float32).astype(np.float64).reshape(pool.raw.shape[:2] + (P, D // 32))
        return (c - 8) * np.repeat(s, 32, -1)


def seen_rows(ctx, rows, n, mask, depth, window, sinks):
    """`seen_by` without its loops."""
    t = np.arange(ctx + rows)
    i = np.arange(n)
    d = i if depth is None else np.asarray(depth, dtype=np.int64)
    j = np.clip(t - ctx, 0, max(n - 1, 0))
    key = np.where(t < ctx, t, ctx + d[j])
    if mask is None:
        own = j[None] <= i[:, None]
    else:
        own = (np.asarray(mask).view(np.uint64)[:, j // 64] >> (j % 64).astype(np.uint64)) & np.uint64(1) != 0
    vis = np.where(t < ctx, True, own) & (i < rows)[:, None]
    if window > 0:
        vis &= (ctx + d[:, None] - key[None] < window) | (key < sinks)[None]
    return vis


def attend_many(q, pool, table, ctx, rows, mask=None, depth=None, window=0, sinks=0, scale=None):
    """`attend` for many rows and long contexts: a kv head's rows at once."""
    q = q.detach().double().cpu().numpy()
    B, n, hq, D = q.shape
    H = pool.raw.shape[1]
    G = hq // H
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, absv = np.zeros((B, n, hq, D)), np.zeros((B, n, hq, D))
    lse, size = np.full((B, n, hq), -np.inf), np.zeros((B, n, hq))
    kk, vv = values(pool, "k"), values(pool, "v")
    for b in range(B):
        c = max(0, min(int(ctx[b]), table.shape[1] * pool.P))
        r = n if rows is None else max(0, min(int(rows[b]), n))
        t = np.arange(c + r)
        page = np.where(t // pool.P < table.shape[1], table[b][np.minimum(t // pool.P, table.shape[1] - 1)], -1)
        there = (page >= 0) & (page < pool.raw.shape[0])
        vis = seen_rows(c, r, n, None if mask is None else mask[b], None if depth is None else depth[b], window, sinks)
        vis &= there[None]
        some, used = vis.any(1), vis.any(0)
        if not some.any():
            continue
        page, slot, see = page[used], t[used] % pool.P, vis[some][:, None][..., used]
        for h in range(H):
            k, v = kk[page, h, slot], vv[page, h, slot]
            y = q[b, some, h * G:(h + 1) * G]
            x = np.where(see, (y @ k.T) * scale, -np.inf)
            m = x.max(-1, keepdims=True)
            e = np.exp(x - m)
            total = e.sum(-1, keepdims=True)
            at = np.ix_([b], np.nonzero(some)[0], range(h * G, (h + 1) * G))
            out[at] = (e @ v / total)[None]
            absv[at] = (e @ np.abs(v) / total)[None]
            lse[at] = (m + np.log(total))[..., 0][None]
            size[at] = np.where(see, np.abs(y) @ np.abs(k).T, 0.0).max(-1)[None] * scale
    return out, lse, absv, size


def check_attend(got, lse, ref):
    """out: its own rounding to bf16 (2^-9 of |o|), and the weights' rounding
    to bf16 before they meet V (2^-9 of the weighted |v|), with as much again
    for fp32 sums; lse: fp32 scores (products exact, D-term sums in fp32,
    2^-17 of the terms' size with all roundings in one direction) and one
    approximate exponential and logarithm."""
    out, want, absv, size = ref
    got = got.double().cpu().numpy()
    bound = 2.0 ** -9 * np.abs(out) + 2.0 ** -8 * absv + 1e-30
    worst = (np.abs(got - out) / bound).max()
    assert worst <= 1.0, worst
    if lse is not None:
        lse = lse.double().cpu().numpy()
        none = np.isinf(want)
        assert (np.isneginf(lse) == none).all()
        err = np.abs(np.where(none, 0.0, lse) - np.where(none, 0.0, want))
        assert (err <= 2.0 ** -17 * (1 + size + np.where(none, 0.0, np.abs(want)))).all(), err.max()
