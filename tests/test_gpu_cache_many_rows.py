"""GPU parity of cache_attend with its 64-bit reference where a kv head has more
rows than the register kernel takes (48): the cases in which the tcgen05 kernel
has code of its own.  Row counts are on both sides of the borders: 48 (kernel),
128 (one or two softmax groups), 256 (units)."""
import math

import numpy as np
import pytest
import torch

import cache_ref
import speculative_decoding_draft_sampling_gb300 as sv
from test_gpu_cache import DEV, NAN, filled, garbage_pool, ints, randn, table_for, trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", [(13, 4), (25, 2), (33, 4), (50, 1), (70, 2)])
def test_same_bits_whatever_ran_before(D, n, G):
    """Row counts that fill no warp: what an earlier call left in shared memory must not show."""
    P, H, ctx = 64, 2, [3000, 900]
    pool, table, _, _ = filled([c + n for c in ctx], H, P, D)
    q = randn(2, n, G * H, D)
    zero, large = torch.zeros((2, 256, G * H, D), dtype=torch.bfloat16, device=DEV), randn(2, 256, G * H, D, scale=40.0)
    got = []
    for before in (zero, large):
        for _ in range(2):
            sv.cache_attend(before, pool, table, ints([c - 256 for c in ctx]))
        r = sv.cache_attend(q, pool, table, ints(ctx), want_lse=True)
        got.append((r.out.clone(), r.lse.clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    ref = cache_ref.attend_many(q, cache_ref.Pool(pool, D), table.cpu().numpy(), ctx, None)
    cache_ref.check_attend(*got[0], ref)


# rows a request, q heads, kv heads: 48, 49, 128, 129, 256 and 300 rows a kv head
SHAPES = [(12, 4, 1), (7, 14, 2), (64, 2, 1), (43, 3, 1), (64, 8, 2), (75, 4, 1)]
FEW = [SHAPES[1], SHAPES[3]]                     # one softmax group, two
shapes = pytest.mark.parametrize("n,hq,H", SHAPES)
few = pytest.mark.parametrize("n,hq,H", FEW)
both = pytest.mark.parametrize("D,P", [(128, 64), (64, 16)])


def attend(q, pool, table, ctx, rows=None, mask=None, depth=None, check=True, **kw):
    """The call, checked against the reference."""
    r = sv.cache_attend(q, pool, table, ints(ctx), None if rows is None else ints(rows),
                        anc_mask=None if mask is None else torch.from_numpy(mask).to(DEV),
                        depth=None if depth is None else torch.from_numpy(depth).to(DEV), want_lse=True, **kw)
    if check:
        kw = {k: v for k, v in kw.items() if k in ("window", "sinks", "scale")}
        cache_ref.check_attend(r.out, r.lse, reference(q, pool, table, ctx, rows, mask, depth, **kw))
    return r


def reference(q, pool, table, ctx, rows=None, mask=None, depth=None, **kw):
    return cache_ref.attend_many(q, cache_ref.Pool(pool, q.shape[-1]), table.cpu().numpy(), ctx, rows, mask, depth, **kw)


def case(ctx, n, hq, H, D, P, rows=None, seed=0, spare_width=0):
    """A filled pool, its table and queries."""
    total = [c + r for c, r in zip(ctx, rows or [n] * len(ctx))]
    width = max(1, max(-(-t // P) for t in total)) + spare_width
    pool, table, _, _ = filled(total, H, P, D, seed=seed, width=width)
    return randn(len(ctx), n, hq, D, seed=seed + 7, scale=2.0), pool, table


@both
@shapes
def test_long_contexts(D, P, n, hq, H):
    """Split over many CTAs, of very different lengths."""
    ctx = [4100, 0, 40, 1500]
    attend(*case(ctx, n, hq, H, D, P, seed=n), ctx)


@both
@shapes
def test_trees_on_long_contexts(D, P, n, hq, H):
    ctx, rows = [2000, 127, 700], [n, n // 2, 1]
    mask, depth = trees(3, n, seed=n)
    attend(*case(ctx, n, hq, H, D, P, rows=rows, seed=n), ctx, rows, mask, depth)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,n,G", [(12, 4, 25, 2), (12, 4, 40, 4), (1, 1, 64, 4)])
def test_scores_that_rise_and_fall(D, B, H, n, G):
    """Each key beats all before it for half of the rows (the maximum moves at every tile, and what was summed is
    rescaled in tensor memory), for the others the first key stays on top; many tiles a share, and few."""
    P, T = 64, 4000
    total = [T + n] * B
    table, pages = table_for(total, P, -(-(T + n) // P))
    pool = garbage_pool(pages, H, P, D)
    ramp = torch.linspace(0, 1, T + n, device=DEV)[None, :, None, None]
    k = (ramp * torch.ones((B, 1, H, D), device=DEV)).to(torch.bfloat16)
    sv.cache_append(k, randn(B, T + n, H, D, seed=8), pool, table, ints([0] * B))
    sign = torch.where(torch.arange(n * G * H, device=DEV).reshape(n, G * H) % 2 == 0, 1.0, -1.0)
    size = torch.linspace(4, 16, n, device=DEV)[:, None]
    q = (sign * size)[None, :, :, None].expand(B, n, G * H, D).to(torch.bfloat16)
    attend(q, pool, table, [T - 3 * b for b in range(B)])


@both
@shapes
def test_large_scores_pick_one_key(D, P, n, hq, H):
    """Scores of several thousands.  Where one key leads by more than 100 (e^-100 is 0 even beside a maximum that
    has yet to move by 2^8) the output is its value, exactly, and lse its score."""
    ctx, G = [150, 1700], hq // H
    q, pool, table = case(ctx, n, hq, H, D, P, seed=2)
    r = sv.cache_attend(q, pool, table, ints(ctx), want_lse=True, scale=40.0)
    out, lse = r.out.double().cpu().numpy(), r.lse.double().cpu().numpy()
    ref = cache_ref.Pool(pool, D)
    keys, vals = cache_ref.values(ref, "k"), cache_ref.values(ref, "v")
    led = 0
    for b, c in enumerate(ctx):
        t = np.arange(c + n)
        page, slot = table[b].cpu().numpy()[t // P], t % P
        see = cache_ref.seen_rows(c, n, n, None, None, 0, 0)
        for h in range(hq):
            k, v, y = keys[page, h // G, slot], vals[page, h // G, slot], q[b, :, h].double().cpu().numpy()
            x = np.where(see, 40.0 * (y @ k.T), -np.inf)
            order = np.sort(x, -1)
            lead = order[:, -1] - order[:, -2] > 100
            led += lead.sum()
            assert (out[b, lead, h] == v[x.argmax(-1)][lead]).all()
            size = 40.0 * (np.abs(y) @ np.abs(k).T).max(-1)
            assert (np.abs(lse[b, lead, h] - order[lead, -1]) <= 2.0 ** -17 * (1 + 2 * size[lead])).all()
    assert led > n * hq


@few
@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 4), (130, 130), (300, 5), (1000, 0), (5000, 4)])
@pytest.mark.parametrize("tree", [False, True])
def test_windows_on_long_contexts(window, sinks, tree, n, hq, H):
    ctx = [0, 3, 1000, 2600]
    mask, depth = trees(4, n, seed=window) if tree else (None, None)
    attend(*case(ctx, n, hq, H, 64, 32, seed=window), ctx, None, mask, depth, window=window, sinks=sinks)


def spoil(pool, table, P, D, positions):
    """NaN and infinite scales, K's and V's, at positions of request 0."""
    half, width = P * (D // 2 + D // 16), P * D // 16
    for t in positions:
        if t // P >= table.shape[1] or int(table[0, t // P]) < 0:
            continue
        for off in (P * D // 2, half + P * D // 2):
            blk = pool[int(table[0, t // P]), :, off:off + width].view(torch.bfloat16).unflatten(-1, (P, D // 32))
            blk[:, t % P] = NAN if t % 2 else math.inf


@both
@pytest.mark.parametrize("n,hq,H", [(3, 4, 2)] + FEW)
@pytest.mark.parametrize("least", [None, 0, 5])
def test_what_no_row_sees_may_be_anything(D, P, n, hq, H, least):
    """Past the end, and between the sinks and the first position that some row's window reaches: for a tree that
    of its shallowest row (`least`; None: a chain)."""
    ctx, window, sinks = [700], 200, 4
    q, pool, table = case(ctx, n, hq, H, D, P, spare_width=1)
    mask = depth = None
    if least is not None:
        mask, depth = trees(1, n, seed=3)
        depth = depth + np.int32(least)
        depth = np.minimum(depth, n).astype(np.int32)
    first = ctx[0] + (0 if depth is None else int(depth.min())) - window + 1
    args = dict(mask=mask, depth=depth, window=window, sinks=sinks)
    clean = attend(q, pool, table, ctx, **args)
    clean = (clean.out.clone(), clean.lse.clone())
    spoil(pool, table, P, D, list(range(sinks, first)) + list(range(ctx[0] + n, table.shape[1] * P)))
    got = attend(q, pool, table, ctx, check=False, **args)
    assert torch.equal(got.out, clean[0]) and torch.equal(got.lse, clean[1])


@few
def test_bad_queries_stay_alone(n, hq, H):
    ctx = [900]
    q, pool, table = case(ctx, n, hq, H, 128, 64)
    good = attend(q, pool, table, ctx)
    good = (good.out.clone(), good.lse.clone())
    keep = torch.ones((1, n, hq), dtype=torch.bool, device=DEV)
    q[0, 1, 1, 5], q[0, n - 1, 0, 0] = NAN, NAN
    keep[0, 1, 1] = keep[0, n - 1, 0] = False
    r = attend(q, pool, table, ctx, check=False)
    assert torch.equal(r.out[keep], good[0][keep]) and torch.equal(r.lse[keep], good[1][keep])
    assert torch.isnan(r.out[~keep]).all()
    # an infinite one may move the maximum of its neighbours (other roundings), no more
    q[0, 1, 1, 5] = math.inf
    r = attend(q, pool, table, ctx, check=False)
    assert torch.isnan(r.out[0, 1, 1]).all()
    out, lse = torch.where(keep[..., None], r.out, 0), torch.where(keep, r.lse, 0)
    q[~keep] = 0
    ref = reference(q, pool, table, ctx)
    off = ~keep.cpu().numpy()
    for x in ref:
        x[off] = 0
    cache_ref.check_attend(out, lse, ref)


@both
@shapes
def test_missing_pages(D, P, n, hq, H):
    """Inside the context, in the first tile and among the drafted rows: left out and reported."""
    ctx = [700, 300]
    q, pool, table = case(ctx, n, hq, H, D, P)
    for bad in (-1, 1 << 30, pool.shape[0]):
        table[0, 5], table[0, 0], table[0, (ctx[0] + n - 1) // P] = bad, -1, bad
        status = ints([0, 0])
        attend(q, pool, table, ctx, status=status)
        assert status.tolist() == [sv.ST_BAD_PAGE, 0]
    table[1] = -1                                # nothing left at all
    r = attend(q, pool, table, ctx)
    assert torch.isneginf(r.lse[1]).all() and not r.out[1].any()


@few
def test_missing_pages_outside_the_window(n, hq, H):
    """A released page that no row's window reaches is not asked for."""
    ctx, P = [1500], 32
    q, pool, table = case(ctx, n, hq, H, 128, P)
    status = ints([0])
    want = attend(q, pool, table, ctx, window=200, sinks=4, status=status)
    want = want.out.clone()
    table[0, 1:(ctx[0] - 200 + 1) // P] = -1
    got = attend(q, pool, table, ctx, window=200, sinks=4, status=status)
    assert status.tolist() == [0] and torch.equal(got.out, want)


@shapes
def test_lengths_outside_the_table(n, hq, H):
    D, P, width = 64, 16, 16
    pool, table, _, _ = filled([width * P] * 3, H, P, D)
    q = randn(3, n, hq, D)
    status = ints([0, 0, 0])
    ctx, rows = [1 << 30, -7, width * P - n], [2, 1, n + 7]
    r = sv.cache_attend(q, pool, table, ints(ctx), ints(rows), want_lse=True, status=status)
    cache_ref.check_attend(r.out, r.lse, reference(q, pool, table, [width * P, 0, width * P - n], [2, 1, n]))
    assert status.tolist() == [sv.ST_BAD_PAGE, 0, 0]


@shapes
def test_rows_without_keys(n, hq, H):
    """Requests without rows, rows past num_rows, rows whose mask is empty, and rows that see one key: its value."""
    ctx, rows = [0, 500, 0, 300], [0, 0, n - 2, 3]
    q, pool, table = case(ctx, n, hq, H, 128, 16, rows=rows, spare_width=1)
    r = attend(q, pool, table, ctx, rows)
    for b, c in enumerate(rows):
        assert not r.out[b, c:].any() and torch.isneginf(r.lse[b, c:]).all()
    mask = np.zeros((4, n, (n + 63) // 64), dtype=np.int64)
    mask[:, 1::3, 0] = 4                         # every third row sees drafted row 2 alone, the others nothing
    r = attend(q, pool, table, ctx, rows, mask)
    value = sv.cache_read(pool, table, ints(ctx), 3, 128)[1][2, 2].repeat_interleave(hq // H, 0)
    assert torch.equal(r.out[2, 1:n - 2:3], value.expand_as(r.out[2, 1:n - 2:3]))
    assert not r.out[2, 0::3].any() and torch.isneginf(r.lse[2, 0::3]).all()


@pytest.mark.parametrize("D", [64, 128])
@few
def test_strided_queries_and_pools(D, n, hq, H):
    P, ctx = 32, [390, 40]
    _, pool, table = case(ctx, n, hq, H, D, P)
    wide = randn(2, n, hq * D + 24, seed=6)
    for off in (0, 8, 3):                        # 16-byte rows, and rows off by a few values
        q = wide[..., off:off + hq * D].unflatten(-1, (hq, D))
        want = attend(q.contiguous(), pool, table, ctx)
        got = attend(q, pool, table, ctx, check=False)
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
    layers = garbage_pool(3, H + 3, P, D, lead=(pool.shape[0],))               # [pages, layers, heads, block]
    layers[:, 1, 1:1 + H] = pool
    got = attend(q, layers[:, 1, 1:1 + H], table, ctx, check=False)
    assert torch.equal(got.out, want.out)


@few
def test_far_pages(n, hq, H):
    """Pages more than 2^32 bytes apart."""
    D, P, ctx = 128, 64, [150, 70]
    q, pool, table = case(ctx, n, hq, H, D, P)
    stride, block = (1 << 32) + (1 << 20), pool.shape[-1]
    big = torch.empty(stride * (pool.shape[0] - 1) + H * block, dtype=torch.uint8, device=DEV)
    far = big.as_strided(pool.shape, (stride, block, 1))
    far.copy_(pool)
    want, got = attend(q, pool, table, ctx), attend(q, far, table, ctx, check=False)
    assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)


@pytest.mark.parametrize("n,hq,H", SHAPES[1:])
def test_same_bits_every_time_and_on_other_streams(n, hq, H):
    ctx = [3000, 40, 900, 1500]
    q, pool, table = case(ctx, n, hq, H, 128, 64)
    want = attend(q, pool, table, ctx)
    want = (want.out.clone(), want.lse.clone())
    c, side = ints(ctx), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        here = sv.cache_attend(q, pool, table, c, want_lse=True)
        there = sv.cache_attend(q, pool, table, c, want_lse=True, stream=side)
        torch.cuda.synchronize()
        for r in (here, there):
            assert torch.equal(r.out, want[0]) and torch.equal(r.lse, want[1])


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 4)])
@pytest.mark.parametrize("n,D,P", [(1024, 64, 64), (511, 128, 16)])
def test_chunk_of_a_prompt(n, D, P, window, sinks):
    """Many rows of one request: several units of 256 rows over the same context."""
    ctx = [1500, 0]
    attend(*case(ctx, n, 4, 2, D, P, rows=[n, n - 300]), ctx, [n, n - 300], window=window, sinks=sinks)
