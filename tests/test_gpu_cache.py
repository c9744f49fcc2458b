"""GPU parity of the paged 4-bit cache with its 64-bit reference: rows written
and read (exact), attention over the cache, accepted-path compaction and the
pages' calls (exact)."""
import math

import numpy as np
import pytest
import torch

import cache_ref
import speculative_decoding_draft_sampling_gb300 as sv

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(*shape, seed=0, scale=1.0):
    return (scale * torch.randn(shape, device=DEV, generator=gen(seed))).to(torch.bfloat16)


def garbage_pool(pages, H, P, D, seed=0, lead=()):
    """Every byte random: scales of any size, NaN and infinities among them."""
    shape = tuple(lead) + (pages, H, sv.cache_block_bytes(D, P))
    return torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=gen(seed + 99))


def table_for(lengths, P, width, seed=0, spare=2):
    """A table of pages in random order that holds these lengths, and the number of pages."""
    need = [-(-t // P) for t in lengths]
    ids = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).tolist()
    rows = []
    for c in need:
        rows.append(ids[:c] + [-1] * (width - c))
        ids = ids[c:]
    return ints(rows), sum(need) + spare


def filled(lengths, H, P, D, seed=0, width=None, scale=1.0):
    """A pool of garbage into which cache_append wrote `lengths` positions of each request."""
    width = width or max(1, max(-(-t // P) for t in lengths))
    table, pages = table_for(lengths, P, width, seed)
    pool = garbage_pool(pages, H, P, D, seed)
    n = max(1, max(lengths))
    k, v = randn(len(lengths), n, H, D, seed=seed + 1, scale=scale), randn(len(lengths), n, H, D, seed=seed + 2, scale=scale)
    status = torch.zeros(len(lengths), dtype=torch.int32, device=DEV)
    sv.cache_append(k, v, pool, table, ints([0] * len(lengths)), ints(lengths), status=status)
    assert status.tolist() == [0] * len(lengths)
    return pool, table, k, v


# ---------------------------------------------------------------------------
# rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,P,H,lengths", [(128, 64, 2, [1, 70, 0]), (64, 16, 3, [33, 16, 17]), (128, 32, 1, [5]),
                                           (64, 64, 5, [64, 65, 1, 2])])
def test_append_matches_definition(D, P, H, lengths):
    pool, table, k, v = filled(lengths, H, P, D, seed=3)
    ref = cache_ref.Pool(pool, D)
    for b, t in enumerate(lengths):
        for h in range(H):
            for which, x in (("k", k), ("v", v)):
                want = cache_ref.held(x[b, :t, h].double().cpu().numpy())
                assert (ref.rows(table[b].cpu().numpy(), t, h, which) == want).all()


def test_append_leaves_the_rest_alone():
    D, P = 128, 32
    table, pages = table_for([40], P, 2)
    pool = garbage_pool(pages, 2, P, D)
    before = cache_ref.Pool(pool, D)
    k = randn(1, 3, 2, D)
    sv.cache_append(k, k, pool, table, ints([37]), ints([2]))
    after = cache_ref.Pool(pool, D)
    for h in range(2):
        for s in (5, 6):
            before.put(int(table[0, 1]), h, s, "k", k[0, s - 5, h].double().cpu().numpy())
            before.put(int(table[0, 1]), h, s, "v", k[0, s - 5, h].double().cpu().numpy())
    assert (before.raw == after.raw).all()


def test_quantisation_extremes():
    """Ties, tiny and huge groups, zeros, NaN and infinities."""
    D, P = 64, 16
    x = torch.zeros((1, 8, 1, D), dtype=torch.float64)
    x[0, 0, 0, :32] = torch.arange(32, dtype=torch.float64) / 4 - 3.5        # scale 0.5, exact halves
    x[0, 1, 0, :32] = 3e38
    x[0, 2, 0, :32] = 2.0 ** -126
    x[0, 2, 0, 32:] = 2.0 ** -115 * torch.arange(32, dtype=torch.float64)
    x[0, 3] = torch.from_numpy(np.random.default_rng(1).standard_normal((1, D)) * 1e-30)
    x[0, 4, 0, :32] = torch.linspace(-7.2, 7.2, 32)
    x[0, 5, 0, 3], x[0, 5, 0, 4], x[0, 5, 0, 5] = math.inf, -math.inf, 2.0
    x[0, 6, 0, 7], x[0, 6, 0, 40] = math.nan, 1.0
    x[0, 7, 0, :] = math.inf
    xb = x.to(torch.bfloat16)
    table, pages = table_for([8], P, 1)
    pool = garbage_pool(pages, 1, P, D)
    status = ints([0])
    sv.cache_append(xb.to(DEV), xb.to(DEV), pool, table, ints([0]), status=status)
    assert status.tolist() == [sv.ST_BAD_ROW]
    k, v = sv.cache_read(pool, table, ints([0]), 8, D)
    want = cache_ref.held(xb.double().numpy()[0, :, 0])
    assert (k.double().cpu().numpy()[0, :, 0] == want).all() and torch.equal(k, v)


def test_every_bf16_pair_of_scale_and_value():
    """Each significand of the largest value against many others: the rounding of x/scale, ties included."""
    D, P = 128, 64
    rows = []
    for a in range(128, 256):
        rest = np.random.default_rng(a).integers(128, 256, 31) * 2.0 ** np.random.default_rng(a + 1).integers(-6, 1, 31)
        rows.append(np.concatenate([[a], np.minimum(rest, a) * np.where(np.arange(31) % 2, 1, -1)]))
    x = torch.from_numpy(np.stack(rows).reshape(1, 32, 1, D)).to(torch.bfloat16)
    table, pages = table_for([32], P, 1)
    pool = garbage_pool(pages, 1, P, D)
    sv.cache_append(x.to(DEV), x.to(DEV), pool, table, ints([0]))
    got = sv.cache_read(pool, table, ints([0]), 32, D)[0].double().cpu().numpy()
    assert (got[0, :, 0] == cache_ref.held(x.double().numpy()[0, :, 0])).all()


@pytest.mark.parametrize("D", [64, 128])
def test_append_strided_and_unaligned(D):
    P, H, n = 16, 2, 5
    wide = randn(2, n, 3 * H * D + 8, seed=5)
    for off in (0, 8, 1):                                        # 16-byte rows, and rows off by one value
        k = wide[..., off:off + H * D].unflatten(-1, (H, D))
        v = wide[..., off + H * D:off + 2 * H * D].unflatten(-1, (H, D))
        table, pages = table_for([n, n], P, 1)
        a, z = garbage_pool(pages, H, P, D), garbage_pool(pages, H, P, D)
        sv.cache_append(k, v, a, table, ints([0, 0]))
        sv.cache_append(k.contiguous(), v.contiguous(), z, table, ints([0, 0]))
        assert torch.equal(a, z)


def test_read_counts_and_missing_pages():
    D, P = 128, 16
    pool, table, k, _ = filled([20, 20], 2, P, D)
    table[1, 1] = -1
    status = ints([0, 0])
    got, _ = sv.cache_read(pool, table, ints([14, 14]), 6, D, ints([4, 6]), status=status)
    want = cache_ref.held(k[:, 14:20].double().cpu().numpy())
    want[0, 4:] = 0
    want[1, 2:] = 0
    assert (got.double().cpu().numpy() == want).all()
    assert status.tolist() == [0, sv.ST_BAD_PAGE]
    for bad in (7 << 20, -5):                                    # ids outside the pool
        table[1, 1] = bad
        status = ints([0, 0])
        got, _ = sv.cache_read(pool, table, ints([14, 14]), 6, D, ints([4, 6]), status=status)
        assert (got.double().cpu().numpy() == want).all() and status.tolist() == [0, sv.ST_BAD_PAGE]
        before = pool.clone()
        sv.cache_append(k[:, :6], k[:, :6], pool, table, ints([20, 16]), ints([0, 6]), status=status)
        assert torch.equal(before, pool)
    status = ints([0, 0])                                        # before the cache and past the table
    sv.cache_read(pool, table, ints([-3, 31]), 2, D, status=status)
    assert status.tolist() == [sv.ST_BAD_PAGE] * 2


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def trees(B, n, seed=0, max_depth=9):
    """Random trees, parents first: masks as int64 words and depths."""
    rng = np.random.default_rng(seed)
    mask = np.zeros((B, n, (n + 63) // 64), dtype=np.uint64)
    depth = np.zeros((B, n), dtype=np.int32)
    for b in range(B):
        for i in range(n):
            if i:
                p = int(rng.integers(max(0, i - 7), i))
                p = p if depth[b, p] < max_depth else 0
                mask[b, i] = mask[b, p]
                depth[b, i] = depth[b, p] + 1
            mask[b, i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return mask.view(np.int64), depth


def attend_case(ctx, n, hq, H, D, P, rows=None, tree=False, window=0, sinks=0, seed=0, qscale=2.0, scale=None, spare_width=0):
    rows_l = rows if rows is not None else [n] * len(ctx)
    total = [c + r for c, r in zip(ctx, rows_l)]
    width = max(1, max(-(-t // P) for t in total)) + spare_width
    pool, table, _, _ = filled(total, H, P, D, seed=seed, width=width)
    q = randn(len(ctx), n, hq, D, seed=seed + 7, scale=qscale)
    mask, depth = trees(len(ctx), n, seed) if tree else (None, None)
    status = ints([0] * len(ctx))
    r = sv.cache_attend(q, pool, table, ints(ctx), None if rows is None else ints(rows),
                        anc_mask=None if mask is None else torch.from_numpy(mask).to(DEV),
                        depth=None if depth is None else torch.from_numpy(depth).to(DEV),
                        window=window, sinks=sinks, scale=scale, want_lse=True, status=status)
    assert status.tolist() == [0] * len(ctx)
    ref = cache_ref.attend(q, cache_ref.Pool(pool, D), table.cpu().numpy(), ctx, rows, mask, depth, window, sinks, scale)
    cache_ref.check_attend(r.out, r.lse, ref)
    return r


@pytest.mark.parametrize("D,P", [(128, 64), (128, 32), (128, 16), (64, 64), (64, 32), (64, 16)])
@pytest.mark.parametrize("n,hq,H", [(1, 4, 1), (1, 1, 1), (4, 8, 2), (9, 7, 1), (3, 10, 2)])
def test_attend_chains(D, P, n, hq, H):
    attend_case([0, 1, 15, 16, 63, 64, 65, 130, 257], n, hq, H, D, P, seed=n + D)


@pytest.mark.parametrize("D,P", [(128, 64), (64, 16)])
@pytest.mark.parametrize("n,hq,H", [(5, 4, 1), (64, 4, 1), (65, 5, 1), (33, 16, 2)])
def test_attend_trees(D, P, n, hq, H):
    attend_case([0, 37, 200], n, hq, H, D, P, rows=[n, n // 2, 1], tree=True, seed=n)


def test_attend_tree_of_many_words():
    attend_case([70], 300, 2, 1, 64, 64, tree=True, seed=4)


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (17, 4), (64, 64), (100, 70), (1000, 4)])
@pytest.mark.parametrize("n,tree", [(1, False), (6, False), (40, True)])
def test_attend_window(window, sinks, n, tree):
    attend_case([0, 3, 64, 180, 333], n, 4, 2, 64, 16, tree=tree, window=window, sinks=sinks, seed=window)


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5)])
def test_attend_long(window, sinks):
    """Contexts long enough to be split, of very different lengths, few requests."""
    attend_case([5000, 9, 1200], 2, 4, 1, 128, 64, window=window, sinks=sinks, seed=11)


def test_attend_rows_without_keys():
    """Empty requests, rows past num_rows, and masks that leave a row nothing: 0 and -inf."""
    D, P = 128, 16
    r = attend_case([0, 0, 20], 4, 4, 1, D, P, rows=[0, 2, 3], spare_width=1)
    assert torch.equal(r.out[0], torch.zeros_like(r.out[0])) and torch.isneginf(r.lse[0]).all()
    assert torch.isneginf(r.lse[1, 2:]).all() and torch.isneginf(r.lse[2, 3]).all()
    pool, table, _, _ = filled([3], 1, P, D)
    mask = torch.tensor([[[1], [0], [6]]], dtype=torch.int64, device=DEV)      # row 1 sees nothing, no context
    q = randn(1, 3, 2, D)
    r = sv.cache_attend(q, pool, table, ints([0]), anc_mask=mask, want_lse=True)
    ref = cache_ref.attend(q, cache_ref.Pool(pool, D), table.cpu().numpy(), [0], None, mask.cpu().numpy())
    cache_ref.check_attend(r.out, r.lse, ref)
    assert torch.isneginf(r.lse[0, 1]).all() and (r.out[0, 1] == 0).all()


def test_attend_one_key_is_its_value():
    pool, table, _, v = filled([1, 1], 1, 16, 64)
    q = randn(2, 1, 3, 64, scale=5.0)
    out = sv.cache_attend(q, pool, table, ints([0, 0])).out
    want = cache_ref.held(v[:, :1].double().cpu().numpy())
    assert (out.double().cpu().numpy() == np.broadcast_to(want, out.shape)).all()


def test_attend_large_scores():
    """Scores far outside exp's range: the running maximum must carry them."""
    attend_case([150, 700], 3, 4, 1, 128, 64, seed=2, qscale=300.0)
    attend_case([150, 700], 3, 4, 1, 128, 64, seed=2, qscale=2.0, scale=40.0)


def test_attend_rising_scores():
    """Each key beats all before it, so that the maximum moves at every tile."""
    D, P, T = 64, 64, 1500
    table, pages = table_for([T + 1], P, 24)
    pool = garbage_pool(pages, 1, P, D)
    k = (torch.linspace(0, 1, T + 1, device=DEV)[None, :, None, None] * torch.ones(D, device=DEV)).to(torch.bfloat16)
    v = randn(1, T + 1, 1, D, seed=8)
    sv.cache_append(k, v, pool, table, ints([0]))
    for sign in (1.0, -1.0):
        q = torch.full((1, 1, 2, D), 16.0 * sign, device=DEV).to(torch.bfloat16)
        r = sv.cache_attend(q, pool, table, ints([T]), want_lse=True)
        cache_ref.check_attend(r.out, r.lse, cache_ref.attend(q, cache_ref.Pool(pool, D), table.cpu().numpy(), [T], None))


def test_attend_ignores_what_no_row_sees():
    """NaN and infinite scales past the end and outside every window change nothing."""
    D, P, ctx, n = 128, 16, 150, 3
    pool, table, _, _ = filled([ctx + n], 2, P, D, width=12)
    q = randn(1, n, 4, D)
    args = dict(window=40, sinks=4, want_lse=True)
    a = sv.cache_attend(q, pool, table, ints([ctx]), **args)
    clean = (a.out.clone(), a.lse.clone())
    r = D // 2 * P
    for t in list(range(4, ctx - 40 + 1)) + list(range(ctx + n, 160)):
        page = int(table[0, t // P])
        if page < 0:
            continue
        for off in (r, r + P * D // 16 + r):
            blk = pool[page, :, off:off + P * D // 16].view(torch.bfloat16).view(2, P, D // 32)
            blk[:, t % P] = NAN if t % 2 else math.inf
    b = sv.cache_attend(q, pool, table, ints([ctx]), **args)
    assert torch.equal(b.out, clean[0]) and torch.equal(b.lse, clean[1])


def test_attend_one_bad_query_stays_alone():
    pool, table, _, _ = filled([200], 1, 64, 128)
    q = randn(1, 4, 4, 128)
    a = sv.cache_attend(q, pool, table, ints([196]), want_lse=True)
    good = (a.out.clone(), a.lse.clone())
    q[0, 1, 2, 5] = NAN
    q[0, 3, 0, 0] = math.inf
    b = sv.cache_attend(q, pool, table, ints([196]), want_lse=True)
    keep = torch.ones((1, 4, 4), dtype=torch.bool, device=DEV)
    keep[0, 1, 2] = keep[0, 3, 0] = False
    assert torch.equal(b.out[keep], good[0][keep]) and torch.equal(b.lse[keep], good[1][keep])
    assert torch.isnan(b.out[0, 1, 2]).all()


def test_attend_missing_pages():
    """Positions without a page are left out and reported; nothing is read there."""
    D, P = 128, 16
    pool, table, _, _ = filled([100, 60], 2, P, D)
    q = randn(2, 2, 4, D)
    for bad in (-1, 1 << 30, pool.shape[0]):
        table[0, 2] = bad
        status = ints([0, 0])
        r = sv.cache_attend(q, pool, table, ints([98, 58]), want_lse=True, status=status)
        assert status.tolist() == [sv.ST_BAD_PAGE, 0]
        ref = cache_ref.attend(q, cache_ref.Pool(pool, D), table.cpu().numpy(), [98, 58], None)
        cache_ref.check_attend(r.out, r.lse, ref)


def test_attend_lengths_outside_the_table():
    """Contexts longer than the table, negative ones and row counts out of range are cut."""
    D, P = 64, 16
    pool, table, _, _ = filled([64, 64, 64], 1, P, D)
    q = randn(3, 2, 2, D)
    status = ints([0, 0, 0])
    r = sv.cache_attend(q, pool, table, ints([1 << 30, -7, 62]), ints([2, 1, 99]), want_lse=True, status=status)
    ref = cache_ref.attend(q, cache_ref.Pool(pool, D), table.cpu().numpy(), [64, 0, 62], [2, 1, 2])
    cache_ref.check_attend(r.out, r.lse, ref)
    assert status.tolist() == [sv.ST_BAD_PAGE, 0, 0]


@pytest.mark.parametrize("D", [64, 128])
def test_attend_strided_q_and_pool(D):
    P, H, n, hq = 32, 2, 4, 6
    pool, table, _, _ = filled([90, 40], H, P, D)
    wide = randn(2, n, hq * D + 24, seed=6)
    base = None
    for off in (0, 8, 3):
        q = wide[..., off:off + hq * D].unflatten(-1, (hq, D))
        ref = sv.cache_attend(q.contiguous(), pool, table, ints([86, 36]), want_lse=True)
        got = sv.cache_attend(q, pool, table, ints([86, 36]), want_lse=True)
        assert torch.equal(got.out, ref.out) and torch.equal(got.lse, ref.lse)
        base = base or ref
    q = wide[..., :hq * D].unflatten(-1, (hq, D))
    layers = garbage_pool(3, 5, P, D, lead=(pool.shape[0],))                   # [pages, layers, heads, block]
    layers[:, 1, 1:1 + H] = pool
    got = sv.cache_attend(q, layers[:, 1, 1:1 + H], table, ints([86, 36]), want_lse=True)
    assert torch.equal(got.out, base.out)


def test_attend_far_pages():
    """Pages more than 2^32 bytes apart."""
    D, P, H = 128, 64, 1
    pool, table, _, _ = filled([150, 70], H, P, D)
    pages = pool.shape[0]
    stride = (1 << 32) + (1 << 20)
    big = torch.empty(stride * (pages - 1) + pool.shape[-1], dtype=torch.uint8, device=DEV)
    far = big.as_strided((pages, H, pool.shape[-1]), (stride, pool.shape[-1], 1))
    far.copy_(pool)
    q = randn(2, 2, 4, D)
    a = sv.cache_attend(q, pool, table, ints([148, 68]), want_lse=True)
    b = sv.cache_attend(q, far, table, ints([148, 68]), want_lse=True)
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
    k, _ = sv.cache_read(far, table, ints([100, 0]), 50, D)
    assert torch.equal(k, sv.cache_read(pool, table, ints([100, 0]), 50, D)[0])


def test_attend_same_bits_every_time_and_on_another_stream():
    D, P = 128, 64
    ctx = [3000, 40, 900, 1500]
    pool, table, _, _ = filled([c + 5 for c in ctx], 2, P, D)
    q = randn(4, 5, 8, D)
    first = sv.cache_attend(q, pool, table, ints(ctx), want_lse=True)
    for _ in range(3):
        again = sv.cache_attend(q, pool, table, ints(ctx), want_lse=True)
        assert torch.equal(first.out, again.out) and torch.equal(first.lse, again.lse)
    c = ints(ctx)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = None if first.ws is None else torch.zeros_like(first.ws)
    with torch.cuda.stream(side):
        other = sv.cache_attend(q, pool, table, c, want_lse=True, ws=ws)
    given = sv.cache_attend(q, pool, table, c, want_lse=True, ws=None if ws is None else torch.zeros_like(ws), stream=side)
    side.synchronize()
    assert torch.equal(first.out, other.out) and torch.equal(first.out, given.out)


def test_attend_in_a_graph():
    D, P = 128, 64
    pool, table, _, _ = filled([2000, 300], 2, P, D)
    q, c = randn(2, 4, 8, D), ints([1996, 296])
    want = sv.cache_attend(q, pool, table, c, want_lse=True)
    out, lse = torch.zeros_like(want.out), torch.zeros_like(want.lse)
    ws = None if want.ws is None else torch.zeros_like(want.ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.cache_attend(q, pool, table, c, out=out, lse=lse, ws=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want.out) and torch.equal(lse, want.lse)


def test_attend_without_lse_and_pinned_lengths():
    pool, table, _, _ = filled([100], 1, 64, 128)
    q = randn(1, 2, 4, 128)
    a = sv.cache_attend(q, pool, table, ints([98]), want_lse=True)
    b = sv.cache_attend(q, pool, table, torch.tensor([98], dtype=torch.int32).pin_memory())
    torch.cuda.synchronize()
    assert b.lse is None and torch.equal(a.out, b.out)


def test_refusals_on_the_device():
    pool, table, _, _ = filled([100], 1, 64, 128)
    q = randn(1, 2, 4, 128)
    bad = [dict(q=q.float()), dict(q=q[..., :64]), dict(pool=pool[..., :-16]), dict(ctx_len=ints([1, 2])),
           dict(ctx_len=torch.ones(1, dtype=torch.int64, device=DEV)), dict(page_table=table.long()),
           dict(page_table=torch.cat([table, table])), dict(pool=pool.cpu()), dict(pool=pool.view(torch.int8)),
           dict(anc_mask=torch.zeros((1, 2, 2), dtype=torch.int64, device=DEV)), dict(depth=ints([[0, 1]])),
           dict(out=torch.empty_like(q)[:, :1]), dict(lse=torch.empty((1, 2, 3), device=DEV)), dict(window=-1),
           dict(q=q[:, :, :3].expand(1, 2, 3, 128), pool=pool.expand(-1, 2, -1)), dict(ctx_len=torch.ones(1, dtype=torch.int32)),
           dict(scale=0.0), dict(num_rows=ints([[1]])), dict(status=ints([1, 1]))]
    for kw in bad:
        a = dict(q=q, pool=pool, page_table=table, ctx_len=ints([98]))
        a.update(kw)
        with pytest.raises(sv.SpecError):
            sv.cache_attend(a.pop("q"), a.pop("pool"), a.pop("page_table"), a.pop("ctx_len"), **a)
    with pytest.raises(sv.SpecError):
        sv.cache_append(q, q, pool, table, ints([0]))                          # 4 heads into a pool of 1
    with pytest.raises(sv.SpecError):
        sv.cache_compact(pool, table, ints([0]), ints([[0]]), ints([0]), 128)  # one layer's pool
    L = sv.cache._lib()
    host = torch.zeros(9216 * 2, dtype=torch.uint8)
    rc = L.spec_cache_read(host.data_ptr() // 16 * 16 + 16, 9216, 9216, 1, sv._p(table), 2, 2, sv._p(ints([0])), None,
                           1, 1, 1, 128, 64, sv._p(q), sv._p(q), None, None)
    assert rc == 1 and b"device memory" in L.spec_last_error()


# ---------------------------------------------------------------------------
# compaction
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,P,layers,H", [(128, 64, 1, 2), (64, 16, 3, 1), (128, 16, 33, 5)])
def test_compact(D, P, layers, H):
    paths = [[0, 1, 2, -1], [0, 3, 17, 18], [0, -1, -1, -1], [0, 2, 3, 30], [0, 1, 9, 20]]
    acc, ctx = [2, 3, 0, 2, 9], [5, 100, 0, 15, 63]
    table, pages = table_for([c + 31 for c in ctx], P, 12)
    pool = garbage_pool(pages, H, P, D, lead=(layers,))
    want = pool.cpu().numpy().copy()
    tab = table.cpu().numpy()
    for layer in range(layers):
        ref = cache_ref.Pool(pool[layer], D)
        for b, path in enumerate(paths):
            rows = {}
            for j in range(min(acc[b], 3) + 1):
                for h in range(H):
                    for w in "kv":
                        t = ctx[b] + path[j]
                        rows[j, h, w] = [x.copy() for x in ref.bytes_of(tab[b, t // P], h, t % P, w)]
            for (j, h, w), (c, s) in rows.items():
                t = ctx[b] + j
                at = ref.bytes_of(tab[b, t // P], h, t % P, w)
                at[0][:], at[1][:] = c, s
        want[layer] = ref.raw
    status = ints([0] * 5)
    sv.cache_compact(pool, table, ints(ctx), ints(paths), ints(acc), D, status=status)
    assert (pool.cpu().numpy() == want).all() and status.tolist() == [0] * 5


def test_compact_long_path():
    """More moves than a batch of loads, sources that are later destinations."""
    D, P, n = 64, 16, 60
    path = [0] + list(range(2, 2 * 29 + 1, 2))
    table, pages = table_for([n], P, 4)
    pool = garbage_pool(pages, 1, P, D, lead=(2,))
    before = [cache_ref.Pool(pool[i], D) for i in range(2)]
    sv.cache_compact(pool, table, ints([0]), ints([path]), ints([len(path) - 1]), D)
    tab = table[0].cpu().numpy()
    for i in range(2):
        after = cache_ref.Pool(pool[i], D)
        for j, t in enumerate(path):
            for w in "kv":
                a, z = before[i].bytes_of(tab[t // P], 0, t % P, w), after.bytes_of(tab[j // P], 0, j % P, w)
                assert (a[0] == z[0]).all() and (a[1] == z[1]).all()


def test_compact_reports_bad_entries():
    D, P = 64, 16
    table, pages = table_for([40, 40], P, 3)
    table[1, 2] = -1
    pool = garbage_pool(pages, 1, P, D, lead=(1,))
    want = pool.clone()
    status = ints([0, 0])
    sv.cache_compact(pool, table, ints([0, 30]), ints([[0, 0, 1], [0, 5, -1]]), ints([2, 1]), D, status=status)
    assert torch.equal(pool, want)
    assert status.tolist() == [64, sv.ST_BAD_PAGE]


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
class Pages:
    """The pages' rules, one request at a time."""

    def __init__(self, s, P):
        self.table, self.held = s.page_table.tolist(), s.num_held.tolist()
        self.ref, self.free, self.left, self.P = s.ref.tolist(), s.free_list.tolist(), int(s.num_free[0]), P

    def need(self, t):
        return -(-max(t, 0) // self.P)

    def reserve(self, length):
        asked, taken, have, bits = 0, 0, self.left, []
        for r, t in enumerate(length):
            bits.append(0)
            need = self.need(t)
            if need > len(self.table[r]):
                bits[-1] = 128
                continue
            need = max(0, need - self.held[r])
            if asked + need > have and need:
                bits[-1] = 256
            elif need:
                for j in range(need):
                    page = self.free[have - 1 - asked - j]
                    self.table[r][self.held[r] + j] = page
                    self.ref[page] = 1
                self.held[r] += need
                taken += need
            asked += need
        self.left -= taken
        return bits

    def release(self, length):
        gone = set()
        for r, t in enumerate(length):
            keep = min(self.need(t), self.held[r])
            for j in range(keep, self.held[r]):
                page = self.table[r][j]
                self.ref[page] -= 1
                gone.add(page)
                self.table[r][j] = -1
            self.held[r] = keep
        for page in sorted(gone):
            if self.ref[page] == 0:
                self.free[self.left] = page
                self.left += 1

    def fork(self, src, dst, length):
        bits, new, asked, have = [], [], 0, self.left
        for s, d in zip(src, dst):
            bits.append(0)
            new.append(-1)
            if not (0 <= s < len(self.held) and 0 <= d < len(self.held)) or s == d:
                bits[-1] = 128
                continue
            full, tail = max(length[s], 0) // self.P, max(length[s], 0) % self.P
            if self.held[d] or full + (tail > 0) > self.held[s]:
                bits[-1] = 128
                continue
            if tail:
                asked += 1
                if asked > have:
                    bits[-1] = 256
                    continue
                new[-1] = self.free[have - asked]
                self.left -= 1
                self.table[d][full] = new[-1]
                self.ref[new[-1]] = 1
            for j in range(full):
                self.table[d][j] = self.table[s][j]
                self.ref[self.table[s][j]] += 1
            self.held[d] = full + (tail > 0)
        return bits, new

    def same(self, s):
        return (self.table == s.page_table.tolist() and self.held == s.num_held.tolist() and self.ref == s.ref.tolist()
                and self.free == s.free_list.tolist() and self.left == int(s.num_free[0]))


@pytest.mark.parametrize("R,M,N,P", [(3, 4, 20, 16), (40, 9, 150, 64), (1500, 3, 3000, 32)])
def test_pages_random_walk(R, M, N, P):
    rng = np.random.default_rng(R)
    s = sv.page_state(R, M, N, DEV)
    ref = Pages(s, P)
    pool = torch.zeros((1, N, 1, sv.cache_block_bytes(64, P)), dtype=torch.uint8, device=DEV)
    length = np.zeros(R, dtype=int)
    for step in range(12):
        if step % 3 == 0:
            want = rng.integers(-2, M * P + 2, R) if step % 2 else np.minimum(length + rng.integers(0, 2 * P, R), M * P)
            status = ints([0] * R)
            sv.cache_reserve(s, ints(want.tolist()), P, status=status)
            assert ref.reserve(want.tolist()) == status.tolist()
            length = np.where(status.cpu().numpy() == 0, np.maximum(want, length), length).clip(0, None)
        elif step % 3 == 1:
            empty = [r for r in range(R) if ref.held[r] == 0]
            full = [r for r in range(R) if ref.held[r] > 0]
            if empty and full:
                dst = list(rng.permutation(empty)) + [R + 3, full[0]]
                src = [int(rng.choice(full)) for _ in dst]
                cut = [min(int(length[r]), ref.held[r] * P) for r in range(R)]
                status = ints([0] * len(dst))
                new = sv.cache_fork(pool, s, ints(src), ints([int(d) for d in dst]), ints(cut), 64, status=status)
                bits, want_new = ref.fork(src, [int(d) for d in dst], cut)
                assert bits == status.tolist() and want_new == new.tolist()
                for f, d in enumerate(dst):
                    if bits[f] == 0:
                        length[d] = cut[src[f]]
        else:
            want = rng.integers(0, M * P, R) * (rng.random(R) < 0.6)
            sv.cache_release(s, ints(want.tolist()), P)
            ref.release(want.tolist())
            length = np.minimum(length, want)
        assert ref.same(s)
    sv.cache_release(s, ints([0] * R), P)
    assert int(s.num_free[0]) == N and sorted(s.free_list.tolist()) == list(range(N)) and not s.ref.any()


@pytest.mark.parametrize("D,P,H,layers", [(128, 64, 2, 3), (64, 16, 1, 1)])
def test_fork_copies_the_last_rows_only(D, P, H, layers):
    s = sv.page_state(4, 4, 12, DEV)
    sv.cache_reserve(s, ints([2 * P + 5, P, 0, 0]), P)
    pool = garbage_pool(12, H, P, D, lead=(layers,))
    before = pool.clone()
    new = sv.cache_fork(pool, s, ints([0, 1]), ints([2, 3]), ints([2 * P + 5, P, 0, 0]), D)
    old, page = int(s.page_table[0, 2]), int(new[0])
    assert int(new[1]) == -1 and s.page_table[2, :2].tolist() == s.page_table[0, :2].tolist()
    for layer in range(layers):
        want, got = cache_ref.Pool(before[layer], D), cache_ref.Pool(pool[layer], D)
        for h in range(H):
            for slot in range(5):
                for w in "kv":
                    src, dst = want.bytes_of(old, h, slot, w), want.bytes_of(page, h, slot, w)
                    dst[0][:], dst[1][:] = src[0], src[1]
        assert (want.raw == got.raw).all()


def test_pages_damaged_state_is_survived():
    """Ids outside the pool and references that nobody holds are reported, and nothing else moves."""
    P = 16
    s = sv.page_state(2, 3, 6, DEV)
    sv.cache_reserve(s, ints([48, 20]), P)
    s.page_table[0, 1] = 1 << 29
    s.ref[s.page_table[1, 0].item()] = 0
    status = ints([0, 0])
    sv.cache_release(s, ints([0, 0]), P, status=status)
    assert status.tolist() == [sv.ST_BAD_PAGE] * 2
    assert int(s.num_free[0]) == 4 and (s.ref >= 0).all()


def test_many_pages():
    """A pool of 2^20 pages: the release's bitmap at its largest."""
    n = 1 << 20
    s = sv.page_state(8, 1 << 17, n, DEV)
    want = ints([16 << 17] * 8)
    sv.cache_reserve(s, want, 16)
    assert int(s.num_free[0]) == 0 and (s.ref == 1).all()
    assert s.page_table.flatten().tolist()[:3] == [0, 1, 2]
    sv.cache_release(s, ints([0] * 8), 16)
    assert int(s.num_free[0]) == n and torch.equal(s.free_list, torch.arange(n, dtype=torch.int32, device=DEV))
