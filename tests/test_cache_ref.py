"""The 64-bit cache reference against closed forms (CPU)."""
import numpy as np
import pytest
import torch

import cache_ref


def test_round5():
    assert cache_ref.round5([1.0, 33 / 32, 1 + 1 / 32 + 1e-9, 1 + 3 / 32, 31.5]).tolist() == [1, 1, 1 + 1 / 16, 1 + 1 / 8, 32]
    assert cache_ref.round5(2.0 ** -121) == 0


def test_quantise_steps():
    x = np.zeros(32)
    x[:15] = np.arange(-7, 8)                 # amax 7: scale 1, codes exact
    c, s = cache_ref.quantise(x)
    assert s.tolist() == [1.0] and c[:15].tolist() == list(range(1, 16))
    assert (cache_ref.held(x) == x).all()
    x[20:23] = [2.5, 3.5, -2.5]               # halves go to the even step
    assert (cache_ref.held(x)[20:23] == [2, 4, -2]).all()


def test_values_fit_bf16():
    x = torch.randn(64, 128, dtype=torch.float64).mul(3).bfloat16().double().numpy()
    v = torch.from_numpy(cache_ref.held(x))
    assert (v.bfloat16().double() == v).all()


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_pool_roundtrip(D, P):
    pool = cache_ref.Pool(torch.zeros((2, 1, P * D * 9 // 8), dtype=torch.uint8), D)
    x = np.random.default_rng(0).standard_normal((2, P, 2, D)).astype(np.float32).astype(np.float64)
    for page in range(2):
        for s in range(P):
            for w, which in enumerate("kv"):
                pool.put(page, 0, s, which, x[page, s, w])
    for w, which in enumerate("kv"):
        got = pool.rows(np.array([1, 0]), 2 * P, 0, which)
        assert (got == cache_ref.held(np.concatenate([x[1, :, w], x[0, :, w]]))).all()


def test_seen_by():
    vis = cache_ref.seen_by(6, 3, 4, None, None, 3, 1)
    assert vis[0].tolist() == [True, False, False, False, True, True, True, False, False]
    assert vis[2].tolist() == [True] + [False] * 5 + [True] * 3
    assert not vis[3].any()
    mask = np.array([[1], [3], [5]], dtype=np.int64)
    vis = cache_ref.seen_by(2, 3, 3, mask, np.array([0, 1, 1]), 2, 0)
    assert vis.tolist() == [[False, True, True, False, False], [False, False, True, True, False], [False, False, True, False, True]]


def test_attend_closed_form():
    D = 64
    pool = cache_ref.Pool(torch.zeros((1, 1, 16 * D * 9 // 8), dtype=torch.uint8), D)
    for t in range(4):
        pool.put(0, 0, t, "v", np.full(D, 7.0 * (t + 1)))
    q = torch.ones((1, 1, 1, D), dtype=torch.bfloat16)        # keys are 0: all weights equal
    out, lse, _, _ = cache_ref.attend(q, pool, np.zeros((1, 1), dtype=int), [3], None)
    assert np.allclose(out, 7.0 * 2.5) and np.allclose(lse, np.log(4))


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (9, 2), (40, 30)])
@pytest.mark.parametrize("tree", [False, True])
def test_attend_many_is_attend(window, sinks, tree):
    """The form for many rows agrees with the one that goes key by key."""
    rng = np.random.default_rng(window + tree)
    D, P, n, H = 64, 16, 70, 2
    raw = rng.integers(0, 256, (9, H, P * D * 9 // 8), dtype=np.uint8)
    pool = cache_ref.Pool(torch.from_numpy(raw), D)
    for page in range(9):
        for h in range(H):
            for slot in range(P):
                for w in "kv":
                    pool.put(page, h, slot, w, rng.standard_normal(D))
    table = np.array([[3, 0, 5, 1, 8, 4, 2], [6, 7, -1, 1 << 20, 0, 3, 5]])
    ctx, rows = [33, 20], [n, 50]
    mask = depth = None
    if tree:
        low = np.tril(rng.integers(0, 2, (2, n, n)), -1) + np.eye(n, dtype=int)
        mask = np.zeros((2, n, 2), dtype=np.uint64)
        for j in range(n):
            mask[:, :, j // 64] |= low[:, :, j].astype(np.uint64) << np.uint64(j % 64)
        mask, depth = mask.view(np.int64), 3 + rng.integers(0, 20, (2, n)).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((2, n, 4, D)))
    want = cache_ref.attend(q, pool, table, ctx, rows, mask, depth, window, sinks)
    got = cache_ref.attend_many(q, pool, table, ctx, rows, mask, depth, window, sinks)
    for a, z in zip(got, want):
        assert (np.isneginf(a) == np.isneginf(z)).all()
        assert np.allclose(a, z, rtol=1e-12, atol=1e-12)
