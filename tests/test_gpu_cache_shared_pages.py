"""Requests that are cut back into a page which a fork made shared: cache_release
reports them, and a fork at the shorter length is the way on."""
import pytest
import torch

import speculative_decoding_draft_sampling_gb300 as sv
from test_gpu_cache import DEV, ints, randn

pytestmark = pytest.mark.gpu

D, H = 64, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def forked(P):
    """Request 0 at 2P + 5 tokens and its fork, request 1; request 2 is free."""
    s = sv.page_state(3, 4, 16, DEV)
    pool = torch.zeros((1, 16, H, sv.cache_block_bytes(D, P)), dtype=torch.uint8, device=DEV)
    length = ints([2 * P + 5, 0, 0])
    sv.cache_reserve(s, length, P)
    k = randn(1, 2 * P + 5, H, D)
    sv.cache_append(k, k, pool[0], s.page_table[:1], ints([0]))
    sv.cache_fork(pool, s, ints([0]), ints([1]), length, D)
    return s, pool


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("cut,bits", [
    ([2, 5, 2, 5], [0, 0]),        # nothing is cut: both end in pages of their own
    ([1, 3, 2, 5], [1, 0]),        # request 0 ends inside a shared page
    ([1, 3, 1, 1], [1, 1]),        # both do
    ([1, 0, 2, 5], [0, 0]),        # a full page is not written to
    ([1, 3, 0, 0], [0, 0]),        # the other one lets go of it in the same call
    ([0, 0, 0, 9], [0, 0]),
])
def test_release_reports_shared_pages(P, cut, bits):
    s, _ = forked(P)
    status = ints([0, 0, 0])
    sv.cache_release(s, ints([cut[0] * P + cut[1], cut[2] * P + cut[3], 0]), P, status=status)
    assert status.tolist() == [sv.ST_SHARED_PAGE * b for b in bits] + [0]


@pytest.mark.parametrize("P", [16, 32])
def test_fork_at_the_shorter_length_goes_on(P):
    s, pool = forked(P)
    table, t = s.page_table, P + 3
    before = sv.cache_read(pool[0], table[1:2], ints([0]), 2 * P + 5, D)[0].clone()
    sv.cache_fork(pool, s, ints([0]), ints([2]), ints([t, 0, 0]), D)
    status = ints([0, 0, 0])
    sv.cache_release(s, ints([0, 2 * P + 5, t]), P, status=status)
    assert status.tolist() == [0, 0, 0]
    more = randn(1, 4, H, D, seed=3)
    sv.cache_append(more, more, pool[0], table[2:3], ints([t]))
    assert torch.equal(sv.cache_read(pool[0], table[1:2], ints([0]), 2 * P + 5, D)[0], before)
    got = sv.cache_read(pool[0], table[2:3], ints([0]), t, D)[0]
    assert torch.equal(got, before[:, :t])
