"""GPU parity of cache_attend with its 64-bit reference where a kv head has more
rows than the register kernel takes (48): the cases in which the tcgen05 kernel
has code of its own."""
import pytest
import torch

import cache_ref
import speculative_decoding_draft_sampling_gb300 as sv
from test_gpu_cache import DEV, filled, ints, randn

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
