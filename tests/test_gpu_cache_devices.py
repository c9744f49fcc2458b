"""Tensors of another device than the pool's are refused.  They need no second GPU:
a tensor without storage that says it lies there is enough for the checks."""
import pytest
import torch

import speculative_decoding_draft_sampling_gb300 as sv
from test_gpu_cache import filled, ints, randn

pytestmark = pytest.mark.gpu


class Elsewhere(torch.Tensor):
    @staticmethod
    def __new__(cls, like):
        return torch.Tensor._make_wrapper_subclass(cls, like.shape, strides=like.stride(), dtype=like.dtype,
                                                   device=torch.device("cuda", 1))

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def refused(call, *args, **kw):
    with pytest.raises(sv.SpecError, match="cuda:1"):
        call(*args, **kw)


def test_tensors_elsewhere_are_refused():
    pool, table, k, _ = filled([100], 1, 64, 128)
    q, n = randn(1, 2, 4, 128), ints([98])
    attend = dict(q=q, pool=pool, page_table=table, ctx_len=n)
    for name, t in dict(attend, num_rows=n, out=torch.empty_like(q), lse=torch.empty((1, 2, 4), device=q.device),
                        status=n, ws=torch.zeros(1 << 24, dtype=torch.uint8, device=q.device)).items():
        if name != "pool":
            refused(sv.cache_attend, **dict(attend, **{name: Elsewhere(t)}))
    refused(sv.cache_append, Elsewhere(k), k, pool, table, n)
    refused(sv.cache_append, k, k, pool, table, Elsewhere(n))
    refused(sv.cache_read, pool, Elsewhere(table), n, 2, 128)
    refused(sv.cache_compact, pool[None], table, n, ints([[0]]), Elsewhere(n), 128)


def test_page_states_elsewhere_are_refused():
    s = sv.page_state(2, 2, 4, torch.device("cuda", 0))
    pool = torch.zeros((1, 4, 1, sv.cache_block_bytes(64, 16)), dtype=torch.uint8, device="cuda")
    n, one = ints([5, 0]), ints([1])
    refused(sv.cache_reserve, s, Elsewhere(n), 16)
    refused(sv.cache_fork, pool, s, ints([0]), Elsewhere(one), n, 64)
    for name in ("page_table", "num_held", "free_list", "num_free"):
        other = sv.page_state(2, 2, 4, torch.device("cuda", 0))
        setattr(other, name, Elsewhere(getattr(other, name)))
        refused(sv.cache_release, other, n, 16)
        refused(sv.cache_fork, pool, other, ints([0]), one, n, 64)
