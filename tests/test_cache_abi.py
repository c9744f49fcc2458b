"""The cache calls' refusals: bad arguments are reported before any device
work (no GPU needed), with a text that names the problem."""
import ctypes

import pytest
import torch

import speculative_decoding_draft_sampling_gb300 as sv
from speculative_decoding_draft_sampling_gb300 import cache

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    sv.build()
    return cache._lib()


def _err(lib):
    return lib.spec_last_error().decode()


def _attend(lib, **kw):
    a = dict(q=16, q_bs=512, q_rs=512, q_hs=128, pool=16, ps=9216, hs=9216, pages=4, table=16, ts=4, width=4, ctx=16,
             rows=0, mask=0, depth=0, window=0, sinks=0, scale=0.1, B=1, n=1, hq=4, hkv=1, d=128, page=64, out=16,
             lse=0, status=0, ws=0, ws_bytes=0, stream=0)
    a.update(kw)
    return lib.spec_cache_attend(*a.values())


@pytest.mark.parametrize("kw,code,text", [
    (dict(hq=5, hkv=2), INVALID, "multiple of kv_heads"),
    (dict(window=-1), INVALID, "window"),
    (dict(sinks=-1), INVALID, "sinks"),
    (dict(scale=0.0), INVALID, "scale"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(depth=16), INVALID, "anc_mask"),
    (dict(n=1025), UNSUPPORTED, "1024"),
    (dict(n=-1), INVALID, "n >= 0"),
    (dict(d=96), UNSUPPORTED, "head_dim"),
    (dict(page=48), UNSUPPORTED, "page_size"),
    (dict(pool=8), INVALID, "16 bytes"),
    (dict(ps=9208), INVALID, "16 bytes"),
    (dict(hs=4608), INVALID, "below a block"),
    (dict(pool=0), INVALID, "null"),
    (dict(pages=1 << 21), UNSUPPORTED, "2^20"),
])
def test_attend_refuses(lib, kw, code, text):
    assert _attend(lib, **kw) == code
    assert text in _err(lib)


def test_empty_calls_are_fine(lib):
    assert _attend(lib, B=0) == 0
    assert _attend(lib, n=0) == 0
    assert lib.spec_cache_append(*[0] * 8, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 5, 1, 128, 64, 0, 0) == 0


def test_block_bytes(lib):
    assert cache.cache_block_bytes(128, 64) == 9216 and cache.cache_block_bytes(64, 16) == 1152
    with pytest.raises(sv.SpecError, match="head_dim"):
        cache.cache_block_bytes(80, 64)


def test_workspace_size(lib):
    assert lib.spec_cache_attend_workspace_size(4, 1025, 32, 8, 128) == 0
    assert lib.spec_cache_attend_workspace_size(4, 4, 30, 8, 128) == 0


def test_page_calls_refuse(lib):
    def reserve(**kw):
        a = dict(table=16, ts=4, width=4, held=16, ref=16, free=16, left=16, pages=8, length=16, R=2, page=64, status=0, stream=0)
        a.update(kw)
        return lib.spec_cache_reserve(*a.values())
    assert reserve(page=8) == UNSUPPORTED and "page_size" in _err(lib)
    assert reserve(pages=0) == INVALID and "num_pages" in _err(lib)
    assert reserve(pages=(1 << 20) + 1) == UNSUPPORTED
    assert reserve(ref=0) == INVALID and "null" in _err(lib)
    assert reserve(ts=3) == INVALID and "table_stride" in _err(lib)
    assert reserve(R=-1) == INVALID
    assert reserve(R=0) == 0


def test_compact_refuses(lib):
    def compact(**kw):
        a = dict(pool=16, layers=2, ls=9216 * 4, ps=9216, hs=9216, pages=4, table=16, ts=4, width=4, ctx=16, path=16,
                 pw=5, acc=16, B=1, heads=1, d=128, page=64, status=0, stream=0)
        a.update(kw)
        return lib.spec_cache_compact(*a.values())
    assert compact(pw=0) == INVALID and "path_width" in _err(lib)
    assert compact(pw=1025) == UNSUPPORTED
    assert compact(layers=0) == INVALID and "layers" in _err(lib)
    assert compact(ls=16) == INVALID and "below a block" in _err(lib)


def test_binding_refuses_host_tensors(lib):
    z = torch.zeros
    with pytest.raises(sv.SpecError, match="CUDA"):
        sv.cache_attend(z(1, 1, 4, 128, dtype=torch.bfloat16), z(4, 1, 9216, dtype=torch.uint8),
                        z(1, 4, dtype=torch.int32), z(1, dtype=torch.int32))
    with pytest.raises(sv.SpecError, match="CUDA"):
        sv.cache_append(z(1, 1, 1, 128, dtype=torch.bfloat16), z(1, 1, 1, 128, dtype=torch.bfloat16),
                        z(4, 1, 9216, dtype=torch.uint8), z(1, 4, dtype=torch.int32), z(1, dtype=torch.int32))
