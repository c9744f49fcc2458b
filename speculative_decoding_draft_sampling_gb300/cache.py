"""The paged 4-bit KV cache that a verification pass reads, writes and cuts
back (C ABI: include/spec_cache.h).

A pool is a uint8 CUDA tensor [pages, kv_heads, block] for one layer, or
[layers, pages, kv_heads, block] where a call works on all layers
(cache_compact, cache_fork); block = cache_block_bytes(head_dim, page_size).
A block holds one page of P tokens of one kv head:

    K codes [P][D/2] | K scales bf16 [P][D/32] | V codes [P][D/2] | V scales bf16 [P][D/32]

page_table [B, M] int32 names the pages of each request in order (-1: none).
`status` arguments are optional int32 [B] tensors; bits are OR-ed in.

  cache_append   quantise rows of K and V into the cache
  cache_read     rows of the cache as bf16 values
  cache_attend   attention of drafted rows over the cache (chains, ancestor
                 masks, sliding window with sinks)
  cache_compact  keep an accepted path's rows, in place
  cache_reserve, cache_fork, cache_release   pages of growing, forked and
                 finished requests
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import SpecError, _check, _cuda, _load

ST_BAD_PAGE, ST_NO_PAGE = 128, 256

_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = _load()
        P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        lib.spec_cache_block_bytes.argtypes = [i32, i32]
        lib.spec_cache_block_bytes.restype = sz
        lib.spec_cache_attend_workspace_size.argtypes = [i32] * 5
        lib.spec_cache_attend_workspace_size.restype = sz
        lib.spec_cache_append.argtypes = [P, i64, i64, i64, P, i64, i64, i64, P, i64, i64, i32, P, i64, i32, P, P,
                                          i32, i32, i32, i32, i32, P, P]
        lib.spec_cache_read.argtypes = [P, i64, i64, i32, P, i64, i32, P, P, i32, i32, i32, i32, i32, P, P, P, P]
        lib.spec_cache_attend.argtypes = [P, i64, i64, i64, P, i64, i64, i32, P, i64, i32, P, P, P, P, i32, i32, f32,
                                          i32, i32, i32, i32, i32, i32, P, P, P, P, sz, P]
        lib.spec_cache_compact.argtypes = [P, i32, i64, i64, i64, i32, P, i64, i32, P, P, i32, P,
                                           i32, i32, i32, i32, P, P]
        lib.spec_cache_reserve.argtypes = [P, i64, i32, P, P, P, P, i32, P, i32, i32, P, P]
        lib.spec_cache_release.argtypes = [P, i64, i32, P, P, P, P, i32, P, i32, i32, P, P]
        lib.spec_cache_fork.argtypes = [P, i32, i64, i64, i64, P, i64, i32, P, P, P, P, i32, P, P, P, i32, i32,
                                        i32, i32, i32, P, P, P]
        for name in ("append", "read", "attend", "compact", "reserve", "release", "fork"):
            getattr(lib, "spec_cache_" + name).restype = i32
        _bound = lib
    return _bound


def cache_block_bytes(head_dim: int, page_size: int) -> int:
    """Bytes of one page of one kv head."""
    n = int(_lib().spec_cache_block_bytes(int(head_dim), int(page_size)))
    if n == 0:
        raise SpecError(f"unsupported cache shape: head_dim is 64 or 128 and page_size 16, 32 or 64 "
                        f"(got {head_dim} and {page_size})")
    return n


_i32, _bf16, _u8 = torch.int32, torch.bfloat16, torch.uint8


# A decoding step makes these calls for every layer, so the checks below look at
# each tensor once and say what is wrong only where something is.
def _ints(t, name: str, *shape) -> int:
    """The address of a contiguous int32 tensor of this shape."""
    if isinstance(t, torch.Tensor) and t.dtype is _i32 and t.shape == shape and t.is_contiguous() \
            and (t.is_cuda or t.is_pinned()):
        return t.data_ptr()
    _cuda(t, name, _i32)
    raise SpecError(f"{name} must be a contiguous {list(shape)} int32 tensor")


def _opt(t, name: str, *shape):
    return None if t is None else _ints(t, name, *shape)


def _pool(pool, dims: int, head_dim: int):
    """(page_size, kv_heads, num_pages) of a pool of `dims` dimensions."""
    if not isinstance(pool, torch.Tensor) or not pool.is_cuda or pool.dtype is not _u8 or pool.dim() != dims \
            or pool.stride(-1) != 1:
        raise SpecError("pool must be a uint8 CUDA tensor "
                        + ("[pages, kv_heads, block]" if dims == 3 else "[layers, pages, kv_heads, block]")
                        + " with unit element stride")
    pages, heads, block = pool.shape[-3:]
    page = block * 8 // (9 * head_dim)
    if page not in (16, 32, 64) or page * head_dim * 9 != block * 8:
        raise SpecError(f"a block of {block} bytes is no page of head_dim {head_dim}")
    return page, heads, pages


def _table(page_table, B: Optional[int] = None):
    """B, M, the row stride and the address of a page table."""
    if isinstance(page_table, torch.Tensor) and page_table.dtype is _i32 and page_table.dim() == 2 \
            and (page_table.is_cuda or page_table.is_pinned()):
        (rows, width), (stride, unit) = page_table.shape, page_table.stride()
        if unit == 1 and (B is None or rows == B):
            return rows, width, stride, page_table.data_ptr()
    _cuda(page_table, "page_table", _i32)
    raise SpecError("page_table must be [B, M] int32 with unit element stride")


def _handle(stream, device: torch.device) -> int:
    """The stream's handle: of the one given, else of the device's current one."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def cache_append(k, v, pool, page_table, start, count=None, *, status=None, stream=None) -> None:
    """Write k, v [B, n, kv_heads, D] bf16 (any strides, unit element stride)
    into the cache in 4 bits: row (b, i), i < count[b] (default n), at position
    start[b] + i.  Groups of 32 values share a scale."""
    if not (isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and k.dtype is _bf16 and v.dtype is _bf16
            and (k.is_cuda or k.is_pinned()) and (v.is_cuda or v.is_pinned())):
        _cuda(k, "k", _bf16)
        _cuda(v, "v", _bf16)
    shape = k.shape
    if len(shape) != 4 or v.shape != shape:
        raise SpecError("k and v must be [B, n, kv_heads, D] with unit element stride")
    B, n, H, D = shape
    kb, kr, kh, k1 = k.stride()
    vb, vr, vh, v1 = v.stride()
    if k1 != 1 or v1 != 1:
        raise SpecError("k and v must be [B, n, kv_heads, D] with unit element stride")
    page, heads, pages = _pool(pool, 3, D)
    if heads != H:
        raise SpecError(f"the pool has {heads} kv heads, k and v {H}")
    _, M, ts, tp = _table(page_table, B)
    ps, hs, _ = pool.stride()
    rc = _lib().spec_cache_append(k.data_ptr(), kb, kr, kh, v.data_ptr(), vb, vr, vh, pool.data_ptr(), ps, hs, pages,
                                  tp, ts, M, _ints(start, "start", B), _opt(count, "count", B), B, n, H, D, page,
                                  _opt(status, "status", B), _handle(stream, pool.device))
    if rc:
        _check(rc, "spec_cache_append")


def cache_read(pool, page_table, start, n: int, head_dim: int, count=None, *, k=None, v=None, status=None,
               stream=None):
    """Rows of the cache as bf16 values, exactly what the codes stand for:
    (k, v), each [B, n, kv_heads, D]; rows i >= count[b] are 0."""
    page, H, pages = _pool(pool, 3, head_dim)
    B, M, ts, tp = _table(page_table)
    shape = (B, n, H, head_dim)
    if k is None:
        k = torch.empty(shape, dtype=_bf16, device=pool.device)
    elif _cuda(k, "k", _bf16).shape != shape or not k.is_contiguous():
        raise SpecError(f"k must be a contiguous {list(shape)} bf16 tensor")
    if v is None:
        v = torch.empty(shape, dtype=_bf16, device=pool.device)
    elif _cuda(v, "v", _bf16).shape != shape or not v.is_contiguous():
        raise SpecError(f"v must be a contiguous {list(shape)} bf16 tensor")
    ps, hs, _ = pool.stride()
    rc = _lib().spec_cache_read(pool.data_ptr(), ps, hs, pages, tp, ts, M, _ints(start, "start", B),
                                _opt(count, "count", B), B, n, H, head_dim, page, k.data_ptr(), v.data_ptr(),
                                _opt(status, "status", B), _handle(stream, pool.device))
    if rc:
        _check(rc, "spec_cache_read")
    return k, v


@dataclass
class CacheAttention:
    out: torch.Tensor               # [B, n, q_heads, D] bf16
    lse: Optional[torch.Tensor]     # [B, n, q_heads] fp32
    ws: Optional[torch.Tensor]


_attend_ws: dict = {}


def _attend_workspace(nbytes: int, device: torch.device, handle: int, stream) -> torch.Tensor:
    """cache_attend's workspace, one per device and stream: its control words
    start at zero and every call leaves them so."""
    key = (device.index, handle)
    buf = _attend_ws.get(key)
    if buf is None or buf.numel() < nbytes:
        if torch.cuda.is_current_stream_capturing():
            raise SpecError("cache_attend needs its workspace before a stream capture: call it once before, or pass ws "
                            "(zeroed)")
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(device)):
            buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        _attend_ws[key] = buf
    return buf


def cache_attend(q, pool, page_table, ctx_len, num_rows=None, *, anc_mask=None, depth=None, window: int = 0,
                 sinks: int = 0, scale: Optional[float] = None, out=None, lse=None, want_lse: bool = False,
                 status=None, ws: Optional[torch.Tensor] = None, stream=None) -> CacheAttention:
    """Attention of drafted rows q [B, n, q_heads, D] bf16 over the cache.

    Request b's cache holds ctx_len[b] context positions and behind them its
    num_rows[b] (default n) drafted rows, written by cache_append.  A row sees
    the context and, of the drafted rows, those in its anc_mask (int64
    [B, n, ceil(n/64)], as tree_build writes it), or without a mask the rows up
    to itself.  Its position is ctx_len[b] + depth[b, i] (default i); with
    window > 0 it sees only keys of position p with p_i - p < window or
    p < sinks.  scale defaults to 1/sqrt(D).  Rows that see nothing are 0, their
    lse -inf; lse (natural log) is written when given or asked for.  A ws of
    one's own starts zeroed and serves one stream."""
    L = _lib()
    if not (isinstance(q, torch.Tensor) and q.dtype is _bf16 and q.dim() == 4 and (q.is_cuda or q.is_pinned())):
        _cuda(q, "q", _bf16)
        raise SpecError("q must be [B, n, q_heads, D] with unit element stride")
    shape = q.shape
    B, n, hq, D = shape
    qb, qr, qh, q1 = q.stride()
    if q1 != 1:
        raise SpecError("q must be [B, n, q_heads, D] with unit element stride")
    page, H, pages = _pool(pool, 3, D)
    _, M, ts, tp = _table(page_table, B)
    dev = pool.device
    if anc_mask is not None:
        _cuda(anc_mask, "anc_mask", torch.int64)
        if anc_mask.shape != (B, n, (n + 63) // 64) or not anc_mask.is_contiguous():
            raise SpecError("anc_mask must be a contiguous [B, n, ceil(n/64)] int64 tensor")
    if out is None:
        out = torch.empty(shape, dtype=_bf16, device=dev)
    elif _cuda(out, "out", _bf16).shape != shape or not out.is_contiguous():
        raise SpecError("out must be a contiguous tensor of q's shape, bf16")
    if lse is not None:
        if _cuda(lse, "lse", torch.float32).shape != shape[:3] or not lse.is_contiguous():
            raise SpecError("lse must be a contiguous [B, n, q_heads] float32 tensor")
    elif want_lse:
        lse = torch.empty(shape[:3], dtype=torch.float32, device=dev)
    handle = _handle(stream, dev)
    if ws is None:
        need = L.spec_cache_attend_workspace_size(B, n, hq, H, D)
        ws = _attend_workspace(need, dev, handle, stream) if need else None
    ps, hs, _ = pool.stride()
    rc = L.spec_cache_attend(q.data_ptr(), qb, qr, qh, pool.data_ptr(), ps, hs, pages, tp, ts, M,
                             _ints(ctx_len, "ctx_len", B), _opt(num_rows, "num_rows", B),
                             None if anc_mask is None else anc_mask.data_ptr(), _opt(depth, "depth", B, n),
                             window, sinks, 1.0 / math.sqrt(D) if scale is None else scale,
                             B, n, hq, H, D, page, out.data_ptr(), None if lse is None else lse.data_ptr(),
                             _opt(status, "status", B), None if ws is None else ws.data_ptr(),
                             0 if ws is None else ws.numel(), handle)
    if rc:
        _check(rc, "spec_cache_attend")
    return CacheAttention(out, lse, ws)


def cache_compact(pool, page_table, ctx_len, path_nodes, num_accepted, head_dim: int, *, status=None,
                  stream=None) -> None:
    """Keep an accepted path's rows: position ctx_len[b] + path_nodes[b, j]
    moves to ctx_len[b] + j, j = 0..num_accepted[b], in every layer of pool
    [layers, pages, kv_heads, block].  In place."""
    page, H, pages = _pool(pool, 4, head_dim)
    B, M, ts, tp = _table(page_table)
    if not isinstance(path_nodes, torch.Tensor) or path_nodes.dim() != 2:
        raise SpecError("path_nodes must be a contiguous [B, path_width] int32 tensor")
    width = path_nodes.shape[1]
    ls, ps, hs, _ = pool.stride()
    rc = _lib().spec_cache_compact(pool.data_ptr(), pool.shape[0], ls, ps, hs, pages, tp, ts, M,
                                   _ints(ctx_len, "ctx_len", B), _ints(path_nodes, "path_nodes", B, width), width,
                                   _ints(num_accepted, "num_accepted", B), B, H, head_dim, page,
                                   _opt(status, "status", B), _handle(stream, pool.device))
    if rc:
        _check(rc, "spec_cache_compact")


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
@dataclass
class PageState:
    """Which request holds which page of a pool (int32 CUDA tensors)."""
    page_table: torch.Tensor   # [R, M], -1 past num_held
    num_held: torch.Tensor     # [R]
    ref: torch.Tensor          # [num_pages]: requests that hold the page
    free_list: torch.Tensor    # [num_pages]: a stack
    num_free: torch.Tensor     # [1]


def page_state(requests: int, max_pages: int, num_pages: int, device) -> PageState:
    """A state in which every page is free; the stack's top is page 0."""
    i32 = dict(dtype=torch.int32, device=device)
    return PageState(torch.full((requests, max_pages), -1, **i32), torch.zeros(requests, **i32),
                     torch.zeros(num_pages, **i32), torch.arange(num_pages - 1, -1, -1, **i32),
                     torch.full((1,), num_pages, **i32))


def _pages(s: PageState):
    R, M, ts, tp = _table(s.page_table)
    n = s.ref.shape[0]
    return R, (tp, ts, M, _ints(s.num_held, "num_held", R), _ints(s.ref, "ref", n),
               _ints(s.free_list, "free_list", n), _ints(s.num_free, "num_free", 1), n)


def cache_reserve(pages: PageState, length, page_size: int, *, status=None, stream=None) -> None:
    """Give each request the pages it lacks for length[r] tokens, off the top
    of the stack, requests in order; one that they do not suffice for gets none
    (ST_NO_PAGE)."""
    R, args = _pages(pages)
    rc = _lib().spec_cache_reserve(*args, _ints(length, "length", R), R, page_size, _opt(status, "status", R),
                                   _handle(stream, pages.ref.device))
    if rc:
        _check(rc, "spec_cache_reserve")


def cache_release(pages: PageState, length, page_size: int, *, status=None, stream=None) -> None:
    """Each request keeps the pages of length[r] tokens (0: none); pages that
    nothing holds any more are free."""
    R, args = _pages(pages)
    rc = _lib().spec_cache_release(*args, _ints(length, "length", R), R, page_size, _opt(status, "status", R),
                                   _handle(stream, pages.ref.device))
    if rc:
        _check(rc, "spec_cache_release")


def cache_fork(pool, pages: PageState, src, dst, length, head_dim: int, *, new_page=None, status=None, stream=None):
    """Request dst[f] (holding nothing) becomes a copy of request src[f] at
    length[src[f]] tokens: full pages are shared, the last partial one is copied
    in every layer of pool [layers, pages, kv_heads, block].  Returns new_page
    [F]: the page of its own that each got, or -1."""
    page, H, count = _pool(pool, 4, head_dim)
    R, args = _pages(pages)
    if args[-1] != count:
        raise SpecError(f"the state has {args[-1]} pages, the pool {count}")
    F = src.shape[0]
    if new_page is None:
        new_page = torch.empty(F, dtype=_i32, device=pool.device)
    ls, ps, hs, _ = pool.stride()
    rc = _lib().spec_cache_fork(pool.data_ptr(), pool.shape[0], ls, ps, hs, *args, _ints(src, "src", F),
                                _ints(dst, "dst", F), _ints(length, "length", R), R, F, H, head_dim, page,
                                _ints(new_page, "new_page", F), _opt(status, "status", F),
                                _handle(stream, pool.device))
    if rc:
        _check(rc, "spec_cache_fork")
    return new_page
