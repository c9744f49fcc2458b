"""The paged 4-bit KV cache that a verification pass reads, writes and cuts
back (C ABI: include/spec_cache.h).

A pool is a uint8 CUDA tensor [pages, kv_heads, block] for one layer, or
[layers, pages, kv_heads, block] where a call works on all layers
(cache_compact, cache_fork); block = cache_block_bytes(head_dim, page_size).
A block holds one page of P tokens of one kv head:

    K codes [P][D/2] | K scales bf16 [P][D/32] | V codes [P][D/2] | V scales bf16 [P][D/32]

page_table [B, M] int32 names the pages of each request in order (-1: none).
`status` arguments are optional int32 [B] tensors; bits are OR-ed in.  A call
runs on the current stream, or on the one given as `stream`, and what it
allocates belongs to that stream, as under `torch.cuda.stream(stream)`.

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
import importlib.machinery
import importlib.util
import os
import sys
from dataclasses import dataclass
from typing import Optional

import torch

from . import LIB_PATH, SpecError, _load

ST_BAD_PAGE, ST_NO_PAGE, ST_SHARED_PAGE = 128, 256, 512

BINDING_PATH = os.path.join(os.path.dirname(LIB_PATH), "_spec_torch.so")


@dataclass
class CacheAttention:
    out: torch.Tensor               # [B, n, q_heads, D] bf16
    lse: Optional[torch.Tensor]     # [B, n, q_heads] fp32
    ws: Optional[torch.Tensor]


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


_bound = None


def _lib():
    """The C library with the cache calls' signatures."""
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


def _binding():
    """The binding (csrc/spec_torch.cpp), set up with the library's functions."""
    lib = _lib()
    if not os.path.exists(BINDING_PATH):
        raise SpecError(f"{BINDING_PATH} is missing: build it with speculative_decoding_draft_sampling_gb300.build() first")
    loader = importlib.machinery.ExtensionFileLoader("_spec_torch", BINDING_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_spec_torch", BINDING_PATH,
                                                                                    loader=loader))
    loader.exec_module(module)
    names = ("spec_last_error", "spec_cache_append", "spec_cache_read", "spec_cache_attend_workspace_size",
             "spec_cache_attend", "spec_cache_compact", "spec_cache_reserve", "spec_cache_release", "spec_cache_fork")
    module.setup(SpecError, CacheAttention, *[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names])
    return module


def cache_block_bytes(head_dim: int, page_size: int) -> int:
    """Bytes of one page of one kv head."""
    n = int(_lib().spec_cache_block_bytes(int(head_dim), int(page_size)))
    if n == 0:
        raise SpecError(f"unsupported cache shape: head_dim is 64 or 128 and page_size 16, 32 or 64 "
                        f"(got {head_dim} and {page_size})")
    return n


CALLS = ("cache_append", "cache_read", "cache_attend", "cache_compact", "cache_reserve", "cache_release", "cache_fork")


def __getattr__(name: str):
    """The first use of a call puts the binding's functions here and into the package."""
    if name in CALLS:
        module = _binding()
        for space in (globals(), vars(sys.modules[__package__])):
            space.update({call: getattr(module, call) for call in CALLS})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
