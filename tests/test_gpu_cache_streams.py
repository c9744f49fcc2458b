"""The cache calls in captured graphs and on given streams: whose memory a call
works in."""
import gc

import pytest
import torch

import speculative_decoding_draft_sampling_gb300 as sv
from test_gpu_cache import DEV, filled, ints, randn

pytestmark = pytest.mark.gpu

D, P, H, CTX = 128, 64, 2, [2000, 300, 700]


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


@pytest.fixture(scope="module")
def cache():
    """A pool, its table, and the requests' context lengths."""
    pool, table, _, _ = filled([c + 64 for c in CTX], H, P, D)
    return pool, table, ints(CTX)


class Step:
    """n rows a request whose attention is captured without a workspace of the caller's."""

    def __init__(self, cache, n, stream, seed=0):
        pool, table, ctx = cache
        self.q = randn(len(CTX), n, 4 * H, D, seed=seed + n)
        self.want = sv.cache_attend(self.q, pool, table, ctx, want_lse=True)
        self.want = (self.want.out.clone(), self.want.lse.clone())
        self.out, self.lse = torch.zeros_like(self.want[0]), torch.zeros_like(self.want[1])
        self.graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(self.graph, stream=stream):
            sv.cache_attend(self.q, pool, table, ctx, out=self.out, lse=self.lse)
        torch.cuda.synchronize()

    def check(self):
        assert torch.equal(self.out, self.want[0]) and torch.equal(self.lse, self.want[1])
        self.out.zero_()
        self.lse.zero_()


@pytest.mark.parametrize("warm", [False, True])
def test_graph_keeps_its_workspace(cache, warm):
    """A small step is captured, then larger calls need more on the same stream, and others take what was freed."""
    pool, table, ctx = cache
    side = torch.cuda.Stream()
    if warm:
        with torch.cuda.stream(side):
            sv.cache_attend(randn(len(CTX), 1, 4 * H, D), pool, table, ctx)
    step = Step(cache, 1, side)
    junk = []
    with torch.cuda.stream(side):
        for n in (3, 8, 12, 64):
            sv.cache_attend(randn(len(CTX), n, 4 * H, D), pool, table, ctx)
            junk += [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for size in (1 << 20, 7 << 20, 12 << 20)]
    torch.cuda.synchronize()
    for _ in range(3):
        step.graph.replay()
        torch.cuda.synchronize()
        step.check()
    assert all(bool((x == 255).all()) for x in junk)


@pytest.mark.parametrize("n,other", [(1, 4), (40, 40)])
def test_graphs_of_one_stream_run_side_by_side(cache, n, other):
    side, streams = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    steps = [Step(cache, n, side), Step(cache, other, side, seed=5)]
    for _ in range(20):
        for step, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                step.graph.replay()
    torch.cuda.synchronize()
    for step in steps:
        step.check()


def test_calls_of_one_capture_share_a_workspace(cache):
    pool, table, ctx = cache
    q = randn(len(CTX), 2, 4 * H, D)
    want = sv.cache_attend(q, pool, table, ctx).out.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        a = sv.cache_attend(q, pool, table, ctx)
        b = sv.cache_attend(q, pool, table, ctx)
        larger = sv.cache_attend(torch.cat([q] * 8, 1), pool, table, ctx)
        c = sv.cache_attend(q, pool, table, ctx)
    assert a.ws.data_ptr() == b.ws.data_ptr() and larger.ws.data_ptr() == c.ws.data_ptr()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        for r in (a, b, c):
            assert torch.equal(r.out, want)
            r.out.zero_()


def test_workspaces_of_dropped_graphs_are_freed(cache):
    side = torch.cuda.Stream()
    size, at = None, {}
    for i in range(25):
        step = Step(cache, 40, side)
        step.graph.replay()
        torch.cuda.synchronize()
        step.check()
        del step
        gc.collect()
        torch.cuda.synchronize()
        at[i] = torch.cuda.memory_allocated()
    size = sv.cache._lib().spec_cache_attend_workspace_size(len(CTX), 40, 4 * H, H, D)
    assert at[24] - at[4] < 5 * size, (at, size)


def stream_of(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def test_what_a_call_allocates_belongs_to_its_stream(cache):
    pool, table, ctx = cache
    side = torch.cuda.Stream()
    q, pages = randn(len(CTX), 2, 4 * H, D), sv.page_state(2, 4, pool.shape[0], DEV)
    sv.cache_reserve(pages, ints([70, 0]), P)
    own = torch.zeros_like(pool)[None]                   # (fork writes into it)
    args = [ints([0] * len(CTX)), ints([0]), ints([1]), ints([70, 0])]
    torch.cuda.synchronize()
    k, v = sv.cache_read(pool, table, args[0], 200, D, stream=side)
    a = sv.cache_attend(q, pool, table, ctx, want_lse=True, stream=side)
    new = sv.cache_fork(own, pages, *args[1:], D, stream=side)
    side.synchronize()
    for t in (k, v, a.out, a.lse, a.ws, new):
        assert stream_of(t) == side.cuda_stream
    assert torch.equal(a.out, sv.cache_attend(q, pool, table, ctx).out)


def test_given_stream_of_a_capture(cache):
    """A stream that joined the capture is given; the current stream's calls are captured too."""
    pool, table, ctx = cache
    q = randn(len(CTX), 2, 4 * H, D)
    want = sv.cache_attend(q, pool, table, ctx).out.clone()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        a = sv.cache_attend(q, pool, table, ctx, stream=side)
        b = sv.cache_attend(q, pool, table, ctx)
        torch.cuda.current_stream().wait_stream(side)
    assert a.ws.data_ptr() != b.ws.data_ptr()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want) and torch.equal(b.out, want)
        a.out.zero_()
        b.out.zero_()
