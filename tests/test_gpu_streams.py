"""On whose memory the verification calls work when a stream is given."""
import pytest
import torch

import speculative_decoding_draft_sampling_gb300 as sv

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def stream_of(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def outputs(stream):
    """Every call's outputs, by name, on small inputs."""
    g = torch.Generator(device=DEV).manual_seed(1)
    B, K, V = 3, 4, 1000
    rand = lambda *shape: torch.rand(shape, device=DEV, generator=g)
    logits, q, u = 4 * rand(B, K + 1, V), torch.softmax(3 * rand(B, K, V), -1), rand(B, K + 1)
    draft = torch.randint(0, V, (B, K), device=DEV, dtype=torch.int32, generator=g)
    conf, state = rand(B, K), sv.eagle_state(B, 200, DEV)
    front, num = torch.zeros((B, 1), dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
    uniforms = rand(B, K + 1)
    torch.cuda.synchronize()
    kw = {} if stream is None else dict(stream=stream)
    res = {}
    r = sv.verify_chain(logits, q, draft, u, 1.0, 50, diag=True, **kw)
    res.update(chain=(r.tokens, r.num_accepted, r.status, r.diag))
    r = sv.verify_greedy(logits, draft, **kw)
    res.update(greedy=(r.tokens, r.num_accepted, r.status))
    t = sv.tree_build(q, 12, **kw)
    res.update(tree=(t.token, t.parent, t.depth, t.score, t.anc_mask, t.num_nodes, t.status))
    if stream is not None:
        stream.synchronize()
    rows = 4 * rand(B, 12, V)
    torch.cuda.synchronize()
    r = sv.verify_tree(rows, t.token, t.parent, t.num_nodes, K, **kw)
    res.update(walk=(r.tokens, r.path_nodes, r.num_accepted, r.status))
    r = sv.verify_tree_sample(rows, t.token, t.parent, t.num_nodes, uniforms, K, 1.0, **kw)
    res.update(sampled=(r.tokens, r.path_nodes, r.num_accepted, r.status))
    r = sv.adaptive_len(conf, 1.0, 0.15, **kw)
    res.update(length=(r.k, r.surv, r.exp_adv, r.l_row_off, r.q_row_off))
    f, n, status = sv.eagle_expand(q[:, :1], state, front, num, 4, 4, **kw)
    res.update(expand=(f, n, status))
    torch.cuda.synchronize()
    return res


def test_outputs_belong_to_the_given_stream():
    side = torch.cuda.Stream()
    want, got = outputs(None), outputs(side)
    for name, tensors in got.items():
        assert all(stream_of(t) == side.cuda_stream for t in tensors), name
        assert torch.equal(tensors[0], want[name][0]), name      # tokens, lengths, nodes


@pytest.fixture
def fresh_workspaces(monkeypatch):
    monkeypatch.setattr(sv, "_ws_cache", {})


def test_outgrown_workspaces_are_nobody_elses(fresh_workspaces):
    at, size = sv.workspace(5 << 20, DEV).data_ptr(), 5 << 20
    assert sv.workspace(6 << 20, DEV).numel() >= 10 << 20
    others = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (5 << 20, 1 << 20, 4 << 20, 5 << 20, 2 << 20)]
    assert all(x.data_ptr() + x.numel() <= at or x.data_ptr() >= at + size for x in others)


def test_graph_keeps_its_workspace(fresh_workspaces):
    """A captured call, then one that needs more, then others that take what is free."""
    g = torch.Generator(device=DEV).manual_seed(2)
    logits = torch.rand((2, 5, 4000), device=DEV, generator=g)
    draft = torch.randint(0, 4000, (2, 4), device=DEV, dtype=torch.int32, generator=g)
    r = sv.verify_greedy(logits, draft)
    want = (r.tokens.clone(), r.num_accepted.clone())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sv.verify_greedy(logits, draft, out=sv.GreedyResult(r.tokens, r.num_accepted, r.status, None))
    sv.workspace(64 << 20, DEV)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in (1 << 12, 1 << 16, 1 << 20, 2 << 20) for _ in range(8)]
    for _ in range(3):
        r.tokens.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.tokens, want[0]) and torch.equal(r.num_accepted, want[1])
    assert all(bool((x == 255).all()) for x in junk)
