"""The cache calls together, as examples/paged_decode.py uses them: decoding by
draft trees with forks commits what decoding a token at a time commits."""
import os
import sys

import pytest

from conftest import ROOT

import speculative_decoding_draft_sampling_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("budget,depth", [(24, 5), (90, 6)])
def test_tree_decoding_is_greedy_decoding(budget, depth):
    sv.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import paged_decode
    got, want, kept, problems = paged_decode.run(budget=budget, depth=depth)
    half = len(got) // 2
    assert problems == 0
    for b in range(half):
        assert len(got[b]) >= len(kept)                  # a token a step at least
        assert got[b] == want[b][:len(got[b])], b
    for b in range(half):                                # the forked half goes on alike
        n = min(len(got[half + b]), len(want[b]))
        assert got[half + b][:n] == want[b][:n], b
    assert sum(kept) > half * len(kept)                  # some drafts were accepted
