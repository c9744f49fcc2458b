"""When the cache calls' binding is built again, and where its functions are found."""
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
import speculative_decoding_draft_sampling_gb300 as sv
from speculative_decoding_draft_sampling_gb300 import _build


def test_binding_of_another_pytorch_is_stale(monkeypatch):
    sv.build()
    assert _build.binding_up_to_date()
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    assert not _build.binding_up_to_date()


@pytest.mark.parametrize("first", ["from speculative_decoding_draft_sampling_gb300.cache import cache_attend as call",
                                   "import speculative_decoding_draft_sampling_gb300 as sv; call = sv.cache_attend",
                                   "import speculative_decoding_draft_sampling_gb300 as sv; call = sv.cache.cache_attend"])
def test_calls_are_found_in_the_package_and_its_module(first):
    """Whichever is asked first, in a process of its own."""
    sv.build()
    code = first + """
import speculative_decoding_draft_sampling_gb300 as sv
assert call is sv.cache_attend is sv.cache.cache_attend and sv.cache_fork is sv.cache.cache_fork
assert "cache_append" in vars(sv) and not hasattr(sv, "cache_nothing") and not hasattr(sv.cache, "cache_nothing")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
