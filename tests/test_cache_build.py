"""When the cache calls' binding is built again."""
import torch

import speculative_decoding_draft_sampling_gb300 as sv
from speculative_decoding_draft_sampling_gb300 import _build


def test_binding_of_another_pytorch_is_stale(monkeypatch):
    sv.build()
    assert _build.binding_up_to_date()
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    assert not _build.binding_up_to_date()
