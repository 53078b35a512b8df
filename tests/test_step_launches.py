"""The number of kernels that a step launches, as the host counts them."""
from types import SimpleNamespace

import pytest

from speculative_decoding_verify_paged_gb300 import HeadTransform, ScoreMod
from speculative_decoding_verify_paged_gb300 import _lib as L
from speculative_decoding_verify_paged_gb300 import step as S


@pytest.mark.parametrize("transform", [None, HeadTransform()])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("mod", [None, ScoreMod(window=5)])
@pytest.mark.parametrize("tree", [False, True])
def test_launches(monkeypatch, transform, shared, mod, tree):
    monkeypatch.setattr(L, "spec_verify_attn_workspace_bytes", lambda *a: 0)
    monkeypatch.setattr(L, "spec_verify_attn_scored_workspace_bytes", lambda *a: 256)
    d = SimpleNamespace(transform=transform, mod=mod, mask_kind=L.SV_MASK_TREE if tree else L.SV_MASK_CAUSAL, num_q_heads=8, total_q=4, max_q=2)
    kv = SimpleNamespace(ref_count=object() if shared else None)
    want = 2 + (1 if transform is not None and shared else 0) + (1 if mod is None else 2) + 2 + (2 if tree else 1)
    assert S.launches_per_step(d, 64, kv) == want
