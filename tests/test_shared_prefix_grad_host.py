"""CPU check: decode behind shared prefixes writes no tensor that autograd follows."""
import pytest
import torch

import paged_kv_block_gb300 as pkb
from paged_kv_block_gb300 import cache as K
from tests.test_cache_binding import i32


def test_outputs_that_require_a_gradient_are_refused(monkeypatch):
    seen = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *a: seen.append(a) or 0
    monkeypatch.setattr(K, "_device", lambda: -1)
    monkeypatch.setattr(K, "_stream", lambda stream, dev: 0)
    monkeypatch.setattr(K, "_call", Recorder())
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    args = (q, torch.zeros(9, 2, 2, 16, 128, dtype=torch.bfloat16),
            torch.zeros(64, dtype=torch.uint8), i32(5), i32(20), i32(4), 99, i32(3), i32(2))
    for bad in (dict(out=torch.zeros_like(q).requires_grad_()),
                dict(lse=torch.zeros(4, 8, requires_grad=True))):
        with pytest.raises(ValueError, match="must not require a gradient"):
            pkb.batch_decode_with_shared_prefix(*args, **bad)
        assert not seen
        with torch.no_grad():
            pkb.batch_decode_with_shared_prefix(*args, **bad)
        assert len(seen) == 1
        seen.clear()
