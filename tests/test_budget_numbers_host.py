"""CPU checks of numbers that the C calls' 32-bit ints cannot hold: refused, not cut off."""
import pytest
import torch

import paged_kv_block_gb300 as pkb
from tests.test_cache_binding import calls, i32  # noqa: F401

FAR = 1 << 32


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def wide(*shape):
    """A tensor of that shape that holds next to nothing."""
    return torch.zeros(1).expand(shape)


@pytest.mark.parametrize("far", [FAR + 1, 1 << 31, -FAR])
def test_numbers_out_of_range_are_refused(calls, far):  # noqa: F811
    state = i32(5, 4), i32(5), i32(9)
    pools = pkb.cache_pools([bf16(9, 2, 2, 16, 8)])
    w = torch.zeros(5, 2, 40)
    cases = [
        lambda: pkb.accumulate_attention_weights(
            bf16(3, 8, 128), torch.zeros(3, 8), bf16(9, 2, 2, 16, 128), i32(3),
            torch.zeros(3, 2, 40), block_tables=i32(3, 5), last_queries=far),
        lambda: pkb.select_cache_tokens(i32(4), w, i32(5), 7, sink=far),
        lambda: pkb.select_cache_tokens(i32(4), w, i32(5), 7, recent=far),
        lambda: pkb.evict_cache_rows(pools, i32(4), i32(4, 2, 7), *state, sink=far),
        lambda: pkb.batch_decode_with_shared_prefix(
            bf16(4, 8, 128), bf16(9, 2, 2, 16, 128), None, i32(5), i32(20), i32(4), far, i32(3),
            i32(2)),
        lambda: pkb.shared_prefix_workspace_size(bf16(4, 8, 128), bf16(9, 2, 2, 16, 128), far, 2),
        lambda: pkb.shared_prefix_workspace_size(bf16(4, 8, 128), bf16(9, 2, 2, 16, 128), 99, far),
        lambda: pkb.evict_cache_workspace_size(far, 20, 16),
        lambda: pkb.evict_cache_workspace_size(2, far, 16),
        lambda: pkb.evict_cache_workspace_size(2, 20, far),
    ]
    for case in cases:
        with pytest.raises(ValueError, match="32 bits"):
            case()
    assert not calls


def test_weights_wider_than_32_bits_are_refused(calls, monkeypatch):  # noqa: F811
    """(Their address and layout are not looked at here.)"""
    monkeypatch.setattr(pkb.eviction, "_plain", lambda *a: 4096)
    monkeypatch.setattr(pkb.eviction, "evict_cache_workspace_size", lambda *a: 64)
    pools = pkb.cache_pools([bf16(9, 2, 2, 16, 8)])
    w = wide(3, 2, FAR + 40)
    with pytest.raises(ValueError, match="32 bits"):
        pkb.accumulate_attention_weights(bf16(3, 8, 128), torch.zeros(3, 8),
                                         bf16(9, 2, 2, 16, 128), i32(3), w,
                                         block_tables=i32(3, 5))
    with pytest.raises(ValueError, match="32 bits"):
        pkb.evict_cache_rows(pools, i32(2), i32(2, 2, 7), i32(3, 4), i32(3), i32(9), weights=w)
    assert not calls
