"""CPU checks of what the cache side's binding hands to the C entry points.  The library is out of
reach: a recorder stands in its place."""
import pytest
import torch

import paged_kv_block_gb300 as pkb
from paged_kv_block_gb300 import build as B
from paged_kv_block_gb300 import cache as K

A16 = 0x7F0000100000


class Recorder:
    """Keeps name, parameters and other arguments of every call; workspaces are 64 bytes."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda n: 64

        def call(params, *rest):
            self.calls.append((name, params._obj, rest))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    """The calls of the binding on host tensors (their device index is -1)."""
    r = Recorder()
    monkeypatch.setattr(K, "_device", lambda: -1)
    monkeypatch.setattr(K, "_stream", lambda stream, dev: 0)
    monkeypatch.setattr(K, "_call", r)
    return r.calls


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


# ---- status words -----------------------------------------------------------------------------

def test_the_status_word_reaches_the_call(calls):
    state, word = (i32(3, 2), i32(3), i32(4)), i32(1)
    pools = pkb.cache_pools([torch.zeros(4, 2, 2, 8, 8, dtype=torch.bfloat16)])
    for call in (lambda **kw: pkb.extend_cache_rows(i32(2), i32(2), *state, 8, **kw),
                 lambda **kw: pkb.fork_cache_rows(pools, i32(2), i32(2), *state, **kw),
                 lambda **kw: pkb.compact_cache(pools, *state, **kw)):
        for other in (None, word, i32(1), None):
            call(status=other)
            p = calls[-1][1]
            assert (p.rows, p.max_pages_per_request, p.page_size, p.num_pages) == (3, 2, 8, 4)
            assert p.status_dev == (None if other is None else other.data_ptr())
        for bad in (i32(0), i32(4)[::2], torch.zeros(1, dtype=torch.int64)):
            with pytest.raises(ValueError):
                call(status=bad)


def test_the_c_calls_refuse_a_status_word_off_its_alignment():
    import ctypes as C
    B.build()
    lib = pkb.lib()
    p = K.CacheParams(rows=4, max_pages_per_request=8, page_size=16, num_pages=32,
                      status_dev=A16 + 2)
    ptrs = (C.c_void_p * 1)(A16)
    s = K.CachePoolsStruct(num_layers=1, num_pages=32, num_kv_heads=2, page_size=16, head_dim=64,
                           combined_cache=1, pools_host=ptrs)
    bad, big, a = pkb.ERR_INVALID_ARGUMENT, 1 << 30, A16
    assert lib.paged_cache_extend_run(C.byref(p), a, a, 1, a, a, a, a, big, None) == bad
    assert lib.paged_cache_fork_run(C.byref(p), C.byref(s), a, a, 1, a, a, a, a, big, None) == bad
    assert lib.paged_cache_compact_run(C.byref(p), C.byref(s), a, a, a, a, a, a, a, big,
                                       None) == bad


# ---- parameters are taken by value --------------------------------------------------------------

def test_a_factor_that_changes_in_place_is_read_at_every_call(calls):
    q, table = torch.zeros(3, 2, 8), torch.zeros(4, dtype=torch.int64)
    cache, m = torch.zeros(4, 2, 2, 8, 8, dtype=torch.bfloat16), torch.tensor(1.0)
    for call in (lambda: pkb.rotary_embedding(q, i32(3), table, attention_factor=m),
                 lambda: pkb.append_paged_kv_cache(q, q, cache, i32(3), freqs=table,
                                                   block_tables=i32(3, 2), attention_factor=m)):
        for value in (1.0, 2.0, 0.5, 1.0):
            m.fill_(value)
            call()
            assert calls[-1][1].attention_factor == value
    # zeros of both signs are equal keys: a call gets the same one whatever came before it
    for value in (0.0, -0.0, 0.0):
        pkb.rotary_embedding(q, i32(3), table, attention_factor=value)
        assert str(calls[-1][1].attention_factor) == "0.0"


def test_a_page_size_that_changes_in_place_is_read_at_every_call(calls):
    state, size = (i32(3, 2), i32(3), i32(4)), torch.tensor(8)
    for call in (lambda: pkb.free_cache_rows(i32(2), *state, size),
                 lambda: pkb.extend_cache_rows(i32(2), i32(2), *state, size)):
        for value in (8, 16, 8):
            size.fill_(value)
            call()
            assert calls[-1][1].page_size == value
    for bad in (8.0, "8"):                            # also after a call with 8
        with pytest.raises(TypeError):
            pkb.free_cache_rows(i32(2), *state, bad)
