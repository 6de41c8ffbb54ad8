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


# ---- autograd ----------------------------------------------------------------------------------

def test_rotation_is_known_to_autograd(calls):
    table, pos = torch.zeros(4, dtype=torch.int64), i32(3)
    q, k = torch.zeros(3, 4, 8, requires_grad=True), torch.zeros(3, 2, 8, requires_grad=True)
    m = torch.tensor(2.0)

    def shapes(p):
        return p.num_tokens, p.num_qo_heads, p.num_kv_heads, p.inverse, p.attention_factor
    qo, ko = pkb.rotary_embedding(q, pos, table, k=k, attention_factor=m)
    assert qo.requires_grad and ko.requires_grad
    m.fill_(3.0)                                      # the forward call's factor counts
    torch.autograd.backward([qo, ko], [torch.ones_like(qo), torch.ones_like(ko)])
    assert [shapes(c[1]) for c in calls] == [(3, 4, 2, 0, 2.0), (3, 4, 2, 1, 2.0)]
    assert q.grad.shape == q.shape and k.grad.shape == k.shape
    # what nobody asks for is not computed
    calls.clear()
    qo, ko = pkb.rotary_embedding(q.detach(), pos, table, k=k, inverse=True)
    assert not qo.requires_grad or qo.grad_fn is ko.grad_fn
    torch.autograd.grad(ko, k, torch.ones_like(ko))
    assert [shapes(c[1]) for c in calls] == [(3, 4, 2, 1, 1.0), (3, 2, 0, 0, 1.0)]
    calls.clear()
    qo, _ = pkb.rotary_embedding(q, pos, table, k=k)
    qo.sum().backward()                              # a gradient of step 0: one value for all
    assert [shapes(c[1]) for c in calls] == [(3, 4, 2, 0, 1.0), (3, 4, 0, 1, 1.0)]
    assert (calls[1][1].q_token_stride, calls[1][1].q_head_stride) == (32, 8)
    with torch.no_grad():
        assert not pkb.rotary_embedding(q, pos, table).requires_grad


def test_outputs_that_autograd_cannot_follow_are_refused(calls):
    table, pos = torch.zeros(4, dtype=torch.int64), i32(3)
    q, k = torch.zeros(3, 4, 8), torch.zeros(3, 2, 8)
    leaf_q, leaf_k = (t.clone().requires_grad_() for t in (q, k))
    for kw in (dict(q=leaf_q, q_out=q), dict(q=leaf_q, q_out=leaf_q), dict(q=q, q_out=leaf_q),
               dict(q=q, k=leaf_k, k_out=k), dict(q=q, k=k, k_out=leaf_k),
               dict(q=q, k=leaf_k, q_out=q)):
        with pytest.raises(ValueError):
            pkb.rotary_embedding(positions=pos, freqs=table, **kw)
    assert not calls
    with torch.no_grad():
        pkb.rotary_embedding(leaf_q, pos, table, q_out=leaf_q)
    assert len(calls) == 1


def test_given_outputs_count_as_changed(calls):
    table, pos = torch.zeros(4, dtype=torch.int64), i32(3)
    q, k = torch.zeros(3, 4, 8), torch.zeros(3, 2, 8)
    w = torch.ones(8, requires_grad=True)
    y = (q * w).sum()                                # saves q
    seen = q._version, k._version
    pkb.rotary_embedding(q, pos, table, k=k, q_out=q, k_out=k)
    assert q._version > seen[0] and k._version > seen[1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    seen, cache = q._version, torch.zeros(4, 2, 2, 8, 8, dtype=torch.bfloat16)
    out = torch.zeros(3, 4, 8, dtype=torch.bfloat16)
    pkb.append_paged_kv_cache(k, k, cache, pos, q=q, q_out=out, block_tables=i32(3, 2))
    assert out._version > 0 and q._version == seen
    with torch.inference_mode():                     # such tensors have no version
        t = torch.zeros(3, 4, 8)
        pkb.rotary_embedding(t, pos, table, q_out=t)


def test_positions_that_change_before_the_gradient_are_noticed(calls):
    q, pos = torch.zeros(3, 4, 8, requires_grad=True), i32(3)
    out = pkb.rotary_embedding(q, pos, torch.zeros(4, dtype=torch.int64))
    pos.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


# ---- a batch of no request --------------------------------------------------------------------

def test_rows_of_no_request_are_padding():
    """A packed batch without requests: its rows are padding, and empty arrays have no address."""
    import ctypes as C
    B.build()
    lib = pkb.lib()
    p = K.AppendParams(batch=0, total_q=5, num_qo_heads=4, num_kv_heads=2, head_dim=64,
                       page_size=16, num_pages=10, combined_cache=1, max_pages_per_request=4,
                       rotary_dim=64, attention_factor=1.0)

    def run(p, lens, pages, **kw):
        a = dict(q=A16, k=A16, v=A16, table=A16, out=A16, kc=A16)
        a.update(kw)
        return lib.paged_append_run(C.byref(p), a["q"], a["k"], a["v"], A16, None, pages, lens,
                                    a["table"], a["out"], a["kc"], None, None, None)
    assert run(p, None, None) == 0
    for bad in (dict(k=None), dict(kc=None), dict(out=A16 + 8), dict(q=None), dict(table=None)):
        assert run(p, None, None, **bad) == pkb.ERR_INVALID_ARGUMENT, bad
    p.batch = 1                                      # a request's length and pages are needed
    assert run(p, None, A16) == run(p, A16, None) == pkb.ERR_INVALID_ARGUMENT
