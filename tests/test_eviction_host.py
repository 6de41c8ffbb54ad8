"""CPU checks of the calls that keep rows within a budget: what the binding hands over and refuses,
and what the C entry points refuse before anything is enqueued."""
import ctypes as C

import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import cache as OC
from oracle import eviction as O
from paged_kv_block_gb300 import build as B
from paged_kv_block_gb300 import cache as K
from paged_kv_block_gb300 import eviction as E
from tests.test_cache_binding import calls, i32  # noqa: F401

A16 = 0x7F0000100000
BAD = pkb.ERR_INVALID_ARGUMENT


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pkb.lib()


# ---- the oracle ---------------------------------------------------------------------------------

def test_select_oracle_by_hand():
    w = np.array([[[[0, 5, 5, np.nan, 9, -np.inf, 5, -0.0]]]], np.float32)
    pick = lambda *a, **kw: O.select(w, [0], [8], *a, **kw)[0][0, 0, 0].tolist()  # noqa: E731
    assert pick(3) == [1, 2, 4] and pick(2) == [1, 4] and pick(5) == [0, 1, 2, 4, 6]
    assert pick(6) == [0, 1, 2, 4, 6, 7] and pick(7) == [0, 1, 2, 4, 5, 6, 7]
    assert pick(3, sink=1, recent=1) == [0, 4, 7] and pick(2, recent=2) == [6, 7]
    assert O.select(w, [0], [3], 4)[0][0, 0, 0].tolist() == [0, 1, 2, -1]
    assert O.select(w, [1], [9], 4)[1] == O.select(w, [0], [9], 4)[1] == O.METADATA


def test_evict_oracle_by_hand():
    pool = np.arange(6 * 2 * 8).reshape(6, 2, 8, 1)
    s = OC.State([[0, 1, 2], [0, 3, -1]], [20, 12], [2, 1, 1, 1, 0, 0], 8, [pool])
    O.evict(s, [0], np.array([[[[0, 2, 3, 5, 7, 9, 11, 17, 19]]]]))
    assert s.tables == [[4, 1, 2], [0, 3, -1]] and s.lens == [9, 12]
    assert s.refs == [1, 1, 0, 1, 1, 0]
    assert s.pools[0][4, 0, :, 0].tolist() == [0, 2, 3, 5, 7, 17, 19, 33]
    assert s.pools[0][1, 1, 0, 0] == 2 * 16 + 8 + 3 and s.status == 0
    assert np.array_equal(s.pools[0][0], pool[0])


def test_weights_oracle_by_hand():
    q, keys = np.zeros((2, 1, 4)), [np.ones((3, 1, 4))]
    w = O.weights(q, np.log([[2.0], [3.0]]), keys, [3], [0, 2], [np.full((1, 3), 8.0)], decay=0.5)
    np.testing.assert_allclose(w[0], [[4 + 1 / 2 + 1 / 3, 1 / 2 + 1 / 3, 1 / 3]])
    w = O.weights(q, np.log([[2.0], [3.0]]), keys, [3], [0, 2], [np.full((1, 3), 8.0)], last=1,
                  causal=False)
    np.testing.assert_allclose(w[0], [[8 + 1 / 3, 1 / 3, 1 / 3]])


# ---- the binding --------------------------------------------------------------------------------

def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_weights_call(calls):  # noqa: F811
    cache, w = bf16(9, 2, 2, 16, 128), torch.zeros(3, 2, 40)
    run = pkb.accumulate_attention_weights
    assert run(bf16(3, 8, 128), torch.zeros(3, 8), cache, i32(3), w, block_tables=i32(3, 5),
               decay=0.5) is w
    name, p, rest = calls[-1]
    assert name == "paged_weights_run"
    assert (p.batch, p.num_qo_heads, p.num_kv_heads, p.head_dim, p.page_size, p.num_pages,
            p.combined_cache, p.max_pages_per_request, p.seq_len_q, p.total_q, p.last_queries,
            p.mask_type, p.width, p.sm_scale, p.decay) == (3, 8, 2, 128, 16, 9, 1, 5, 1, 3, 0, 1,
                                                           40, 0.0, 0.5)
    assert rest[1] and rest[3] is None and rest[4] is None
    seen = w._version
    run(bf16(3, 4, 8, 128), torch.zeros(3, 4, 8), (bf16(9, 2, 16, 128),) * 2, i32(3), w,
        paged_kv_indptr=i32(4), paged_kv_indices=i32(7), mask_type="dense", sm_scale=2.0)
    p = calls[-1][1]
    assert (p.seq_len_q, p.total_q, p.mask_type, p.sm_scale, p.combined_cache) == (4, 12, 0, 2.0, 0)
    assert w._version > seen
    run(bf16(7, 8, 128), torch.zeros(7, 8), cache, i32(3), w, block_tables=i32(3, 5),
        qo_indptr=i32(4), last_queries=2)
    assert (calls[-1][1].total_q, calls[-1][1].last_queries) == (7, 2) and calls[-1][2][3]
    good = dict(query=bf16(3, 8, 128), lse=torch.zeros(3, 8), paged_kv_cache=cache,
                seq_lens_kv=i32(3), weights=w, block_tables=i32(3, 5))
    for bad in (dict(query=bf16(2, 8, 128)), dict(query=bf16(3, 8, 64)),
                dict(query=torch.zeros(3, 8, 128)), dict(query=bf16(3, 128, 8).transpose(1, 2)),
                dict(lse=torch.zeros(8, 3).T), dict(lse=torch.zeros(3, 9)),
                dict(lse=torch.zeros(3, 8).double()), dict(weights=torch.zeros(3, 3, 40)),
                dict(weights=torch.zeros(3, 2, 80)[..., ::2]), dict(weights=torch.zeros(6, 40)),
                dict(weights=torch.zeros(3, 2, 40, requires_grad=True)),
                dict(block_tables=i32(4, 5)), dict(block_tables=None),
                dict(paged_kv_indptr=i32(4)), dict(qo_indptr=i32(3)),
                dict(seq_lens_kv=torch.zeros(3, dtype=torch.int64)), dict(status=i32(0)),
                dict(mask_type="full"), dict(last_queries=1.5)):
        n = len(calls)
        with pytest.raises((ValueError, TypeError, KeyError)):
            run(**{**good, **bad})
        assert len(calls) == n, bad


def test_select_call(calls):  # noqa: F811
    w = torch.zeros(3, 5, 2, 40)
    kept = pkb.select_cache_tokens(i32(4), w, i32(5), 7, sink=1, recent=2)
    p = calls[-1][1]
    assert kept.shape == (3, 4, 2, 7) and kept.dtype is torch.int32
    assert (p.num_layers, p.rows, p.num_kv_heads, p.width) == (3, 5, 2, 40)
    assert (p.keep, p.sink, p.recent) == (7, 1, 2)
    assert calls[-1][2][1] == 4
    assert pkb.select_cache_tokens(i32(4), w[0], i32(5), 7).shape == (4, 2, 7)
    for bad in (dict(weights=w.double()), dict(weights=w[..., ::2]), dict(weights=w[0, 0]),
                dict(seq_lens=i32(4)), dict(keep=0), dict(keep=2.5), dict(kept=i32(3, 4, 2, 6)),
                dict(kept=i32(3, 4, 2, 14)[..., ::2]), dict(rows=i32(8)[::2])):
        n = len(calls)
        with pytest.raises((ValueError, TypeError)):
            pkb.select_cache_tokens(**{**dict(rows=i32(4), weights=w, seq_lens=i32(5), keep=7),
                                       **bad})
        assert len(calls) == n, bad


def test_evict_call(calls, monkeypatch):  # noqa: F811
    monkeypatch.setattr(E, "evict_cache_workspace_size", lambda *a: 64)
    pools = pkb.cache_pools([bf16(9, 2, 2, 16, 8)] * 3)
    state, w = (i32(5, 4), i32(5), i32(9)), torch.zeros(3, 5, 2, 40)
    word, seen = i32(1), w._version
    pkb.evict_cache_rows(pools, i32(4), i32(3, 4, 2, 7), *state, weights=w, sink=3, status=word)
    name, p, rest = calls[-1]
    assert name == "paged_cache_evict_run" and p.status_dev == word.data_ptr()
    assert rest[2] == 4 and rest[4:6] == (7, 3) and rest[7] == 40 and w._version > seen
    pkb.evict_cache_rows(pools, i32(4), i32(3, 4, 2, 7), *state)
    assert calls[-1][2][6] is None
    one = pkb.cache_pools([bf16(9, 2, 2, 16, 8)])
    pkb.evict_cache_rows(one, i32(4), i32(4, 2, 7), *state, weights=w[0])
    for bad in (dict(kept=i32(3, 3, 2, 7)), dict(kept=i32(4, 2, 7)), dict(weights=w[:, :4]),
                dict(weights=w[0]), dict(weights=w.half()), dict(kept=i32(3, 4, 2, 7).float()),
                dict(weights=torch.zeros(3, 5, 2, 40, requires_grad=True)), dict(sink=0.5),
                dict(page_refs=i32(9).long()), dict(status=i32(0))):
        n = len(calls)
        with pytest.raises((ValueError, TypeError)):
            pkb.evict_cache_rows(**{**dict(pools=pools, rows=i32(4), kept=i32(3, 4, 2, 7),
                                           block_tables=state[0], seq_lens=state[1],
                                           page_refs=state[2]), **bad})
        assert len(calls) == n, bad


# ---- the C entry points -------------------------------------------------------------------------

def test_weights_refusals(lib):
    base = dict(batch=2, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=10,
                combined_cache=1, max_pages_per_request=4, seq_len_q=1, total_q=2, last_queries=0,
                mask_type=1, width=64, sm_scale=0.0, decay=1.0)

    def run(params=None, **kw):
        p = E.WeightsParams(**{**base, **(params or {})})
        a = dict(q=A16, lse=A16, k=A16, qo=None, indptr=None, pages=A16, lens=A16, w=A16,
                 status=None)
        a.update(kw)
        return lib.paged_weights_run(C.byref(p), *a.values(), None)
    for params in (dict(batch=-1), dict(num_qo_heads=7), dict(num_kv_heads=0), dict(head_dim=64),
                   dict(num_qo_heads=130), dict(page_size=12), dict(page_size=136),
                   dict(page_size=0), dict(num_pages=0), dict(num_pages=1 << 25), dict(width=0), dict(mask_type=2),
                   dict(decay=float("nan")), dict(sm_scale=float("inf")), dict(last_queries=-1),
                   dict(total_q=3), dict(seq_len_q=2), dict(total_q=-1), dict(seq_len_q=-1),
                   dict(max_pages_per_request=0), dict(num_kv_heads=4096, num_qo_heads=4096,
                                                       num_pages=1 << 20)):
        assert run(params) == BAD, params
    for kw in (dict(q=None), dict(lse=None), dict(k=None), dict(pages=None), dict(lens=None),
               dict(w=None), dict(q=A16 + 8), dict(k=A16 + 8), dict(lse=A16 + 2), dict(w=A16 + 1),
               dict(qo=A16 + 2), dict(indptr=A16 + 2), dict(status=A16 + 2), dict(lens=A16 + 1)):
        assert run(**kw) == BAD, kw
    assert lib.paged_weights_run(None, *[A16] * 9, None) == BAD
    assert run(dict(batch=0, total_q=0)) == 0              # nothing to do, nothing enqueued
    assert run(dict(total_q=0), qo=A16) == 0


def test_select_refusals(lib):
    base = dict(num_layers=2, rows=4, num_kv_heads=2, width=64, keep=8, sink=2, recent=2)

    def run(params=None, n=2, **kw):
        p = E.SelectParams(**{**base, **(params or {})})
        a = dict(w=A16, lens=A16, kept=A16, status=None)
        rows = kw.pop("rows", A16)
        a.update(kw)
        return lib.paged_cache_select_run(C.byref(p), rows, n, *a.values(), None)
    for params in (dict(num_layers=0), dict(rows=-1), dict(num_kv_heads=0), dict(width=0),
                   dict(keep=0), dict(sink=-1), dict(recent=-1), dict(sink=7), dict(recent=9),
                   dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert run(params) == BAD, params
    for kw in (dict(n=-1), dict(rows=None), dict(w=None), dict(lens=None), dict(kept=None),
               dict(rows=A16 + 2), dict(w=A16 + 2), dict(kept=A16 + 1), dict(status=A16 + 3),
               dict(n=1 << 30)):
        assert run(**kw) == BAD, kw
    assert run(n=0) == 0


def test_evict_refusals(lib):
    p = K.CacheParams(rows=4, max_pages_per_request=8, page_size=16, num_pages=32)
    ptrs = (C.c_void_p * 1)(A16)
    pools = dict(num_layers=1, num_pages=32, num_kv_heads=2, page_size=16, head_dim=64,
                 combined_cache=1, pools_host=ptrs)

    def run(params=p, n=2, keep=20, sink=0, width=64, size=1 << 20, pools=pools, **kw):
        a = dict(rows=A16, kept=A16, w=A16, bt=A16, sl=A16, pr=A16, ws=A16)
        a.update(kw)
        return lib.paged_cache_evict_run(C.byref(params), C.byref(K.CachePoolsStruct(**pools)),
                                         a["rows"], n, a["kept"], keep, sink, a["w"], width,
                                         a["bt"], a["sl"], a["pr"], a["ws"], size, None)
    for kw in (dict(n=-1), dict(n=4097), dict(keep=0), dict(keep=-1), dict(sink=-1), dict(sink=21),
               dict(width=0), dict(rows=None), dict(kept=None), dict(bt=None), dict(sl=None),
               dict(pr=None), dict(rows=A16 + 2), dict(kept=A16 + 2), dict(w=A16 + 2),
               dict(ws=A16 + 8), dict(pr=A16 + 1), dict(pools={**pools, "page_size": 32}),
               dict(pools={**pools, "num_pages": 31}), dict(pools={**pools, "head_dim": 12}),
               dict(params=K.CacheParams(rows=4, max_pages_per_request=8, page_size=16,
                                         num_pages=32, status_dev=A16 + 2))):
        assert run(**kw) == BAD, kw
    need = pkb.evict_cache_workspace_size(2, 20, 16)
    assert run(size=need - 1) == run(ws=None) == pkb.ERR_WORKSPACE
    assert need >= 16 + 2 * 16 + 2 * 2 * 2 * 4
    for bad in ((-1, 20, 16), (4097, 20, 16), (2, 0, 16), (2, 20, 12), (2, 20, 0), (2, 20, 256)):
        assert pkb.evict_cache_workspace_size(*bad) == 0
    assert pkb.evict_cache_workspace_size(4096, 2 ** 31 - 1, 8) > 2 ** 42
