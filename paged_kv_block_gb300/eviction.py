"""Binding of the calls of include/paged_cache.h that keep rows within a budget of tokens: adding up
the attention weight of every cached token, selecting the tokens to keep, cutting rows back.

Argument marshalling only, by the rules of cache.py.
"""
from __future__ import annotations

import ctypes as C
import functools
import operator

import torch

from . import cache as _cache

_F32, _BF16 = torch.float32, torch.bfloat16
_MASK = {"dense": 0, "causal": 1}


class WeightsParams(C.Structure):
    _fields_ = [("batch", C.c_int), ("num_qo_heads", C.c_int), ("num_kv_heads", C.c_int),
                ("head_dim", C.c_int), ("page_size", C.c_int), ("num_pages", C.c_int),
                ("combined_cache", C.c_int), ("max_pages_per_request", C.c_int),
                ("seq_len_q", C.c_int), ("total_q", C.c_int), ("last_queries", C.c_int),
                ("mask_type", C.c_int), ("width", C.c_int), ("sm_scale", C.c_float),
                ("decay", C.c_float)]


class SelectParams(C.Structure):
    _fields_ = [("num_layers", C.c_int), ("rows", C.c_int), ("num_kv_heads", C.c_int),
                ("width", C.c_int), ("keep", C.c_int), ("sink", C.c_int), ("recent", C.c_int)]


_P = C.c_void_p
EXPORTS = {
    "paged_weights_run": (C.c_int, [C.POINTER(WeightsParams)] + [_P] * 10),
    "paged_cache_select_run": (C.c_int, [C.POINTER(SelectParams), _P, C.c_int] + [_P] * 5),
    "paged_cache_evict_workspace_size": (C.c_size_t, [C.c_int, C.c_int, C.c_int]),
    "paged_cache_evict_run": (C.c_int, [C.POINTER(_cache.CacheParams),
                                        C.POINTER(_cache.CachePoolsStruct), _P, C.c_int, _P,
                                        C.c_int, C.c_int, _P, C.c_int, _P, _P, _P, _P, C.c_size_t,
                                        _P]),
}


def _int(x, name):
    """A whole number that the C call's int holds (ctypes would cut it off without a word)."""
    x = operator.index(x)
    if not -_cache._INT_MAX - 1 <= x <= _cache._INT_MAX:
        raise ValueError(f"{name} is {x}, out of 32 bits")
    return x


def _struct(cls, fields):
    """The parameter struct; its whole numbers are checked here, once per set of arguments."""
    for (name, kind), x in zip(cls._fields_, fields):
        if kind is C.c_int:
            _int(x, name)
    return C.byref(cls(*fields))


@functools.lru_cache(maxsize=512)
def _weights_params(*fields):
    return _struct(WeightsParams, fields)


@functools.lru_cache(maxsize=512)
def _select_params(*fields):
    return _struct(SelectParams, fields)


def _plain(t, dtype, dev, name, shape):
    """Address of a contiguous tensor of that dtype and shape on the current device."""
    if (t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()
            or t.shape != shape):
        _cache._on_device(t, dev, name)
        raise ValueError(f"{name} must be contiguous {dtype} of shape {list(shape)}")
    return t.data_ptr()


def _written(t, name):
    """A tensor that the call writes: autograd cannot follow it, and learns of the change."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} is written in place and must not require a gradient")


def accumulate_attention_weights(query, lse, paged_kv_cache, seq_lens_kv, weights, *,
                                 block_tables=None, paged_kv_indptr=None, paged_kv_indices=None,
                                 qo_indptr=None, last_queries=0, mask_type="causal",
                                 sm_scale=None, decay=1.0, status=None, stream=None):
    """Add to `weights` [B, Hkv, W] (fp32, in place) the attention that every cached token got in
    an attention call: the sum, over the request's queries and the query heads of a KV head, of
    exp(sm_scale q.k - lse).  Returns weights.

    query and lse are that call's: [B, Hq, D] with lse [B, Hq], [B, SQ, Hq, D] with [B, SQ, Hq], or
    packed [total, Hq, D] with [total, Hq] and qo_indptr.  The page table is block_tables [B, C] or
    paged_kv_indptr with paged_kv_indices; the cache a combined one or a (K, V) pair.  Older weights
    are multiplied by `decay`; the entries of the call's own query tokens (the last of each request)
    start at 0, those of a forked row are the program's to copy from its parent's.  last_queries = n
    counts only the last n queries of each request.
    The attention call must have had no window; this one has no gradient.  status: an int32 word
    that device-side findings are OR-ed into."""
    dev = _cache._device()
    kc, _, combined, P, Hkv, ps, D = _cache._geometry(paged_kv_cache, dev)
    B = _cache._count(seq_lens_kv, "seq_lens_kv")
    shape = query.shape
    sq = cols = 0
    qo = indptr = None
    if qo_indptr is not None:
        if len(shape) != 3:
            raise ValueError("packed query must be [total, Hq, D]")
        qo = _cache._ints_of(qo_indptr, dev, "qo_indptr", B + 1)
        total = shape[0]
    else:
        if len(shape) not in (3, 4) or shape[0] != B:
            raise ValueError("query must be [B, Hq, D] or [B, SQ, Hq, D]")
        sq = 1 if len(shape) == 3 else shape[1]
        total = B * sq
    if shape[-1] != D or total > _cache._INT_MAX:
        raise ValueError("query must have the cache's columns")
    qp = _plain(query, _BF16, dev, "query", shape)
    lp = _plain(lse, _F32, dev, "lse", shape[:-1])
    if weights.dim() != 3:
        raise ValueError("weights must be [B, Hkv, W]")
    W = weights.shape[2]
    wp = _plain(weights, _F32, dev, "weights", (B, Hkv, W))
    _written(weights, "weights")
    if block_tables is not None:
        if paged_kv_indptr is not None or paged_kv_indices is not None:
            raise ValueError("either block_tables or the CSR table")
        if block_tables.dim() != 2 or block_tables.shape[0] != B:
            raise ValueError("block_tables must be [B, C]")
        pages = _cache._ints(block_tables, dev, "block_tables")
        cols = block_tables.shape[1]
    else:
        if paged_kv_indptr is None or paged_kv_indices is None:
            raise ValueError("a page table is needed")
        indptr = _cache._ints_of(paged_kv_indptr, dev, "paged_kv_indptr", B + 1)
        pages = _cache._ints(paged_kv_indices, dev, "paged_kv_indices")
    lens = _cache._ints(seq_lens_kv, dev, "seq_lens_kv")
    if status is not None:
        status = _cache._status(status, dev)
    rc = _cache._call.paged_weights_run(
        _weights_params(B, shape[-2], Hkv, D, ps, P, combined, cols, sq, total,
                        operator.index(last_queries), _MASK[mask_type], W,
                        float(sm_scale or 0.0), float(decay) + 0.0),
        qp, lp, kc, qo, indptr, pages, lens, wp, status, _cache._stream(stream, dev))
    if rc:
        _cache._check(rc, "paged_weights_run")
    _cache._increment_version(weights)
    return weights


def select_cache_tokens(rows, weights, seq_lens, keep, *, sink=0, recent=0, kept=None, status=None,
                        stream=None):
    """The tokens to keep of each listed row, by `weights` [layers, rows, Hkv, W] (or [rows, Hkv,
    W]): the first `sink`, the last `recent` and those of the highest weight between them, `keep` in
    all.  Returns kept [layers, n, Hkv, keep] (or [n, Hkv, keep]) int32, ascending; rows of at
    most `keep` tokens keep them all, followed by -1.
    status: an int32 word that device-side findings are OR-ed into."""
    dev = _cache._device()
    shape = weights.shape
    if len(shape) not in (3, 4):
        raise ValueError("weights must be [layers, rows, Hkv, W] or [rows, Hkv, W]")
    N = shape[0] if len(shape) == 4 else 1
    R, Hkv, W = shape[-3:]
    if max(shape) > _cache._INT_MAX:
        raise ValueError("weights is too large")
    wp = _plain(weights, _F32, dev, "weights", shape)
    n = _cache._count(rows, "rows")
    rp = _cache._ints(rows, dev, "rows")
    lens = _cache._ints_of(seq_lens, dev, "seq_lens", R)
    keep = operator.index(keep)
    if not 1 <= keep <= _cache._INT_MAX:
        raise ValueError("keep must be positive")
    want = (n, Hkv, keep) if len(shape) == 3 else (N, n, Hkv, keep)
    if kept is None:
        kept = _cache._new(want, torch.int32, weights.device, stream)
    elif kept.shape != want:
        raise ValueError(f"kept must be {list(want)}")
    kp = _cache._ints(kept, dev, "kept")
    if status is not None:
        status = _cache._status(status, dev)
    rc = _cache._call.paged_cache_select_run(
        _select_params(N, R, Hkv, W, keep, operator.index(sink), operator.index(recent)),
        rp, n, wp, lens, kp, status, _cache._stream(stream, dev))
    if rc:
        _cache._check(rc, "paged_cache_select_run")
    return kept


def evict_cache_workspace_size(n: int, keep: int, page_size: int) -> int:
    return int(_cache._call.paged_cache_evict_workspace_size(
        _int(n, "n"), _int(keep, "keep"), _int(page_size, "page_size")))


def evict_cache_rows(pools, rows, kept, block_tables, seq_lens, page_refs, *, weights=None, sink=0,
                     workspace=None, status=None, stream=None) -> None:
    """Cut each listed row back to the tokens of `kept` [layers, n, Hkv, keep] (from
    select_cache_tokens; [n, Hkv, keep] with one layer): in every layer and KV head they move to
    the row's first slots, and so do their `weights` [layers, rows, Hkv, W]; pages past them are
    given back, and pages that other rows share are replaced by fresh ones before they change.
    Rows of at most `keep` tokens stay as they are.  The others have no more in common with other
    rows than their first `sink` tokens.

    sink: the `sink` that the lists were selected with; pages that lie wholly in it stay shared.
    Rows that the free pages do not suffice for stay as they are; `status` and the workspace tell,
    as in extend_cache_rows."""
    dev = _cache._device()
    p, bt, sl, pr = _cache._rows_state(block_tables, seq_lens, page_refs, pools.page_size, dev,
                                       status)
    N, Hkv = pools.struct.num_layers, pools.struct.num_kv_heads
    n = _cache._count(rows, "rows")
    shape = kept.shape
    if tuple(shape[:-1]) != (N, n, Hkv) and not (N == 1 and tuple(shape[:-1]) == (n, Hkv)):
        raise ValueError(f"kept must be [{N}, {n}, {Hkv}, keep]")
    keep, sink = _int(shape[-1], "keep"), _int(sink, "sink")
    kp = _cache._ints(kept, dev, "kept")
    wp, W = None, 0
    if weights is not None:
        R = block_tables.shape[0]
        W = _int(weights.shape[-1], "the width of weights") if weights.dim() else 0
        want = (R, Hkv, W) if N == 1 and weights.dim() == 3 else (N, R, Hkv, W)
        wp = _plain(weights, _F32, dev, "weights", want)
        _written(weights, "weights")
    ps = pools.page_size
    ws = _cache._workspace(workspace, lambda k: evict_cache_workspace_size(k, keep, ps), n, rows,
                           dev, stream)
    rc = _cache._call.paged_cache_evict_run(
        p, pools.ref(dev), _cache._ints(rows, dev, "rows"), n, kp, keep, sink, wp, W, bt, sl, pr,
        ws.data_ptr(), ws.nbytes, _cache._stream(stream, dev))
    if rc:
        _cache._check(rc, "paged_cache_evict_run")
    if weights is not None:
        _cache._increment_version(weights)


__all__ = ["accumulate_attention_weights", "select_cache_tokens", "evict_cache_rows",
           "evict_cache_workspace_size", "WeightsParams", "SelectParams"]
