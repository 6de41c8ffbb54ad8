"""Binding of the cache side of libpagedattn (include/paged_cache.h): rotary positions, appending
to the paged K/V cache, and the pages' ownership.

Argument marshalling only, like the rest of the binding: shapes, types and devices are checked
here, values on the device by the kernels.  The functions take torch tensors on the current
CUDA device and enqueue on the current stream unless `stream` is given.
"""
from __future__ import annotations

import ctypes as C

import torch

ROPE_LAYOUT = {"half": 0, "interleaved": 1}
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "wavelength": 4}
_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
MAX_POOLS = 256


class RopeScaling(C.Structure):
    _fields_ = [("rotary_dim", C.c_int), ("kind", C.c_int), ("base", C.c_double),
                ("factor", C.c_double), ("original_max_position", C.c_double),
                ("low", C.c_double), ("high", C.c_double)]


class RopeParams(C.Structure):
    _fields_ = [("num_tokens", C.c_int), ("num_qo_heads", C.c_int), ("num_kv_heads", C.c_int),
                ("head_dim", C.c_int), ("rotary_dim", C.c_int), ("layout", C.c_int),
                ("dtype", C.c_int), ("inverse", C.c_int), ("attention_factor", C.c_float),
                ("q_token_stride", C.c_int64), ("q_head_stride", C.c_int64),
                ("k_token_stride", C.c_int64), ("k_head_stride", C.c_int64),
                ("q_out_token_stride", C.c_int64), ("q_out_head_stride", C.c_int64),
                ("k_out_token_stride", C.c_int64), ("k_out_head_stride", C.c_int64)]


class AppendParams(C.Structure):
    _fields_ = [("batch", C.c_int), ("seq_len_q", C.c_int), ("total_q", C.c_int),
                ("num_qo_heads", C.c_int), ("num_kv_heads", C.c_int), ("head_dim", C.c_int),
                ("page_size", C.c_int), ("num_pages", C.c_int), ("combined_cache", C.c_int),
                ("max_pages_per_request", C.c_int), ("rotary_dim", C.c_int),
                ("layout", C.c_int), ("attention_factor", C.c_float), ("in_dtype", C.c_int),
                ("q_token_stride", C.c_int64), ("k_token_stride", C.c_int64),
                ("v_token_stride", C.c_int64)]


class CacheParams(C.Structure):
    _fields_ = [("rows", C.c_int), ("max_pages_per_request", C.c_int), ("page_size", C.c_int),
                ("num_pages", C.c_int)]


class CachePoolsStruct(C.Structure):
    _fields_ = [("num_layers", C.c_int), ("num_pages", C.c_int), ("num_kv_heads", C.c_int),
                ("page_size", C.c_int), ("head_dim", C.c_int), ("combined_cache", C.c_int),
                ("pools_host", C.POINTER(C.c_void_p))]


_P = C.c_void_p
EXPORTS = {
    "paged_rope_frequencies": (C.c_int, [C.POINTER(RopeScaling), C.POINTER(C.c_double),
                                         C.POINTER(C.c_float)]),
    "paged_rope_table": (C.c_int, [C.POINTER(C.c_double), C.c_int, C.POINTER(C.c_uint64)]),
    "paged_rope_run": (C.c_int, [C.POINTER(RopeParams)] + [_P] * 7),
    "paged_append_run": (C.c_int, [C.POINTER(AppendParams)] + [_P] * 13),
    "paged_cache_free_run": (C.c_int, [C.POINTER(CacheParams), _P, C.c_int] + [_P] * 5),
    "paged_cache_extend_workspace_size": (C.c_size_t, [C.c_int]),
    "paged_cache_extend_run": (C.c_int, [C.POINTER(CacheParams), _P, _P, C.c_int, _P, _P, _P, _P,
                                         C.c_size_t, _P]),
    "paged_cache_fork_workspace_size": (C.c_size_t, [C.c_int]),
    "paged_cache_fork_run": (C.c_int, [C.POINTER(CacheParams), C.POINTER(CachePoolsStruct), _P,
                                       _P, C.c_int, _P, _P, _P, _P, C.c_size_t, _P]),
    "paged_cache_compact_workspace_size": (C.c_size_t, [C.c_int]),
    "paged_cache_compact_run": (C.c_int, [C.POINTER(CacheParams), C.POINTER(CachePoolsStruct)]
                                + [_P] * 7 + [C.c_size_t, _P]),
    "paged_cache_copy_run": (C.c_int, [C.POINTER(CachePoolsStruct), C.POINTER(CachePoolsStruct),
                                       _P, _P, C.c_int, _P, _P]),
}


def _lib():
    from . import lib
    return lib()


def _check(code, what):
    if code != 0:
        from . import PagedAttnError
        raise PagedAttnError(code, what)


def _stream(stream):
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _on_device(t, name):
    """The current device has to hold `t`: the call runs there."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is not on the current device")


def _ints(t, name, n=None):
    """Address of a contiguous int32 tensor on the current device (of n elements)."""
    _on_device(t, name)
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements")
    return t.data_ptr()


def _status(t):
    """Address of an optional 4-byte status word (int32 or uint32, any shape)."""
    if t is None:
        return None
    _on_device(t, "status")
    if t.element_size() != 4 or t.numel() < 1 or not t.is_contiguous():
        raise ValueError("status must hold a 32-bit word")
    return t.data_ptr()


def _table(freqs, name="freqs"):
    _on_device(freqs, name)
    if freqs.dtype != torch.int64 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError(f"{name} must be a table made by rope_frequencies")
    return freqs.data_ptr()


def _workspace(workspace, nbytes, device):
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    _on_device(workspace, "workspace")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def _nbytes(t):
    return t.numel() * t.element_size()


# ---------------------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------------------

def rope_frequencies(rotary_dim, *, base=10000.0, scaling="none", factor=1.0,
                     original_max_position=0.0, low=0.0, high=0.0, inv_freq=None, device=None):
    """(freqs, attention_factor): the table of the rotary kernels for the first `rotary_dim`
    columns (an int64 tensor of rotary_dim / 2 fixed-point turns per position, on `device` or
    the current CUDA device), and the factor that the scaling asks for.

    scaling: "none", "linear", "ntk", "yarn" or "wavelength" (formulas in the C header), for a
    context `factor` times the original.  inv_freq gives the angles per position themselves
    (rotary_dim / 2 values, in radians) instead.  Make the table once and keep it."""
    n = rotary_dim // 2
    out, m = (C.c_double * max(n, 1))(), C.c_float(1.0)
    if inv_freq is not None:
        if len(inv_freq) != n or rotary_dim % 2:
            raise ValueError("inv_freq must have rotary_dim / 2 values")
        values = inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else list(inv_freq)
        for i, f in enumerate(values):
            out[i] = float(f)
    else:
        s = RopeScaling(rotary_dim=rotary_dim, kind=ROPE_SCALING[scaling], base=base,
                        factor=factor, original_max_position=original_max_position, low=low,
                        high=high)
        _check(_lib().paged_rope_frequencies(C.byref(s), out, C.byref(m)),
               "paged_rope_frequencies")
    table = (C.c_uint64 * max(n, 1))()
    _check(_lib().paged_rope_table(out, n, table), "paged_rope_table")
    host = torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in table[:n]],
                        dtype=torch.int64)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return host.to(device), m.value


def _rows(t, name):
    """(tokens, heads, D, token stride, head stride) of [T, H, D] or [B, S, H, D] rows whose
    columns are contiguous and whose leading dimensions step evenly."""
    _on_device(t, name)
    if t.dim() == 4:
        B, S, H, D = t.shape
        sb, ts, hs, e = t.stride()
        if B > 1 and S > 1 and sb != S * ts:
            raise ValueError(f"{name}: batch and sequence must step evenly")
        if S == 1:
            ts = sb
        T = B * S
    elif t.dim() == 3:
        T, H, D = t.shape
        ts, hs, e = t.stride()
    else:
        raise ValueError(f"{name} must be [tokens, heads, D] or [batch, seq, heads, D]")
    if D > 1 and e != 1:
        raise ValueError(f"{name}: the columns of a head must be contiguous")
    return T, H, D, ts, hs


def rotary_embedding(q, positions, freqs, *, k=None, layout="half", attention_factor=1.0,
                     inverse=False, q_out=None, k_out=None, stream=None):
    """Rotate q (and k) [T, heads, D] or [B, S, heads, D] at int32 `positions` (one per token),
    the first 2 * len(freqs) columns of each head; returns q_out, or (q_out, k_out) with k.

    q_out=q rotates in place.  inverse=True turns back by the same angles (times the same
    attention_factor): the gradient of the input from the gradient of the output."""
    T, Hq, D, qt, qh = _rows(q, "q")
    dt = q.dtype
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    p = RopeParams(num_tokens=T, num_qo_heads=Hq, num_kv_heads=0, head_dim=D,
                   rotary_dim=2 * freqs.numel(), layout=ROPE_LAYOUT[layout], dtype=_DTYPE[dt],
                   inverse=int(inverse), attention_factor=attention_factor, q_token_stride=qt,
                   q_head_stride=qh)
    pos = _ints(positions, "positions", T)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=dt, device=q.device)
        p.q_out_token_stride, p.q_out_head_stride = Hq * D, D
    else:
        if q_out.shape != q.shape or q_out.dtype != dt:
            raise ValueError("q_out must have q's shape and dtype")
        _, _, _, p.q_out_token_stride, p.q_out_head_stride = _rows(q_out, "q_out")
    kp = kop = None
    if k is not None:
        Tk, Hk, Dk, p.k_token_stride, p.k_head_stride = _rows(k, "k")
        if Tk != T or Dk != D or k.dtype != dt:
            raise ValueError("k must have q's tokens, columns and dtype")
        if Hk < 1:
            raise ValueError("k must have heads")
        p.num_kv_heads = Hk
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=dt, device=q.device)
            p.k_out_token_stride, p.k_out_head_stride = Hk * D, D
        else:
            if k_out.shape != k.shape or k_out.dtype != dt:
                raise ValueError("k_out must have k's shape and dtype")
            _, _, _, p.k_out_token_stride, p.k_out_head_stride = _rows(k_out, "k_out")
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    if T == 0:
        return q_out if k is None else (q_out, k_out)
    _check(_lib().paged_rope_run(C.byref(p), q.data_ptr(), kp, pos, _table(freqs),
                                 q_out.data_ptr(), kop, _stream(stream)), "paged_rope_run")
    return q_out if k is None else (q_out, k_out)


# ---------------------------------------------------------------------------------------
# Appending to the cache
# ---------------------------------------------------------------------------------------

def _geometry(cache):
    """(K address, V address or None, combined, P, Hkv, page size, D) of a combined cache
    [P, 2, Hkv, ps, D] or a (K, V) pair of pools [P, Hkv, ps, D]; all bf16, contiguous."""
    pair = isinstance(cache, (tuple, list))
    k = cache[0] if pair else cache
    for t in (cache if pair else (cache,)):
        _on_device(t, "the cache")
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("the cache must be contiguous bf16")
    if pair:
        if len(cache) != 2 or k.dim() != 4 or cache[1].shape != k.shape:
            raise ValueError("K and V pools must both be [P, Hkv, page_size, D]")
        P, Hkv, ps, D = k.shape
        return k.data_ptr(), cache[1].data_ptr(), 0, P, Hkv, ps, D
    if k.dim() != 5 or k.shape[1] != 2:
        raise ValueError("a combined cache must be [P, 2, Hkv, page_size, D]")
    P, _, Hkv, ps, D = k.shape
    return k.data_ptr(), None, 1, P, Hkv, ps, D


def append_paged_kv_cache(k, v, paged_kv_cache, seq_lens_kv, *, block_tables=None,
                          paged_kv_indptr=None, paged_kv_indices=None, qo_indptr=None, q=None,
                          q_out=None, freqs=None, layout="half", attention_factor=1.0,
                          status=None, stream=None):
    """Write new K/V rows into the paged cache, keys rotated at their positions, and rotate the
    new queries; returns q_out (bf16) or None without q.

    k, v, q: [total, heads, D] with qo_indptr [B + 1], or one token per request [B, heads, D],
    or [B, SQ, heads, D]; bf16, fp16 or fp32, rows may be slices of a fused projection.  The
    page table is block_tables [B, C] or paged_kv_indptr with paged_kv_indices.  seq_lens_kv
    [B] counts the new tokens in.  freqs (from rope_frequencies) None writes keys as they are.
    status: an int32 word that device-side findings are OR-ed into."""
    kc, vc, combined, P, Hkv, ps, D = _geometry(paged_kv_cache)
    B = seq_lens_kv.numel()
    T, Hk, Dk, kt, kh = _rows(k, "k")
    Tv, Hv, Dv, vt, vh = _rows(v, "v")
    if Hk != Hkv or Dk != D or (Tv, Hv, Dv) != (T, Hk, Dk) or v.dtype != k.dtype:
        raise ValueError("k and v must have the cache's heads and columns, and the same dtype")
    if k.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {k.dtype}")
    if (kh != D or vh != D) and Hkv > 1:
        raise ValueError("the heads of k and v must be adjacent")
    p = AppendParams(batch=B, seq_len_q=0, total_q=0, num_qo_heads=0, num_kv_heads=Hkv,
                     head_dim=D, page_size=ps, num_pages=P, combined_cache=combined,
                     max_pages_per_request=0,
                     rotary_dim=0 if freqs is None else 2 * freqs.numel(),
                     layout=ROPE_LAYOUT[layout], attention_factor=attention_factor,
                     in_dtype=_DTYPE[k.dtype], k_token_stride=kt, v_token_stride=vt)
    if qo_indptr is not None:
        if k.dim() != 3:
            raise ValueError("packed k must be [total, heads, D]")
        qo = _ints(qo_indptr, "qo_indptr", B + 1)
        p.total_q = T
    else:
        qo = None
        if k.shape[0] != B:
            raise ValueError("k must have one entry per request")
        p.seq_len_q = T // B if B else 0
    if block_tables is not None:
        if paged_kv_indptr is not None or paged_kv_indices is not None:
            raise ValueError("either block_tables or the CSR table")
        if block_tables.dim() != 2 or block_tables.shape[0] != B:
            raise ValueError("block_tables must be [B, C]")
        indptr, pages = None, _ints(block_tables, "block_tables")
        p.max_pages_per_request = block_tables.shape[1]
    else:
        if paged_kv_indptr is None or paged_kv_indices is None:
            raise ValueError("a page table is needed")
        indptr = _ints(paged_kv_indptr, "paged_kv_indptr", B + 1)
        pages = _ints(paged_kv_indices, "paged_kv_indices")
    qp = qop = None
    if q is not None:
        Tq, Hq, Dq, p.q_token_stride, qh = _rows(q, "q")
        if Tq != T or Dq != D or q.dtype != k.dtype or (qh != D and Hq > 1):
            raise ValueError("q must have k's tokens, columns and dtype, and adjacent heads")
        p.num_qo_heads = Hq
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        elif q_out.shape != q.shape or q_out.dtype != torch.bfloat16 or not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous bf16 of q's shape")
        else:
            _on_device(q_out, "q_out")
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if T == 0 or B == 0:
        return q_out
    _check(_lib().paged_append_run(C.byref(p), qp, k.data_ptr(), v.data_ptr(), qo, indptr, pages,
                                   _ints(seq_lens_kv, "seq_lens_kv"),
                                   None if freqs is None else _table(freqs), qop, kc, vc,
                                   _status(status), _stream(stream)), "paged_append_run")
    return q_out


# ---------------------------------------------------------------------------------------
# Which row owns which page
# ---------------------------------------------------------------------------------------

class CachePools:
    """The pools of every layer, as the page operations take them: a handle that is made once
    and holds on to the tensors."""

    def __init__(self, layers):
        layers = list(layers)
        if not layers:
            raise ValueError("no layers")
        got = [_geometry(c) for c in layers]
        if any(g[2:] != got[0][2:] for g in got):
            raise ValueError("the layers' pools must have the same shape")
        ptrs = [p for g in got for p in g[:2] if p is not None]
        if len(ptrs) > MAX_POOLS:
            raise ValueError(f"more than {MAX_POOLS} pools")
        self.layers = layers
        self.device = (layers[0][0] if isinstance(layers[0], (tuple, list)) else layers[0]).device
        _, _, combined, self.num_pages, Hkv, self.page_size, D = got[0]
        self._ptrs = (C.c_void_p * len(ptrs))(*ptrs)
        self.struct = CachePoolsStruct(num_layers=len(layers), num_pages=self.num_pages,
                                       num_kv_heads=Hkv, page_size=self.page_size, head_dim=D,
                                       combined_cache=combined, pools_host=self._ptrs)


def cache_pools(layers) -> CachePools:
    """Handle of the layers' caches: combined caches [P, 2, Hkv, ps, D] or (K, V) pairs of
    pools [P, Hkv, ps, D], one per layer, all of one shape."""
    return CachePools(layers)


def _rows_state(block_tables, seq_lens, page_refs, page_size):
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [rows, C]")
    R, cols = block_tables.shape
    p = CacheParams(rows=R, max_pages_per_request=cols, page_size=page_size,
                    num_pages=page_refs.numel())
    return (p, _ints(block_tables, "block_tables"), _ints(seq_lens, "seq_lens", R),
            _ints(page_refs, "page_refs"))


def free_cache_rows(rows, block_tables, seq_lens, page_refs, page_size, *, status=None,
                    stream=None) -> None:
    """Free the listed rows: their pages' counts go down by one, their lengths to 0."""
    p, bt, sl, pr = _rows_state(block_tables, seq_lens, page_refs, page_size)
    _check(_lib().paged_cache_free_run(C.byref(p), _ints(rows, "rows"), rows.numel(), bt, sl, pr,
                                       _status(status), _stream(stream)), "paged_cache_free_run")


def extend_cache_workspace_size(n: int) -> int:
    return int(_lib().paged_cache_extend_workspace_size(int(n)))


def extend_cache_rows(rows, new_tokens, block_tables, seq_lens, page_refs, page_size, *,
                      workspace=None, stream=None) -> None:
    """Make each listed row longer by new_tokens tokens, with fresh pages (the lowest free ids,
    in the order listed) where needed.  Rows that the free pages do not suffice for stay as
    they are; the workspace's status word says so."""
    p, bt, sl, pr = _rows_state(block_tables, seq_lens, page_refs, page_size)
    n = rows.numel()
    ws = _workspace(workspace, extend_cache_workspace_size(n), rows.device)
    _check(_lib().paged_cache_extend_run(C.byref(p), _ints(rows, "rows"),
                                         _ints(new_tokens, "new_tokens", n), n, bt, sl, pr,
                                         ws.data_ptr(), _nbytes(ws), _stream(stream)),
           "paged_cache_extend_run")


def fork_cache_workspace_size(n: int) -> int:
    return int(_lib().paged_cache_fork_workspace_size(int(n)))


def fork_cache_rows(pools, parents, children, block_tables, seq_lens, page_refs, *,
                    workspace=None, stream=None) -> None:
    """Make the (empty) row children[i] a copy of row parents[i]: full pages are shared, the
    live tokens of a partly filled last page are copied into a fresh one, in every layer."""
    p, bt, sl, pr = _rows_state(block_tables, seq_lens, page_refs, pools.page_size)
    n = children.numel()
    ws = _workspace(workspace, fork_cache_workspace_size(n), children.device)
    _check(_lib().paged_cache_fork_run(C.byref(p), C.byref(pools.struct),
                                       _ints(parents, "parents", n),
                                       _ints(children, "children"), n, bt, sl, pr,
                                       ws.data_ptr(), _nbytes(ws), _stream(stream)),
           "paged_cache_fork_run")


def compact_cache_workspace_size(num_pages: int) -> int:
    return int(_lib().paged_cache_compact_workspace_size(int(num_pages)))


def compact_cache(pools, block_tables, seq_lens, page_refs, *, block_tables_out=None,
                  page_refs_out=None, num_live=None, workspace=None, stream=None):
    """Move the live pages to the pools' front, in every layer; returns (block_tables, page_refs,
    num_live [1]) after the move.  In place unless the *_out tensors are given."""
    p, bt, sl, pr = _rows_state(block_tables, seq_lens, page_refs, pools.page_size)
    tables = block_tables if block_tables_out is None else block_tables_out
    refs = page_refs if page_refs_out is None else page_refs_out
    if num_live is None:
        num_live = torch.empty(1, dtype=torch.int32, device=page_refs.device)
    ws = _workspace(workspace, compact_cache_workspace_size(p.num_pages), page_refs.device)
    _check(_lib().paged_cache_compact_run(C.byref(p), C.byref(pools.struct), bt, sl, pr,
                                          _ints(tables, "block_tables_out", block_tables.numel()),
                                          _ints(refs, "page_refs_out", page_refs.numel()),
                                          _ints(num_live, "num_live", 1), ws.data_ptr(),
                                          _nbytes(ws), _stream(stream)),
           "paged_cache_compact_run")
    return tables, refs, num_live


def copy_cache_pages(pools, src_pages, dst_pages, *, dst_pools=None, status=None,
                     stream=None) -> None:
    """Copy page src_pages[i] to page dst_pages[i] in every layer, within `pools` or to the same
    layers of `dst_pools`."""
    dst = pools if dst_pools is None else dst_pools
    n = src_pages.numel()
    _check(_lib().paged_cache_copy_run(C.byref(pools.struct), C.byref(dst.struct),
                                       _ints(src_pages, "src_pages"),
                                       _ints(dst_pages, "dst_pages", n), n, _status(status),
                                       _stream(stream)), "paged_cache_copy_run")


__all__ = ["rope_frequencies", "rotary_embedding", "append_paged_kv_cache", "CachePools",
           "cache_pools", "free_cache_rows", "extend_cache_rows", "extend_cache_workspace_size",
           "fork_cache_rows", "fork_cache_workspace_size", "compact_cache",
           "compact_cache_workspace_size", "copy_cache_pages", "RopeScaling", "RopeParams",
           "AppendParams", "CacheParams", "CachePoolsStruct"]
