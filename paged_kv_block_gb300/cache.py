"""Binding of the cache side of libpagedattn (include/paged_cache.h): rotary positions, appending
to the paged K/V cache, and the pages' ownership.

Argument marshalling only, like the rest of the binding: shapes, types and devices are checked
here, values on the device by the kernels.  The functions take torch tensors on the current
CUDA device and enqueue on the current stream unless `stream` is given; what they allocate
belongs to that stream, as under torch.cuda.stream(stream).
"""
from __future__ import annotations

import ctypes as C
import functools
import operator

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
                ("num_pages", C.c_int), ("status_dev", C.c_void_p)]


class CachePoolsStruct(C.Structure):
    _fields_ = [("num_layers", C.c_int), ("num_pages", C.c_int), ("num_kv_heads", C.c_int),
                ("page_size", C.c_int), ("head_dim", C.c_int), ("combined_cache", C.c_int),
                ("pools_host", C.POINTER(C.c_void_p))]


_P = C.c_void_p
EXPORTS = {
    "paged_rope_frequencies": (C.c_int, [C.POINTER(RopeScaling), C.POINTER(C.c_double),
                                         C.POINTER(C.c_float)]),
    "paged_rope_table": (C.c_int, [C.POINTER(C.c_double), C.c_int, C.POINTER(C.c_uint64)]),
    "paged_rope_run": (C.c_int, [C.POINTER(RopeParams)] + [_P] * 8),
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


_I32, _I64, _BF16 = torch.int32, torch.int64, torch.bfloat16
_INT_MAX = 2 ** 31 - 1
# The current stream's handle without building a Stream object, where this torch has the call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_grad_enabled = torch.is_grad_enabled
_increment_version = torch.autograd.graph.increment_version    # autograd learns of what is written
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

def _device():
    """Index of the current CUDA device; one that no tensor is on where there is no GPU."""
    try:
        return _current_device()
    except (RuntimeError, AssertionError):
        if torch.cuda.is_available():
            raise
        return -2


def _lib():
    from . import lib
    return lib()


class _Calls:
    """The library's functions by name, looked up once."""

    def __getattr__(self, name):
        f = getattr(_lib(), name)
        setattr(self, name, f)
        return f


_call = _Calls()


def _check(code, what):
    from . import PagedAttnError
    raise PagedAttnError(code, what)


def _stream(stream, dev):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream().cuda_stream


def _on_device(t, dev, name):
    """The current device has to hold `t`: the call runs there."""
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} is not on the current device")


def _ints(t, dev, name):
    """Address of a contiguous int32 tensor on the current device."""
    if t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous():
        _on_device(t, dev, name)
        raise ValueError(f"{name} must be a contiguous int32 tensor")
    return t.data_ptr()


def _count(t, name):
    """Number of elements, as the int that the C call takes."""
    n = t.numel()
    if n > _INT_MAX:
        raise ValueError(f"{name} has more than 2^31 - 1 elements")
    return n


def _ints_of(t, dev, name, n):
    """The same, of n elements."""
    if (t.numel() != n or t.dtype is not _I32 or t.get_device() != dev
            or not t.is_contiguous()):
        if t.numel() != n:
            raise ValueError(f"{name} must have {n} elements")
        return _ints(t, dev, name)
    return t.data_ptr()


def _status(t, dev):
    """Address of a 4-byte status word (int32 or uint32, any shape)."""
    _on_device(t, dev, "status")
    if t.element_size() != 4 or t.numel() < 1 or not t.is_contiguous():
        raise ValueError("status must hold a 32-bit word")
    return t.data_ptr()


def _new(shape, dtype, device, stream):
    """A new tensor from the pool of the stream that the call runs on: from another stream's,
    the allocator could hand the memory out again while the call's kernels still use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty(t, dtype, stream):
    """A new contiguous tensor of t's shape (empty_like is the cheaper call)."""
    if stream is None and t.dtype is dtype and t.is_contiguous():
        return torch.empty_like(t)
    return _new(t.shape, dtype, t.device, stream)


def _factor(m):
    """The attention factor as a float; -0.0 as 0.0, its equal."""
    return float(m) + 0.0


def _table(freqs, dev):
    if freqs.dtype is not _I64 or freqs.get_device() != dev or not freqs.is_contiguous():
        _on_device(freqs, dev, "freqs")
        raise ValueError("freqs must be a table made by rope_frequencies")
    return freqs.data_ptr()


def _workspace(workspace, size, n, like, dev, stream):
    """The caller's workspace, or a new one of size(n) bytes."""
    if workspace is None:
        return _new(size(n), torch.uint8, like.device, stream)
    _on_device(workspace, dev, "workspace")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


# Parameter structs depend on the static arguments alone, so equal calls share one (read-only).
# Every field is a Python number: a tensor would be found again by its identity, changed or not.
@functools.lru_cache(maxsize=512)
def _rope_params(*fields):
    return C.byref(RopeParams(*fields))


@functools.lru_cache(maxsize=512)
def _append_params(*fields):
    return C.byref(AppendParams(*fields))


@functools.lru_cache(maxsize=512)
def _cache_params(*fields):
    return C.byref(CacheParams(*fields))


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
        rc = _call.paged_rope_frequencies(C.byref(s), out, C.byref(m))
        if rc:
            _check(rc, "paged_rope_frequencies")
    table = (C.c_uint64 * max(n, 1))()
    rc = _call.paged_rope_table(out, n, table)
    if rc:
        _check(rc, "paged_rope_table")
    host = torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in table[:n]],
                        dtype=torch.int64)
    if device is None:
        device = torch.device("cuda", _device())
    return host.to(device), m.value


def _rows(t, dev, name):
    """(tokens, heads, D, token stride, head stride) of [T, H, D] or [B, S, H, D] rows whose
    columns are contiguous and whose leading dimensions step evenly."""
    if t.get_device() != dev:
        _on_device(t, dev, name)
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        T, H, D = shape
        ts, hs, e = stride
    elif len(shape) == 4:
        B, S, H, D = shape
        sb, ts, hs, e = stride
        if S == 1:
            ts = sb
        elif B > 1 and sb != S * ts:
            raise ValueError(f"{name}: batch and sequence must step evenly")
        T = B * S
    else:
        raise ValueError(f"{name} must be [tokens, heads, D] or [batch, seq, heads, D]")
    if T > _INT_MAX or H > _INT_MAX:
        raise ValueError(f"{name} is too large")
    if e != 1 and D > 1:
        raise ValueError(f"{name}: the columns of a head must be contiguous")
    if H <= 1:                               # the stride of a single head or token says nothing
        hs = D
    if T <= 1:
        ts = H * D
    elif ts == 0 and hs == 0:                # to the C call that means contiguous rows
        raise ValueError(f"{name}: all rows are one; repeat it or rotate it once")
    return T, H, D, ts, hs


class _Rotation(torch.autograd.Function):
    """rotary_embedding with its gradient, the rotation by the negative angles."""

    @staticmethod
    def forward(ctx, q, k, positions, freqs, layout, attention_factor, inverse, status, stream):
        ctx.save_for_backward(positions, freqs)
        ctx.how = dict(layout=layout, attention_factor=attention_factor, inverse=not inverse,
                       status=status)
        ctx.set_materialize_grads(False)
        return rotary_embedding(q, positions, freqs, k=k, layout=layout, inverse=inverse,
                                attention_factor=attention_factor, status=status, stream=stream)

    @staticmethod
    def backward(ctx, *grads):
        positions, freqs = ctx.saved_tensors
        if positions.is_cuda and torch.cuda.is_current_stream_capturing():
            # An eager graph of the same leaves would tie the captured stream to its own.
            raise ValueError("the gradient of rotary_embedding is not captured into graphs: call "
                             "it with inverse=True on the gradient of its output")
        wanted = [i for i, g in enumerate(grads) if g is not None and ctx.needs_input_grad[i]]
        out = [None] * 9
        if wanted:
            g = [grads[i].contiguous() for i in wanted]
            turned = rotary_embedding(g[0], positions, freqs, k=g[1] if len(g) > 1 else None,
                                      **ctx.how)
            for i, t in zip(wanted, turned if len(g) > 1 else (turned,)):
                out[i] = t
        return tuple(out)


def rotary_embedding(q, positions, freqs, *, k=None, layout="half", attention_factor=1.0,
                     inverse=False, q_out=None, k_out=None, status=None, stream=None):
    """Rotate q (and k) [T, heads, D] or [B, S, heads, D] at int32 `positions` (one per token),
    the first 2 * len(freqs) columns of each head; returns q_out, or (q_out, k_out) with k.

    q_out=q rotates in place.  inverse=True turns back by the same angles (times the same
    attention_factor): the gradient of the input from the gradient of the output.
    status: an int32 word that device-side findings are OR-ed into.

    Autograd knows the call: q and k may require gradients, then without q_out and k_out.  A
    gradient is not captured into a CUDA graph; call inverse=True there."""
    needs = q.requires_grad or (k is not None and k.requires_grad)
    given = None
    if q_out is not None or k_out is not None:
        given = (q_out,) if k_out is None else (k_out,) if q_out is None else (q_out, k_out)
        if (needs or given[0].requires_grad or given[-1].requires_grad) and _grad_enabled():
            raise ValueError("q_out and k_out are for tensors that require no gradient")
    elif needs and _grad_enabled():
        return _Rotation.apply(q, k, positions, freqs, layout, _factor(attention_factor),
                               bool(inverse), status, stream)
    dev = _device()
    T, Hq, D, qt, qh = _rows(q, dev, "q")
    dt = q.dtype
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    if q_out is None:
        q_out = _empty(q, dt, stream)
        qot, qoh = Hq * D, D
    else:
        if q_out.shape != q.shape or q_out.dtype != dt:
            raise ValueError("q_out must have q's shape and dtype")
        _, _, _, qot, qoh = _rows(q_out, dev, "q_out")
    Hk = kt = kh = kot = koh = 0
    kp = kop = None
    if k is not None:
        Tk, Hk, Dk, kt, kh = _rows(k, dev, "k")
        if Tk != T or Dk != D or k.dtype != dt:
            raise ValueError("k must have q's tokens, columns and dtype")
        if Hk < 1:
            raise ValueError("k must have heads")
        if k_out is None:
            k_out = _empty(k, dt, stream)
            kot, koh = Hk * D, D
        else:
            if k_out.shape != k.shape or k_out.dtype != dt:
                raise ValueError("k_out must have k's shape and dtype")
            _, _, _, kot, koh = _rows(k_out, dev, "k_out")
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    pos = _ints_of(positions, dev, "positions", T)
    table = _table(freqs, dev)
    if status is not None:
        status = _status(status, dev)
    if T:
        rc = _call.paged_rope_run(
            _rope_params(T, Hq, Hk, D, 2 * freqs.numel(), ROPE_LAYOUT[layout], _DTYPE[dt],
                         int(inverse), _factor(attention_factor), qt, qh, kt, kh, qot, qoh, kot,
                         koh),
            q.data_ptr(), kp, pos, table, q_out.data_ptr(), kop, status, _stream(stream, dev))
        if rc:
            _check(rc, "paged_rope_run")
        if given is not None:
            _increment_version(given)
    return q_out if k is None else (q_out, k_out)


# ---------------------------------------------------------------------------------------
# Appending to the cache
# ---------------------------------------------------------------------------------------

def _geometry(cache, dev):
    """(K address, V address or None, combined, P, Hkv, page size, D) of a combined cache
    [P, 2, Hkv, ps, D] or a (K, V) pair of pools [P, Hkv, ps, D]; all bf16, contiguous."""
    if isinstance(cache, (tuple, list)):
        k, v = cache
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("K and V pools must both be [P, Hkv, page_size, D]")
        P, Hkv, ps, D = k.shape
        return _pool(k, dev), _pool(v, dev), 0, P, Hkv, ps, D
    shape = cache.shape
    if len(shape) != 5 or shape[1] != 2:
        raise ValueError("a combined cache must be [P, 2, Hkv, page_size, D]")
    return _pool(cache, dev), None, 1, shape[0], shape[2], shape[3], shape[4]


def _pool(t, dev):
    if t.dtype is not _BF16 or t.get_device() != dev or not t.is_contiguous():
        _on_device(t, dev, "the cache")
        raise ValueError("the cache must be contiguous bf16")
    return t.data_ptr()


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
    The call has no gradient: what it returns never requires one.
    status: an int32 word that device-side findings are OR-ed into."""
    dev = _device()
    kc, vc, combined, P, Hkv, ps, D = _geometry(paged_kv_cache, dev)
    B = _count(seq_lens_kv, "seq_lens_kv")
    T, Hk, Dk, kt, kh = _rows(k, dev, "k")
    Tv, Hv, Dv, vt, vh = _rows(v, dev, "v")
    dt = k.dtype
    if Hk != Hkv or Dk != D or Tv != T or Hv != Hk or Dv != D or v.dtype is not dt:
        raise ValueError("k and v must have the cache's heads and columns, and the same dtype")
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    if kh != D or vh != D:
        raise ValueError("the heads of k and v must be adjacent")
    if kt == 0 or vt == 0:                   # to the C call that means contiguous rows
        raise ValueError("the tokens of k and v must be rows of their own")
    total = sq = cols = Hq = qt = 0
    qo = indptr = qp = qop = table = given = None
    if qo_indptr is not None:
        if k.dim() != 3:
            raise ValueError("packed k must be [total, heads, D]")
        qo = _ints_of(qo_indptr, dev, "qo_indptr", B + 1)
        total = T
    else:
        if k.shape[0] != B:
            raise ValueError("k must have one entry per request")
        sq = T // B if B else 0
    if block_tables is not None:
        if paged_kv_indptr is not None or paged_kv_indices is not None:
            raise ValueError("either block_tables or the CSR table")
        if block_tables.dim() != 2 or block_tables.shape[0] != B:
            raise ValueError("block_tables must be [B, C]")
        pages = _ints(block_tables, dev, "block_tables")
        cols = block_tables.shape[1]
    else:
        if paged_kv_indptr is None or paged_kv_indices is None:
            raise ValueError("a page table is needed")
        indptr = _ints_of(paged_kv_indptr, dev, "paged_kv_indptr", B + 1)
        pages = _ints(paged_kv_indices, dev, "paged_kv_indices")
    if q is not None:
        Tq, Hq, Dq, qt, qh = _rows(q, dev, "q")
        if Tq != T or Dq != D or q.dtype is not dt or qh != D or (qt == 0 and Hq > 0):
            raise ValueError("q must have k's tokens, columns and dtype, adjacent heads, and "
                             "tokens in rows of their own")
        if q_out is None:
            q_out = _empty(q, _BF16, stream)
        elif (q_out.shape != q.shape or q_out.dtype is not torch.bfloat16
              or not q_out.is_contiguous()):
            raise ValueError("q_out must be contiguous bf16 of q's shape")
        else:
            _on_device(q_out, dev, "q_out")
            given = q_out
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rotary = 0
    if freqs is not None:
        table, rotary = _table(freqs, dev), 2 * freqs.numel()
    lens = _ints(seq_lens_kv, dev, "seq_lens_kv")
    if status is not None:
        status = _status(status, dev)
    if T:
        rc = _call.paged_append_run(
            _append_params(B, sq, total, Hq, Hkv, D, ps, P, combined, cols, rotary,
                           ROPE_LAYOUT[layout], _factor(attention_factor), _DTYPE[dt], qt, kt, vt),
            qp, k.data_ptr(), v.data_ptr(), qo, indptr, pages, lens, table, qop, kc, vc, status,
            _stream(stream, dev))
        if rc:
            _check(rc, "paged_append_run")
        if given is not None:
            _increment_version(given)
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
        dev = _device()
        got = [_geometry(c, dev) for c in layers]
        if any(g[2:] != got[0][2:] for g in got):
            raise ValueError("the layers' pools must have the same shape")
        ptrs = [p for g in got for p in g[:2] if p is not None]
        if len(ptrs) > MAX_POOLS:
            raise ValueError(f"more than {MAX_POOLS} pools")
        self.layers, self.device_index = layers, dev
        _, _, combined, self.num_pages, Hkv, self.page_size, D = got[0]
        self._ptrs = (C.c_void_p * len(ptrs))(*ptrs)
        self.struct = CachePoolsStruct(num_layers=len(layers), num_pages=self.num_pages,
                                       num_kv_heads=Hkv, page_size=self.page_size, head_dim=D,
                                       combined_cache=combined, pools_host=self._ptrs)
        self._ref = C.byref(self.struct)

    def ref(self, dev):
        """The C struct, for a call on the current device."""
        if self.device_index != dev:
            raise ValueError("the pools are not on the current device")
        return self._ref


def cache_pools(layers) -> CachePools:
    """Handle of the layers' caches: combined caches [P, 2, Hkv, ps, D] or (K, V) pairs of
    pools [P, Hkv, ps, D], one per layer, all of one shape."""
    return CachePools(layers)


def _rows_state(block_tables, seq_lens, page_refs, page_size, dev, status=None):
    """(params, address of the tables, lengths, counts) of the three arrays."""
    shape = block_tables.shape
    if len(shape) != 2 or max(shape) > _INT_MAX:
        raise ValueError("block_tables must be [rows, C]")
    fields = shape[0], shape[1], operator.index(page_size), _count(page_refs, "page_refs")
    return (_cache_params(*fields) if status is None else
            C.byref(CacheParams(*fields, _status(status, dev))),
            _ints(block_tables, dev, "block_tables"),
            _ints_of(seq_lens, dev, "seq_lens", shape[0]), _ints(page_refs, dev, "page_refs"))


def free_cache_rows(rows, block_tables, seq_lens, page_refs, page_size, *, status=None,
                    stream=None) -> None:
    """Free the listed rows: their pages' counts go down by one, their lengths to 0."""
    dev = _device()
    p, bt, sl, pr = _rows_state(block_tables, seq_lens, page_refs, page_size, dev)
    rc = _call.paged_cache_free_run(p, _ints(rows, dev, "rows"), _count(rows, "rows"), bt, sl,
                                    pr,
                                    None if status is None else _status(status, dev),
                                    _stream(stream, dev))
    if rc:
        _check(rc, "paged_cache_free_run")


def extend_cache_workspace_size(n: int) -> int:
    return int(_call.paged_cache_extend_workspace_size(int(n)))


def extend_cache_rows(rows, new_tokens, block_tables, seq_lens, page_refs, page_size, *,
                      workspace=None, status=None, stream=None) -> None:
    """Make each listed row longer by new_tokens tokens, with fresh pages (the lowest free ids,
    in the order listed) where needed.

    Rows that the free pages do not suffice for stay as they are, their lengths too: appending
    to one would write over its last tokens.  `status`, an int32 word that findings are OR-ed
    into, tells (ERR_CAPACITY's bit 2, for items that broke the contract 4), and so does the
    workspace's word, which every call clears."""
    dev = _device()
    p, bt, sl, pr = _rows_state(block_tables, seq_lens, page_refs, page_size, dev, status)
    n = _count(rows, "rows")
    ws = _workspace(workspace, extend_cache_workspace_size, n, rows, dev, stream)
    rc = _call.paged_cache_extend_run(p, _ints(rows, dev, "rows"),
                                      _ints_of(new_tokens, dev, "new_tokens", n), n, bt, sl, pr,
                                      ws.data_ptr(), ws.nbytes, _stream(stream, dev))
    if rc:
        _check(rc, "paged_cache_extend_run")


def fork_cache_workspace_size(n: int) -> int:
    return int(_call.paged_cache_fork_workspace_size(int(n)))


def fork_cache_rows(pools, parents, children, block_tables, seq_lens, page_refs, *,
                    workspace=None, status=None, stream=None) -> None:
    """Make the (empty) row children[i] a copy of row parents[i]: full pages are shared, the
    live tokens of a partly filled last page are copied into a fresh one, in every layer.
    Children that the free pages do not suffice for stay empty; `status` and the workspace tell,
    as in extend_cache_rows."""
    dev = _device()
    p, bt, sl, pr = _rows_state(block_tables, seq_lens, page_refs, pools.page_size, dev, status)
    n = _count(children, "children")
    ws = _workspace(workspace, fork_cache_workspace_size, n, children, dev, stream)
    rc = _call.paged_cache_fork_run(p, pools.ref(dev), _ints_of(parents, dev, "parents", n),
                                    _ints(children, dev, "children"), n, bt, sl, pr,
                                    ws.data_ptr(), ws.nbytes, _stream(stream, dev))
    if rc:
        _check(rc, "paged_cache_fork_run")


def compact_cache_workspace_size(num_pages: int) -> int:
    return int(_call.paged_cache_compact_workspace_size(int(num_pages)))


def compact_cache(pools, block_tables, seq_lens, page_refs, *, block_tables_out=None,
                  page_refs_out=None, num_live=None, workspace=None, status=None, stream=None):
    """Move the live pages to the pools' front, in every layer; returns (block_tables, page_refs,
    num_live [1]) after the move.  In place unless the *_out tensors are given.  `status` and the
    workspace tell of bad table entries, as in extend_cache_rows."""
    dev = _device()
    p, bt, sl, pr = _rows_state(block_tables, seq_lens, page_refs, pools.page_size, dev, status)
    tables, refs, bto, pro = block_tables, page_refs, bt, pr
    if block_tables_out is not None:
        tables = block_tables_out
        if tables.shape != block_tables.shape:
            raise ValueError("block_tables_out must have block_tables' shape")
        bto = _ints(tables, dev, "block_tables_out")
    if page_refs_out is not None:
        refs = page_refs_out
        pro = _ints_of(refs, dev, "page_refs_out", page_refs.numel())
    if num_live is None:
        num_live = _new(1, _I32, page_refs.device, stream)
    ws = _workspace(workspace, compact_cache_workspace_size, page_refs.numel(), page_refs, dev,
                    stream)
    rc = _call.paged_cache_compact_run(p, pools.ref(dev), bt, sl, pr, bto, pro,
                                       _ints_of(num_live, dev, "num_live", 1), ws.data_ptr(),
                                       ws.nbytes, _stream(stream, dev))
    if rc:
        _check(rc, "paged_cache_compact_run")
    return tables, refs, num_live


def copy_cache_pages(pools, src_pages, dst_pages, *, dst_pools=None, status=None,
                     stream=None) -> None:
    """Copy page src_pages[i] to page dst_pages[i] in every layer, within `pools` or to the same
    layers of `dst_pools`."""
    dev = _device()
    src = pools.ref(dev)
    n = _count(src_pages, "src_pages")
    rc = _call.paged_cache_copy_run(src, src if dst_pools is None else dst_pools.ref(dev),
                                    _ints(src_pages, dev, "src_pages"),
                                    _ints_of(dst_pages, dev, "dst_pages", n), n,
                                    None if status is None else _status(status, dev),
                                    _stream(stream, dev))
    if rc:
        _check(rc, "paged_cache_copy_run")


__all__ = ["rope_frequencies", "rotary_embedding", "append_paged_kv_cache", "CachePools",
           "cache_pools", "free_cache_rows", "extend_cache_rows", "extend_cache_workspace_size",
           "fork_cache_rows", "fork_cache_workspace_size", "compact_cache",
           "compact_cache_workspace_size", "copy_cache_pages", "RopeScaling", "RopeParams",
           "AppendParams", "CacheParams", "CachePoolsStruct"]
