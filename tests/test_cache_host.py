"""CPU checks of the cache side: frequencies and the fixed-point table against exact arithmetic,
the oracle's pins, workspace sizes, and the refusals of the C entry points and of the binding.
No call here reaches a launch: every refused call returns before anything is enqueued, so the
placeholder addresses are never used."""
import ctypes as C
import math
import random
from decimal import Decimal

import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import cache as O
from paged_kv_block_gb300 import build as B
from paged_kv_block_gb300 import cache as K

A16 = 0x7F0000100000
BAD = pkb.ERR_INVALID_ARGUMENT


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pkb.lib()


def _turns(table):
    return [int(v) % (1 << 64) for v in table.tolist()]


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "wavelength"])
@pytest.mark.parametrize("rotary_dim", [2, 20, 64, 128])
def test_frequencies_match_their_formula(lib, scaling, rotary_dim):
    kw = dict(base=10000.0, scaling=scaling, factor=8.0)
    s = K.RopeScaling(rotary_dim=rotary_dim, kind=K.ROPE_SCALING[scaling], base=10000.0,
                      factor=8.0, original_max_position=4096.0)
    got, m = (C.c_double * (rotary_dim // 2))(), C.c_float()
    assert lib.paged_rope_frequencies(C.byref(s), got, C.byref(m)) == 0
    want, wm = O.frequencies(rotary_dim, original=4096.0, **kw)
    # a handful of float64 roundings and a pow on either side
    np.testing.assert_allclose(list(got), want, rtol=1e-13)
    assert m.value == pytest.approx(wm, abs=1e-7)


def test_scalings_keep_fast_pairs_and_slow_down_slow_ones(lib):
    plain, _ = O.frequencies(128)
    for scaling in ("yarn", "wavelength"):
        f, _ = O.frequencies(128, scaling=scaling, factor=8.0, original=8192.0)
        assert f[0] == plain[0]                              # one radian per position: kept
        assert f[-1] == pytest.approx(plain[-1] / 8, rel=1e-12)
        assert (np.diff(f / plain) <= 1e-15).all()           # ever slower towards the last pair
    f, _ = O.frequencies(128, scaling="ntk", factor=8.0)
    assert f[0] == 1.0 and f[-1] == pytest.approx(plain[-1] / 8, rel=1e-12)


def test_table_is_the_nearest_fraction_of_a_turn(lib):
    r = random.Random(3)
    f = [1.0, 0.5, 1e-4, 2 * math.pi, 7.0, 100.25, -0.3, 0.0, 1e-300, 1048576.0]
    f += [10000.0 ** -r.random() for _ in range(54)]
    table, _ = pkb.rope_frequencies(2 * len(f), inv_freq=f, device="cpu")
    for x, got in zip(f, _turns(table)):
        exact = Decimal(x) / (2 * O.PI) * (1 << 64)
        off = abs(Decimal(got) - exact) % (1 << 64)
        off = min(off, (1 << 64) - off)
        # half a unit of 2^-64, and the error of 1 / (2 pi) as two doubles (2^-106 of the value)
        assert off <= Decimal("0.5001") + abs(exact) * Decimal(2) ** -104, (x, off)


def test_table_refuses_what_it_cannot_hold(lib):
    for bad in (float("inf"), float("nan"), 2.0 ** 21):
        with pytest.raises(pkb.PagedAttnError):
            pkb.rope_frequencies(2, inv_freq=[bad], device="cpu")
    with pytest.raises(ValueError):
        pkb.rope_frequencies(4, inv_freq=[1.0], device="cpu")
    for kw in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=514),
               dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, scaling="linear", factor=0.0),
               dict(rotary_dim=8, scaling="yarn", factor=2.0),
               dict(rotary_dim=8, scaling="wavelength", factor=2.0, original_max_position=100.0,
                    low=4.0, high=1.0)):
        with pytest.raises(pkb.PagedAttnError):
            pkb.rope_frequencies(kw.pop("rotary_dim"), device="cpu", **kw)


# ---- pins of the oracle -------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_oracle_rotation_pins(layout):
    rng = np.random.RandomState(0)
    f, _ = O.frequencies(8)
    x = rng.randn(3, 2, 12)
    # position 0 is the identity, lengths of pairs stay, the inverse undoes, and q . k depends on
    # the distance of the positions only
    y, _ = O.rotate(x, [0, 0, 0], f, layout=layout)
    assert np.array_equal(y, x)
    y, _ = O.rotate(x, [5, -7, 2 ** 31 - 1], f, layout=layout)
    np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-13)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    back, _ = O.rotate(y, [5, -7, 2 ** 31 - 1], f, layout=layout, inverse=True)
    np.testing.assert_allclose(back, x, rtol=0, atol=1e-14)
    q, k = x[:1, :1, :8], x[1:2, :1, :8]
    dots = [(O.rotate(q, [p + 11], f, layout=layout)[0] * O.rotate(k, [p], f, layout=layout)[0]).sum()
            for p in (0, 100, 10 ** 6)]
    np.testing.assert_allclose(dots, dots[0], rtol=0, atol=1e-12)
    # one pair at one radian per position, by hand
    one, _ = O.rotate(np.array([[[1.0, 0.0]]]), [1], [1.0], layout=layout)
    np.testing.assert_allclose(one.ravel(), [math.cos(1), math.sin(1)], rtol=1e-15)


def test_oracle_page_state_keeps_its_invariants():
    """Random calls: every count equals the live entries that name the page, a partly filled
    page has one owner, and what a row reads never changes but by its own calls."""
    rng = random.Random(5)
    ps, P, R, Ccols = 8, 40, 6, 12
    pool = np.arange(P * ps, dtype=np.int64).reshape(P, 1, ps, 1)
    s = O.State([[-1] * Ccols for _ in range(R)], [0] * R, [0] * P, ps, [pool])
    held = [[] for _ in range(R)]
    stamp = 0
    for step in range(400):
        op = rng.choice(["extend", "free", "fork", "compact"])
        r = rng.randrange(R)
        if op == "extend":
            m = rng.randrange(20)
            n = s.lens[r]
            s.extend([r], [m])
            for t in range(n, s.lens[r]):
                stamp += 1
                s.pools[0][s.tables[r][t // ps], 0, t % ps, 0] = stamp
                held[r].append(stamp)
        elif op == "free":
            s.free([r, r])
            held[r] = []
        elif op == "fork":
            c = rng.randrange(R)
            if s.lens[c] == 0 and c != r:
                s.fork([r], [c])
                if s.lens[c]:
                    held[c] = list(held[r])
        else:
            live = s.compact()
            assert all(x > 0 for x in s.refs[:live]) and not any(s.refs[live:])
        count = [0] * P
        for i in range(R):
            used = s.tables[i][:s.pages(s.lens[i])]
            for j, p in enumerate(used):
                count[p] += 1
                if j == len(used) - 1 and s.lens[i] % ps:
                    assert s.refs[p] == 1
            assert [int(s.pools[0][used[t // ps], 0, t % ps, 0]) for t in range(s.lens[i])] == held[i]
        assert count == s.refs


# ---- refusals ---------------------------------------------------------------------------------

def _rope(lib, q=A16, k=A16, pos=A16, table=A16, qo=A16, ko=A16, **kw):
    f = dict(num_tokens=4, num_qo_heads=4, num_kv_heads=2, head_dim=64, rotary_dim=64, layout=0,
             dtype=0, inverse=0, attention_factor=1.0)
    f.update(kw)
    return lib.paged_rope_run(C.byref(K.RopeParams(**f)), q, k, pos, table, qo, ko, None, None)


def test_rope_refusals(lib):
    for kw in (dict(num_tokens=-1), dict(num_qo_heads=0), dict(num_kv_heads=-1),
               dict(head_dim=60), dict(head_dim=0), dict(head_dim=520), dict(rotary_dim=0),
               dict(rotary_dim=7), dict(rotary_dim=66), dict(layout=2), dict(dtype=3),
               dict(attention_factor=float("nan")), dict(attention_factor=float("inf")),
               dict(pos=A16 + 2), dict(table=A16 + 4), dict(q=None), dict(qo=None), dict(pos=None), dict(table=None), dict(k=None),
               dict(ko=None), dict(num_kv_heads=0), dict(q=A16 + 1), dict(ko=A16 + 1),
               dict(dtype=2, q=A16 + 2), dict(q_token_stride=512, q_head_stride=64),
               dict(k_token_stride=512, k_head_stride=64), dict(num_qo_heads=65535)):
        assert _rope(lib, **kw) == BAD, kw
    assert _rope(lib, num_tokens=0) == 0
    assert _rope(lib, num_tokens=0, num_kv_heads=0, k=None, ko=None) == 0


def test_rope_refuses_outputs_whose_rows_overlap(lib):
    # (token stride, head stride) of 4 tokens of 4 heads (q) or 2 heads (k) of 64 columns
    for ts, hs in ((256, 0), (0, 64), (64, 64), (192, 64), (256, 63), (63, 256), (64, 255)):
        assert _rope(lib, qo=2 * A16, q_out_token_stride=ts, q_out_head_stride=hs) == BAD
        # in place, the input's rows are the output's
        assert _rope(lib, q_token_stride=ts, q_head_stride=hs, q_out_token_stride=ts,
                     q_out_head_stride=hs) == BAD
    for ts, hs in ((128, 0), (0, 64), (64, 64), (127, 64), (64, 255)):
        assert _rope(lib, ko=2 * A16, k_out_token_stride=ts, k_out_head_stride=hs) == BAD


def _append(lib, q=A16, k=A16, v=A16, qo=None, indptr=None, pages=A16, lens=A16, table=A16,
            qout=A16, kc=A16, vc=None, status=None, **kw):
    f = dict(batch=2, seq_len_q=1, total_q=0, num_qo_heads=4, num_kv_heads=2, head_dim=64,
             page_size=16, num_pages=10, combined_cache=1, max_pages_per_request=4, rotary_dim=64,
             layout=0, attention_factor=1.0, in_dtype=0)
    f.update(kw)
    return lib.paged_append_run(C.byref(K.AppendParams(**f)), q, k, v, qo, indptr, pages, lens,
                                table, qout, kc, vc, status, None)


def test_append_refusals(lib):
    for kw in (dict(batch=-1), dict(seq_len_q=-1), dict(num_qo_heads=-1), dict(num_kv_heads=0),
               dict(head_dim=12), dict(page_size=12), dict(page_size=136), dict(num_pages=0),
               dict(max_pages_per_request=0), dict(rotary_dim=5), dict(rotary_dim=-2),
               dict(rotary_dim=66), dict(layout=-1), dict(in_dtype=7), dict(k=None), dict(v=None),
               dict(q=None), dict(qout=None), dict(pages=None), dict(lens=None), dict(kc=None),
               dict(table=None), dict(vc=A16), dict(combined_cache=0), dict(kc=A16 + 8),
               dict(combined_cache=0, vc=A16 + 8), dict(qout=A16 + 8), dict(k=A16 + 1),
               dict(attention_factor=float("inf")), dict(num_qo_heads=0), dict(table=A16 + 4),
               dict(pages=A16 + 2), dict(lens=A16 + 1), dict(status=A16 + 2), dict(qo=A16 + 2),
               dict(indptr=A16 + 2),
               dict(batch=1 << 20, seq_len_q=1 << 12), dict(qo=A16, total_q=-1)):
        assert _append(lib, **kw) == BAD, kw
    assert _append(lib, batch=0) == 0
    assert _append(lib, seq_len_q=0) == 0
    assert _append(lib, qo=A16, total_q=0) == 0
    assert _append(lib, rotary_dim=0, table=None, batch=0) == 0


def _params(**kw):
    f = dict(rows=4, max_pages_per_request=8, page_size=16, num_pages=32)
    f.update(kw)
    return K.CacheParams(**f)


def _pool_struct(ptrs=(A16,), **kw):
    a = (C.c_void_p * max(len(ptrs), 1))(*ptrs)
    f = dict(num_layers=len(ptrs), num_pages=32, num_kv_heads=2, page_size=16, head_dim=64,
             combined_cache=1, pools_host=a)
    f.update(kw)
    s = K.CachePoolsStruct(**f)
    s.keep = a
    return s


BAD_STATE = [dict(rows=-1), dict(max_pages_per_request=0), dict(page_size=4), dict(page_size=20),
             dict(num_pages=0), dict(num_pages=(1 << 24) + 1)]
BAD_POOLS = [dict(num_layers=0), dict(num_layers=257), dict(num_kv_heads=0), dict(head_dim=4),
             dict(head_dim=520), dict(page_size=12), dict(num_pages=0), dict(ptrs=(None,)),
             dict(ptrs=(A16 + 8,)), dict(pools_host=None), dict(combined_cache=0, num_layers=129),
             dict(num_kv_heads=16384, page_size=128, head_dim=512)]


def test_page_call_refusals(lib):
    big = 1 << 30
    for kw in BAD_STATE:
        p = _params(**kw)
        assert lib.paged_cache_free_run(C.byref(p), A16, 1, A16, A16, A16, None, None) == BAD
        assert lib.paged_cache_extend_run(C.byref(p), A16, A16, 1, A16, A16, A16, A16, big, None) == BAD
    p = _params()
    for i in range(4):
        for bad in (None, A16 + 2):
            a = [A16] * 4
            a[i] = bad
            assert lib.paged_cache_free_run(C.byref(p), a[0], 1, a[1], a[2], a[3], None, None) == BAD
    for i in range(5):
        for bad in (None, A16 + 2):
            a = [A16] * 5
            a[i] = bad
            assert lib.paged_cache_extend_run(C.byref(p), a[0], a[1], 1, a[2], a[3], a[4], A16, big,
                                              None) == BAD
    assert lib.paged_cache_extend_run(C.byref(p), *[A16] * 2, 1, *[A16] * 3, A16 + 4, big, None) == BAD
    assert lib.paged_cache_free_run(C.byref(p), A16, -1, A16, A16, A16, None, None) == BAD
    assert lib.paged_cache_free_run(C.byref(p), None, 0, None, None, None, None, None) == 0
    for n in (-1, 4097):
        assert lib.paged_cache_extend_run(C.byref(p), A16, A16, n, A16, A16, A16, A16, big, None) == BAD
        assert lib.paged_cache_fork_run(C.byref(p), C.byref(_pool_struct()), A16, A16, n, A16, A16,
                                        A16, A16, big, None) == BAD
        assert pkb.extend_cache_workspace_size(n) == 0 and pkb.fork_cache_workspace_size(n) == 0
    need = pkb.extend_cache_workspace_size(3)
    for ws, n in ((None, big), (A16, need - 1)):
        assert lib.paged_cache_extend_run(C.byref(p), A16, A16, 3, A16, A16, A16, ws, n,
                                          None) == pkb.ERR_WORKSPACE
    s = _pool_struct()
    fork = lib.paged_cache_fork_run
    for kw in BAD_POOLS:
        assert fork(C.byref(p), C.byref(_pool_struct(**kw)), A16, A16, 1, A16, A16, A16, A16, big,
                    None) == BAD, kw
        assert lib.paged_cache_copy_run(C.byref(_pool_struct(**kw)), C.byref(s), A16, A16, 1, None,
                                        None) == BAD
    for kw in (dict(num_pages=31), dict(page_size=32)):
        t = _pool_struct(**kw)
        assert fork(C.byref(p), C.byref(t), A16, A16, 1, A16, A16, A16, A16, big, None) == BAD
        assert lib.paged_cache_compact_run(C.byref(p), C.byref(t), A16, A16, A16, A16, A16, A16,
                                           A16, big, None) == BAD
    assert fork(C.byref(p), C.byref(s), A16, A16, 2, A16, A16, A16, A16, 16, None) == pkb.ERR_WORKSPACE
    for kw in (dict(page_size=32), dict(head_dim=128), dict(num_kv_heads=4), dict(ptrs=(A16, A16))):
        assert lib.paged_cache_copy_run(C.byref(s), C.byref(_pool_struct(**kw)), A16, A16, 1, None,
                                        None) == BAD
    assert lib.paged_cache_copy_run(C.byref(s), C.byref(s), None, None, 0, None, None) == 0
    assert lib.paged_cache_copy_run(C.byref(s), C.byref(s), A16, None, 1, None, None) == BAD
    # compact: outputs are their inputs or do not overlap them
    def compact(bt=A16, ln=A16, rf=A16, bto=A16, rfo=A16, live=A16, ws=A16, n=big):
        return lib.paged_cache_compact_run(C.byref(p), C.byref(s), bt, ln, rf, bto, rfo, live, ws, n,
                                           None)
    for kw in (dict(bt=None), dict(ln=None), dict(rf=None), dict(bto=None), dict(rfo=None),
               dict(live=None), dict(bto=A16 + 16), dict(rfo=A16 + 64), dict(live=A16 + 2),
               dict(ws=A16 + 8)):
        assert compact(**kw) == BAD, kw
    for kw in (dict(ws=None), dict(n=pkb.compact_cache_workspace_size(32) - 1)):
        assert compact(**kw) == pkb.ERR_WORKSPACE


def test_workspace_sizes(lib):
    assert pkb.extend_cache_workspace_size(-1) == 0 and pkb.fork_cache_workspace_size(-1) == 0
    assert 0 < pkb.extend_cache_workspace_size(0) <= pkb.extend_cache_workspace_size(1000)
    assert pkb.compact_cache_workspace_size(0) == 0
    assert pkb.compact_cache_workspace_size((1 << 24) + 1) == 0
    assert pkb.compact_cache_workspace_size(1000) >= 3 * 4000


def test_binding_refuses_host_tensors(lib):
    q, pos = torch.zeros(2, 1, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkb.rotary_embedding(q, pos, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        pkb.append_paged_kv_cache(q, q, torch.zeros(1, 2, 1, 8, 8, dtype=torch.bfloat16), pos,
                                  block_tables=pos.view(2, 1))
    with pytest.raises(ValueError):
        pkb.cache_pools([torch.zeros(1, 2, 1, 8, 8, dtype=torch.bfloat16)])
    with pytest.raises(ValueError):
        pkb.cache_pools([])
    with pytest.raises(ValueError):
        pkb.free_cache_rows(pos, pos.view(2, 1), pos, pos, 16)


# ---- what the binding hands to the C entry points -----------------------------------------------

class _Recorder:
    """In place of the library: keeps the parameters of the last call."""

    def __init__(self):
        self.params = None

    def __getattr__(self, name):
        def call(params, *rest):
            self.params = params._obj
            return 0
        return call


@pytest.fixture
def recorded(monkeypatch):
    """The binding on host tensors (their device index is -1), with the library out of reach."""
    r = _Recorder()
    monkeypatch.setattr(K, "_device", lambda: -1)
    monkeypatch.setattr(K, "_stream", lambda stream, dev: 0)
    monkeypatch.setattr(K, "_call", r)
    return r


def test_rope_rows_that_step_by_nothing(recorded):
    pos, table = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)

    def rope(q, **kw):
        recorded.params = None
        pkb.rotary_embedding(q, pos[:q.numel() // (q.shape[-1] * q.shape[-2])], table, **kw)
        return recorded.params

    # two strides of zero mean packed rows to the C call, which would read past a single row
    one = torch.zeros(8)
    for shape in ((3, 2, 8), (1, 3, 2, 8)):
        for kw in (dict(q=one.expand(shape)), dict(q=torch.zeros(shape), k=one.expand(shape)),
                   dict(q=torch.zeros(shape), q_out=one.expand(shape)),
                   dict(q=torch.zeros(shape), k=torch.zeros(shape), k_out=one.expand(shape))):
            with pytest.raises(ValueError):
                rope(**kw)
            assert recorded.params is None
    # a single head or token has no step, whatever its stride says
    p = rope(torch.as_strided(one, (3, 1, 8), (0, 0, 1)))
    assert (p.q_token_stride, p.q_head_stride) == (0, 8)
    p = rope(torch.as_strided(one, (1, 2, 8), (0, 0, 1)))
    assert (p.q_token_stride, p.q_head_stride) == (16, 0)
    p = rope(torch.as_strided(torch.zeros(24), (3, 1, 8), (8, 5, 1)))
    assert (p.q_token_stride, p.q_head_stride) == (8, 8)


def test_append_rows_that_step_by_nothing(recorded):
    cache = torch.zeros(4, 2, 2, 8, 8, dtype=torch.bfloat16)
    table = torch.zeros(3, 2, dtype=torch.int32)
    lens = torch.ones(3, dtype=torch.int32)
    row, full = torch.zeros(1, 2, 8), torch.zeros(3, 2, 8)
    for k, v, q in ((row.expand(3, 2, 8), full, full), (full, row.expand(3, 2, 8), full),
                    (full, full, row.expand(3, 2, 8))):
        recorded.params = None
        with pytest.raises(ValueError):
            pkb.append_paged_kv_cache(k, v, cache, lens, block_tables=table, q=q)
        assert recorded.params is None
    pkb.append_paged_kv_cache(row, row, cache, lens[:1], block_tables=table[:1])
    assert recorded.params.k_token_stride in (0, 16)


def test_what_a_call_allocates_belongs_to_its_stream(recorded, monkeypatch):
    # A workspace goes back to the allocator when the call returns, while its kernels may still
    # run: it has to come from the pool of the stream that they run on.
    current, seen = [], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()

    def spy(make):
        def call(*a, **kw):
            seen.append(current[-1] if current else None)
            return make(*a, **kw)
        return call

    class Sizes(_Recorder):
        def __getattr__(self, name):
            return (lambda n: 64) if name.endswith("_size") else super().__getattr__(name)

    cache = torch.zeros(4, 2, 2, 8, 8, dtype=torch.bfloat16)
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32)
    q, t = torch.zeros(3, 2, 8), torch.zeros(4, dtype=torch.int64)
    pools = pkb.cache_pools([cache])
    monkeypatch.setattr(K, "_call", Sizes())
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch, "empty", spy(torch.empty))
    monkeypatch.setattr(torch, "empty_like", spy(torch.empty_like))
    state = (i32(3, 2), i32(3), i32(4))
    for made, call in (
            (1, lambda s: pkb.rotary_embedding(q, i32(3), t, stream=s)),
            (2, lambda s: pkb.rotary_embedding(q, i32(3), t, k=q.transpose(0, 1).contiguous()
                                               .transpose(0, 1), stream=s)),
            (1, lambda s: pkb.append_paged_kv_cache(q, q, cache, i32(3), q=q, stream=s,
                                                    block_tables=i32(3, 2))),
            (1, lambda s: pkb.extend_cache_rows(i32(2), i32(2), *state, 8, stream=s)),
            (1, lambda s: pkb.fork_cache_rows(pools, i32(2), i32(2), *state, stream=s)),
            (2, lambda s: pkb.compact_cache(pools, *state, stream=s))):
        for stream in (None, "side"):
            seen.clear()
            call(stream)
            assert seen == [stream] * made
