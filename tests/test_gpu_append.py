"""Appending to the paged cache on the GPU against the float64 oracle: which slots are written, with
what, and that nothing else is."""
import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import cache as O
from tests.test_gpu_rope import close

pytestmark = pytest.mark.gpu
DEV = "cuda"


def problem(seed, new, prefix, *, Hq=4, Hkv=2, D=64, ps=16, combined=False, dtype=torch.bfloat16,
            pad=0, spare=3):
    """Packed rows of `new[b]` tokens behind `prefix[b]` cached ones, shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    lens = [n + p for n, p in zip(new, prefix)]
    need = [-(-L // ps) for L in lens]
    P, B = sum(need) + spare, len(new)
    perm = torch.randperm(P, generator=g).tolist()
    C = max(need + [1]) + 1
    tables = torch.full((B, C), P + 1000, dtype=torch.int32)      # dead entries: never read
    for b in range(B):
        for j in range(need[b]):
            tables[b, j] = perm.pop()
    total = sum(new) + pad
    fused = torch.randn(total, Hq + 2 * Hkv, D, generator=g).to(dtype).to(DEV)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
    shape = (P, 2, Hkv, ps, D) if combined else (2, P, Hkv, ps, D)
    cache = torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)
    return dict(q=fused[:, :Hq], k=fused[:, Hq:Hq + Hkv], v=fused[:, Hq + Hkv:],
                qo=torch.tensor(starts, dtype=torch.int32, device=DEV), starts=starts,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), tables=tables.to(DEV),
                cache=cache, combined=combined, ps=ps, P=P, D=D, Hkv=Hkv)


def kv(s, cache=None):
    """(K, V) views [P, Hkv, ps, D] of the problem's cache."""
    c = s["cache"] if cache is None else cache
    return (c[:, 0], c[:, 1]) if s["combined"] else (c[0], c[1])


def check(s, out, before, freqs, *, layout="half", m=1.0, q_before=None):
    lens, tables = s["lens"].tolist(), s["tables"].tolist()
    where, positions = O.append(s["k"], s["v"], lens, tables, s["ps"], s["P"], starts=s["starts"])
    owned = [t for t, p in enumerate(positions) if p is not None]
    pos = [p if p is not None else 0 for p in positions]
    f = freqs if freqs is not None else np.zeros(0)
    want_k, size_k = O.rotate(s["k"], pos, f, layout=layout, m=m)
    want_v = s["v"].double().cpu().numpy()
    K, V = kv(s)
    t, page, slot = (np.array(x, dtype=np.int64) for x in zip(*where)) if where else (np.zeros(0, np.int64),) * 3
    ti, pi, si = (torch.from_numpy(x).to(DEV) for x in (t, page, slot))
    close(K[pi, :, si], want_k[t], size_k[t])
    zero = np.zeros_like(want_v[t])
    close(V[pi, :, si], want_v[t], zero)
    if s["v"].dtype == torch.bfloat16:
        assert torch.equal(V[pi, :, si], s["v"][ti])
    # nothing but those slots has changed
    bk, bv = kv(s, before)
    mask = torch.ones(s["P"], s["ps"], dtype=torch.bool, device=DEV)
    mask[pi, si] = False
    for new, old in ((K, bk), (V, bv)):
        assert torch.equal(new.transpose(1, 2)[mask], old.transpose(1, 2)[mask])
    if out is not None:
        want_q, size_q = O.rotate(s["q"], pos, f, layout=layout, m=m)
        close(out[owned], want_q[owned], size_q[owned], torch.bfloat16)
        if q_before is not None:
            rest = [t for t in range(len(positions)) if positions[t] is None]
            assert torch.equal(out[rest], q_before[rest])


def table_args(s, csr):
    if not csr:
        return dict(block_tables=s["tables"])
    B, C = s["tables"].shape
    return dict(paged_kv_indptr=torch.arange(B + 1, dtype=torch.int32, device=DEV) * C,
                paged_kv_indices=s["tables"].flatten())


def cache_arg(s):
    return s["cache"] if s["combined"] else (s["cache"][0], s["cache"][1])


@pytest.mark.parametrize("combined,csr", [(False, False), (True, True), (True, False), (False, True)])
@pytest.mark.parametrize("ps", [16, 24, 128])
@pytest.mark.parametrize("layout,R", [("half", 64), ("interleaved", 64), ("half", 20), (None, 0)])
def test_packed(combined, csr, ps, layout, R):
    s = problem(ps + R, [1, 17, 0, 40, 130], [300, 0, 25, 15, 0], ps=ps, combined=combined)
    before = s["cache"].clone()
    table = f = None
    if R:
        table, _ = pkb.rope_frequencies(R)
        f, _ = O.frequencies(R)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pkb.append_paged_kv_cache(s["k"], s["v"], cache_arg(s), s["lens"], q=s["q"],
                                    qo_indptr=s["qo"], freqs=table, layout=layout or "half",
                                    status=status, **table_args(s, csr))
    check(s, out, before, f, layout=layout or "half")
    assert status.item() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,R,layout", [(128, 128, "half"), (256, 64, "interleaved"),
                                        (80, 30, "half"), (8, 6, "interleaved")])
def test_types_and_head_sizes(dtype, D, R, layout):
    s = problem(D, [3, 20], [30, 0], D=D, dtype=dtype, combined=True, Hq=5, Hkv=1)
    before = s["cache"].clone()
    table, m = pkb.rope_frequencies(R, scaling="yarn", factor=4.0, original_max_position=2048)
    f, wm = O.frequencies(R, scaling="yarn", factor=4.0, original=2048.0)
    out = pkb.append_paged_kv_cache(s["k"], s["v"], cache_arg(s), s["lens"], q=s["q"],
                                    qo_indptr=s["qo"], freqs=table, layout=layout,
                                    attention_factor=m, block_tables=s["tables"])
    check(s, out, before, f, layout=layout, m=wm)


@pytest.mark.parametrize("SQ", [1, 4])
@pytest.mark.parametrize("B", [1, 3, 70])
def test_fixed_form(B, SQ):
    """[B, heads, D] and [B, SQ, heads, D] rows: the layouts of decode attention."""
    s = problem(B * 10 + SQ, [SQ] * B, [(37 * b) % 90 for b in range(B)], combined=True)
    before = s["cache"].clone()
    table, _ = pkb.rope_frequencies(64)
    f, _ = O.frequencies(64)

    def shaped(x):
        return x if SQ == 1 else x.unflatten(0, (B, SQ))
    out = pkb.append_paged_kv_cache(shaped(s["k"]), shaped(s["v"]), cache_arg(s), s["lens"],
                                    q=shaped(s["q"]), freqs=table, **table_args(s, True))
    assert out.shape == shaped(s["q"]).shape
    check(s, out.reshape(B * SQ, -1, 64), before, f)


@pytest.mark.parametrize("many", [31, 32, 33, 700, 1025, 40000])
def test_without_queries_and_many_requests(many):
    """K and V alone; up to more requests than a warp finds in three steps, most of them with one
    token, some with none."""
    new = [0] + [1] * many + [0, 0, 300, 2, 0]
    s = problem(5, new, [b % 20 for b in range(len(new))], Hq=1, Hkv=1, D=8, ps=8)
    before = s["cache"].clone()
    table, _ = pkb.rope_frequencies(8)
    assert pkb.append_paged_kv_cache(s["k"], s["v"], cache_arg(s), s["lens"], qo_indptr=s["qo"],
                                     freqs=table, block_tables=s["tables"]) is None
    check(s, None, before, O.frequencies(8)[0])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,D,R", [(32, 8, 128, 128), (0, 1, 80, 40), (4, 2, 256, 64), (3, 3, 64, 20),
                                        (7, 1, 8, 0)])
def test_long_calls_equal_short_ones(layout, dtype, Hq, Hkv, D, R):
    """Many tokens in one call give the bits of calls with one request each."""
    s = problem(D, [1300, 1, 0, 1250], [70, 3, 40, 0], Hq=max(Hq, 1), Hkv=Hkv, D=D, dtype=dtype,
                combined=True)
    table = pkb.rope_frequencies(R)[0] if R else None
    one = s["cache"].clone()
    q = s["q"] if Hq else None
    out = pkb.append_paged_kv_cache(s["k"], s["v"], s["cache"], s["lens"], q=q, qo_indptr=s["qo"],
                                    freqs=table, layout=layout, block_tables=s["tables"])
    for b, (a, e) in enumerate(zip(s["starts"][:-1], s["starts"][1:])):
        zero = torch.tensor([0, e - a], dtype=torch.int32, device=DEV)
        part = pkb.append_paged_kv_cache(s["k"][a:e], s["v"][a:e], one, s["lens"][b:b + 1],
                                         q=None if q is None else q[a:e], qo_indptr=zero,
                                         freqs=table, layout=layout,
                                         block_tables=s["tables"][b:b + 1].contiguous())
        assert q is None or torch.equal(part, out[a:e])
    assert torch.equal(one.view(torch.int16), s["cache"].view(torch.int16))
    # rows that do not lie in one run
    kc, vc, qc = s["k"].contiguous(), s["v"].contiguous(), None if q is None else q.contiguous()
    for kk, vv, qq in ((kc, vc, qc), (kc, s["v"], q), (s["k"], vc, qc)):
        one.fill_(1.0)
        part = pkb.append_paged_kv_cache(kk, vv, one, s["lens"], q=qq, qo_indptr=s["qo"],
                                         freqs=table, layout=layout, block_tables=s["tables"])
        assert q is None or torch.equal(part, out)
        same = one == s["cache"]
        assert (same | (one == 1.0)).all()
    assert same.sum() >= 2 * s["k"].numel()


@pytest.mark.parametrize("big", [False, True])
def test_padding_rows_are_left_alone(big):
    """Rows behind the last request: nothing of q_out or of the cache is written for them."""
    new = [900, 800, 1000] if big else [5, 9]
    s = problem(11, new, [0] * len(new), pad=13, Hq=2, Hkv=1, D=16)
    before = s["cache"].clone()
    table, _ = pkb.rope_frequencies(16)
    mark = torch.full(s["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV)
    q_out = mark.clone()
    pkb.append_paged_kv_cache(s["k"], s["v"], cache_arg(s), s["lens"], q=s["q"], q_out=q_out,
                              qo_indptr=s["qo"], freqs=table, block_tables=s["tables"])
    check(s, q_out, before, O.frequencies(16)[0], q_before=mark)


def test_bad_pages_and_lengths_are_reported_and_skipped():
    """Page ids outside the pool, a length that outgrows the table, and more new tokens than the
    length counts: those tokens write nothing into the cache, all others do."""
    s = problem(12, [20, 20, 20, 4], [0, 0, 10, 0], combined=True)
    s["tables"][0, 1] = -1
    s["tables"][1, 0] = s["P"]
    s["lens"][2] = s["tables"].shape[1] * s["ps"] + 5
    s["lens"][3] = 2
    before = s["cache"].clone()
    table, _ = pkb.rope_frequencies(64)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    # row 2 grew past its live entries: give it real pages up to the table's end
    s["tables"][2] = s["tables"][2, 0]
    spare = sorted(set(range(s["P"])) - set(s["tables"].flatten().tolist()))
    s["tables"][2, -2:] = torch.tensor(spare[:2], dtype=torch.int32)
    out = pkb.append_paged_kv_cache(s["k"], s["v"], cache_arg(s), s["lens"], q=s["q"],
                                    qo_indptr=s["qo"], freqs=table, block_tables=s["tables"],
                                    status=status)
    check(s, out, before, O.frequencies(64)[0])
    assert status.item() == O.METADATA
    # the word is OR-ed into, never cleared
    status.fill_(8)
    pkb.append_paged_kv_cache(s["k"], s["v"], cache_arg(s), s["lens"], q=s["q"], qo_indptr=s["qo"],
                              freqs=table, block_tables=s["tables"], status=status)
    assert status.item() == 8 | O.METADATA


def test_far_part_of_a_large_pool():
    """A page whose elements lie past 2^32 bytes and 2^31 elements of the pool."""
    P, Hkv, ps, D = 70000, 1, 128, 256
    cache = torch.zeros(P, 2, Hkv, ps, D, dtype=torch.bfloat16, device=DEV)      # 9.2 GB
    g = torch.Generator().manual_seed(3)
    k = torch.randn(2, 1, D, generator=g).to(torch.bfloat16).to(DEV)
    tables = torch.tensor([[P - 1], [40000]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([128, 1], dtype=torch.int32, device=DEV)
    pkb.append_paged_kv_cache(k, k + 1, cache, lens, block_tables=tables)
    assert torch.equal(cache[P - 1, 0, :, 127], k[0]) and torch.equal(cache[40000, 0, :, 0], k[1])
    assert torch.equal(cache[P - 1, 1, :, 127], k[0] + 1)
    assert cache[P - 1].ne(0).sum() <= 2 * D and cache[:10].eq(0).all()


def test_graph_replay_follows_the_lengths():
    """A captured decode step: the lengths advance on the device between replays."""
    s = problem(13, [1, 1, 1], [14, 15, 30], combined=True)
    table, _ = pkb.rope_frequencies(64)
    q_out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)

    def step():
        pkb.append_paged_kv_cache(s["k"], s["v"], s["cache"], s["lens"], q=s["q"], q_out=q_out,
                                  freqs=table, block_tables=s["tables"])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    s["lens"].sub_(1)                 # positions that the live pages hold
    before = s["cache"].clone()
    graph.replay()
    check(s, q_out, before, O.frequencies(64)[0])


def test_two_streams_at_once():
    """Long calls on two streams, each into its own cache."""
    ss = [problem(30 + k, [900, 1, 1200], [3, 50, 0], combined=True) for k in range(2)]
    table, _ = pkb.rope_frequencies(64)
    want = []
    for s in ss:
        c = s["cache"].clone()
        q = pkb.append_paged_kv_cache(s["k"], s["v"], c, s["lens"], q=s["q"], qo_indptr=s["qo"],
                                      freqs=table, block_tables=s["tables"])
        want.append((q, c))
    torch.cuda.synchronize()
    outs = [torch.zeros(s["q"].shape, dtype=torch.bfloat16, device=DEV) for s in ss]
    streams = [torch.cuda.Stream() for _ in ss]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, st, out in zip(ss, streams, outs):
            pkb.append_paged_kv_cache(s["k"], s["v"], s["cache"], s["lens"], q=s["q"], q_out=out,
                                      qo_indptr=s["qo"], freqs=table, block_tables=s["tables"],
                                      stream=st)
    torch.cuda.synchronize()
    for s, out, (q, c) in zip(ss, outs, want):
        assert torch.equal(out, q) and torch.equal(s["cache"], c)


def test_refusals():
    s = problem(14, [2, 3], [0, 0])
    base = dict(k=s["k"], v=s["v"], paged_kv_cache=cache_arg(s), seq_lens_kv=s["lens"],
                qo_indptr=s["qo"], block_tables=s["tables"], q=s["q"])
    K, V = cache_arg(s)
    for kw in (dict(block_tables=None), dict(qo_indptr=s["qo"][:2]), dict(qo_indptr=None),
               dict(seq_lens_kv=s["lens"][:1]), dict(seq_lens_kv=s["lens"].long()),
               dict(block_tables=s["tables"].long()), dict(block_tables=s["tables"][:1]),
               dict(k=s["k"][:, :1]), dict(v=s["v"].float()), dict(k=s["k"].double(), v=s["v"].double()),
               dict(k=s["k"][..., :32], v=s["v"][..., :32]), dict(q=s["q"][:3]), dict(q=s["q"].float()),
               dict(paged_kv_cache=(K.half(), V.half())), dict(paged_kv_cache=(K, V[:2])),
               dict(paged_kv_cache=K), dict(paged_kv_cache=(K.transpose(1, 2), V.transpose(1, 2))),
               dict(q=None, q_out=s["q"].contiguous()), dict(q_out=s["q"]),
               dict(paged_kv_indptr=s["qo"]), dict(status=torch.zeros(1, device=DEV).double())):
        a = dict(base)
        a.update(kw)
        with pytest.raises(ValueError):
            pkb.append_paged_kv_cache(**a)
