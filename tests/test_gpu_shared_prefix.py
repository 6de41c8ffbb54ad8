"""Decode attention for requests that share a prefix, against float64 attention of every request for
itself, within the parity tolerances of the decode form."""
import math

import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from tests.gpu_util import check_lse, check_out

pytestmark = pytest.mark.gpu
DEV = "cuda"
METADATA = 4


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Problem:
    """groups: lists of (prefix, [tail lengths]).  Full pages of a prefix are one page for all its
    requests (or, scattered, a page of each request's own that only the first one's table may be
    used for); everything that is no live token is NaN."""

    def __init__(self, seed, groups, Hq=8, Hkv=2, SQ=1, ps=16, combined=True):
        g = torch.Generator().manual_seed(seed)
        D = 128
        self.SQ, self.ps, self.combined = SQ, ps, combined
        lens, first, tables, rows = [], [0], [], []
        for prefix, tails in groups:
            shared = torch.randn(2, prefix, Hkv, D, generator=g).to(torch.bfloat16)
            for t in tails:
                own = torch.randn(2, t, Hkv, D, generator=g).to(torch.bfloat16)
                rows.append(torch.cat([shared, own], 1))
                lens.append(prefix + t)
            first.append(len(lens))
        self.lens, self.first, self.prefixes = lens, first, [p for p, _ in groups]
        B = len(lens)
        P = sum(-(-n // ps) for n in lens) + 5
        perm = torch.randperm(P, generator=g).tolist()
        C = max([-(-n // ps) for n in lens] + [1])
        pool = torch.full((P, 2, Hkv, ps, D), math.nan).to(torch.bfloat16)
        at = 0
        for gi, (prefix, tails) in enumerate(groups):
            for b in range(first[gi], first[gi + 1]):
                row = []
                for j in range(-(-lens[b] // ps)):
                    if b > first[gi] and (j + 1) * ps <= prefix:
                        row.append(tables[first[gi]][j])
                        continue
                    row.append(perm[at])
                    x = rows[b][:, j * ps:(j + 1) * ps].transpose(1, 2)
                    pool[perm[at], :, :, :x.shape[2]] = x
                    at += 1
                tables.append(row + [-1] * (C - len(row)))
        self.tables = tables
        shape = (B, Hq, D) if SQ == 1 else (B, SQ, Hq, D)
        self.q = (1.5 * torch.randn(shape, generator=g)).to(torch.bfloat16)
        self.rows = [r.double().numpy() for r in rows]
        self.cache = pool.to(DEV) if combined else tuple(pool[:, i].contiguous().to(DEV)
                                                         for i in range(2))

    def reference(self, causal=True, scale=None):
        q = self.q.double().numpy().reshape(len(self.lens), self.SQ, -1, 128)
        out, lse = np.zeros(q.shape), np.full(q.shape[:-1], -np.inf)
        scale = scale or 128 ** -0.5
        for b, n in enumerate(self.lens):
            k, v = self.rows[b]
            G = q.shape[2] // k.shape[1]
            for i in range(self.SQ):
                see = max(0, n - self.SQ + i + 1) if causal else n
                for h in range(q.shape[2] if see else 0):
                    x = k[:see, h // G] @ q[b, i, h] * scale
                    e = np.exp(x - x.max())
                    out[b, i, h] = e @ v[:see, h // G] / e.sum()
                    lse[b, i, h] = x.max() + np.log(e.sum())
        return out.reshape(self.q.shape), lse.reshape(self.q.shape[:-1])

    def run(self, *, causal=True, first=None, prefixes=None, status=0, tables=None, **kw):
        tables = tables or self.tables
        C = len(tables[0])
        args = (self.q.to(DEV), self.cache, kw.pop("workspace", None),
                i32([C * b for b in range(len(tables) + 1)]), i32(sum(tables, [])), i32(self.lens),
                max(self.lens + [1]), i32(self.first if first is None else first),
                i32(self.prefixes if prefixes is None else prefixes))
        lse = torch.full(self.q.shape[:-1], 7.0, device=DEV)
        mask = "causal" if causal else "dense"
        params = pkb.decode_params(args[0], self.cache, args[6], seq_len_q=self.SQ)
        ws = torch.full((pkb.paged_decode_shared_workspace_size(params, args[8].numel()),), 0x7F,
                        dtype=torch.uint8, device=DEV)
        out, _ = pkb.batch_decode_with_shared_prefix(
            *args[:2], ws, *args[3:], seq_len_q=self.SQ, mask_type=mask, lse=lse, **kw)
        assert pkb.paged_attn_workspace_status(ws)[1] == status
        return out, lse

    def check(self, causal=True, **kw):
        out, lse = self.run(causal=causal, **kw)
        want, want_lse = self.reference(causal)
        check_out(out, want)
        check_lse(lse, want_lse)
        return out, lse


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (5, 1), (7, 1), (16, 1), (64, 8)])
@pytest.mark.parametrize("SQ", [1, 2, 4])
def test_heads_and_queries(Hq, Hkv, SQ):
    p = Problem(Hq + SQ, [(300, [4, 20, 133]), (64, [5]), (129, [7, 4])], Hq, Hkv, SQ)
    p.check()
    p.check(causal=False)


@pytest.mark.parametrize("ps,combined", [(8, True), (24, False), (32, True), (128, False)])
@pytest.mark.parametrize("prefix", [1, 63, 128, 200, 1025])
def test_prefixes_and_pages(ps, combined, prefix):
    Problem(prefix, [(prefix, [1, 64, 65, 3])], ps=ps, combined=combined).check()


def test_rows_of_several_tiles():
    """More rows than a tile holds, a last tile with few, groups of all sizes."""
    Problem(1, [(700, [1 + i % 40 for i in range(150)])]).check()
    Problem(2, [(500, [3] * 65), (260, [9] * 64), (5, [2] * 2), (900, [70])], 16, 4).check()
    Problem(3, [(400, [4] * 33)], 16, 1, SQ=4).check()


def test_long_prefix():
    Problem(4, [(6000, [17, 400, 1, 90, 3])], 4, 1).check()


def test_prefix_that_not_everyone_sees():
    """Longer than a member, than its first query's position, or negative: cut back."""
    p = Problem(5, [(300, [1, 2, 1, 5])], SQ=2)            # causal: 301 keys, queries at 299, 300
    p.check()
    p.check(causal=False)
    for cut in (301, 10 ** 9, 2 ** 31 - 1):
        q = Problem(6, [(300, [0, 2, 5])])
        q.check(prefixes=[cut], causal=False) if cut == 301 else q.check(prefixes=[cut])
    p.check(prefixes=[-5])
    p.check(prefixes=[0])


def test_tails_of_nothing():
    """A fresh fork's query may be the prefix's last token."""
    p = Problem(7, [(256, [0, 0, 0]), (100, [0, 30])])
    p.check()
    p.check(causal=False)


def test_empty_rows():
    p = Problem(8, [(0, [0, 5, 1]), (40, [3, 3])])
    out, lse = p.check()
    assert not out[0].any() and torch.isneginf(lse[0]).all()


def test_requests_outside_groups():
    p = Problem(9, [(200, [1, 30]), (150, [4, 4, 9]), (90, [2, 2])])
    p.check(first=[2, 5], prefixes=[150])
    p.check(first=[0], prefixes=[])
    p.check(first=[0, 0, 2, 2, 5, 7, 7], prefixes=[9, 200, 9, 150, 90, 9])
    p.check(first=[0, 1, 2], prefixes=[200, 200])          # groups of one


@pytest.mark.parametrize("first", [[0, 5, 3], [-1, 2, 5], [0, 2, 8]])
def test_broken_groups_share_nothing(first):
    p = Problem(10, [(200, [1, 30]), (150, [4, 4, 9])])
    p.check(first=first, prefixes=[200, 150], status=METADATA)


def test_the_prefix_is_read_from_the_first_request():
    """The other members' entries before the prefix's last 128 keys are never used."""
    p = Problem(11, [(500, [9, 9, 30])])
    tables = [list(r) for r in p.tables]
    for b in (1, 2):
        tables[b][:384 // 16] = [10 ** 6] * (384 // 16)
    p.check(tables=tables)


def test_bad_page():
    p = Problem(12, [(300, [9, 30])])
    tables = [list(r) for r in p.tables]
    tables[0][2] = 10 ** 6
    p.run(tables=tables, status=METADATA)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_output_types_and_scales(dtype):
    p = Problem(13, [(300, [9, 30]), (40, [3, 3])])
    out, lse = p.run(out_dtype=dtype, bmm2_scale=0.5, bmm1_scale=0.05)
    want, want_lse = p.reference(scale=0.05)
    assert out.dtype == dtype
    check_out(out, 0.5 * want)
    check_lse(lse, want_lse)
    given = torch.empty_like(out)
    assert p.run(out=given, bmm2_scale=0.5, bmm1_scale=0.05)[0] is given
    assert torch.equal(given, out)


def test_equals_plain_decode():
    p = Problem(14, [(1000, [9, 300, 41]), (777, [1] * 20)])
    out, lse = p.run()
    C = len(p.tables[0])
    other = torch.empty_like(lse)
    plain, _ = pkb.batch_decode_with_paged_kv_cache(
        p.q.to(DEV), p.cache, None, i32([C * b for b in range(len(p.tables) + 1)]),
        i32(sum(p.tables, [])), i32(p.lens), max(p.lens), lse=other)
    check_out(out, plain.double().cpu().numpy())
    check_lse(lse, other.double().cpu().numpy(), 1e-4)


def test_repeats_bit_for_bit_captured_and_on_another_stream():
    p = Problem(15, [(1000, [9, 300, 41]), (777, [1] * 20)])
    out, lse = p.run()
    again, again_lse = p.run()
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    C = len(p.tables[0])
    args = (p.q.to(DEV), p.cache)
    rest = (i32([C * b for b in range(len(p.tables) + 1)]), i32(sum(p.tables, [])), i32(p.lens),
            max(p.lens), i32(p.first), i32(p.prefixes))
    ws = torch.empty(pkb.shared_prefix_workspace_size(*args, max(p.lens), 2), dtype=torch.uint8,
                     device=DEV)
    o, l2 = torch.empty_like(out), torch.empty_like(lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkb.batch_decode_with_shared_prefix(*args, ws, *rest, out=o, lse=l2, mask_type="causal")
    for _ in range(3):
        o.zero_()
        graph.replay()
        assert torch.equal(o, out) and torch.equal(l2, lse)
    rest[2].sub_(1)                          # the replay reads the lengths of the moment
    graph.replay()
    p.lens = [n - 1 for n in p.lens]
    p.rows = [r[:, :-1] for r in p.rows]
    check_out(o, p.reference()[0])
    side.wait_stream(torch.cuda.current_stream())
    other, _ = pkb.batch_decode_with_shared_prefix(*args, None, *rest, mask_type="causal",
                                                   stream=side)
    side.synchronize()
    assert torch.equal(other, o)


def test_nan_queries_stay_in_their_rows():
    p = Problem(16, [(300, [9, 30, 4])])
    clean, _ = p.run()
    p.q[1] = math.nan
    out, _ = p.run()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    assert out[1].isnan().all()


def test_an_empty_batch():
    q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(4, 2, 2, 16, 128, dtype=torch.bfloat16, device=DEV)
    out, _ = pkb.batch_decode_with_shared_prefix(q, cache, None, i32([0]), i32([]), i32([]), 16,
                                                 i32([0]), i32([]))
    assert out.shape == q.shape


class Padded(Problem):
    """A problem whose requests `empty` have ended: length 0 and a page table of what nobody may
    read."""

    def __init__(self, empty, *args, **kw):
        super().__init__(*args, **kw)
        for b in empty:
            self.lens[b], self.rows[b] = 0, self.rows[b][:, :0]
            self.tables[b] = [10 ** 6] * len(self.tables[b])


@pytest.mark.parametrize("Hq,SQ", [(8, 1), (8, 3), (16, 4)])
def test_empty_members_of_a_group(Hq, SQ):
    """They change nothing for the others, which still share: beside a member without pages of its
    own for the prefix."""
    groups = [(500, [9, 12, 30, 4]), (200, [7, 9]), (150, [5, 6, 7])]
    p = Padded([0, 2, 5, 6, 7, 8], 17, groups, Hq, 2, SQ)
    tables = [list(r) for r in p.tables]
    tables[3][:384 // 16] = [10 ** 6] * (384 // 16)
    for causal in (True, False):
        out, lse = p.check(causal, tables=tables)
        for b in (0, 2, 5):
            assert not out[b].any() and torch.isneginf(lse[b]).all()


@pytest.mark.parametrize("Hq,SQ", [(4, 1), (16, 2)])
def test_batches_that_exceed_the_plan_s_shared_memory(Hq, SQ):
    """Over 8,192 requests and over 1,024 groups."""
    p = Problem(18, [(40, [2 + i % 3, 2, 2 + i % 5]) for i in range(2900)], Hq, 1, SQ, ps=8)
    out, lse = p.run()
    tables, C = p.tables, len(p.tables[0])
    other = torch.empty_like(lse)
    plain, _ = pkb.batch_decode_with_paged_kv_cache(
        p.q.to(DEV), p.cache, None, i32([C * b for b in range(len(tables) + 1)]),
        i32(sum(tables, [])), i32(p.lens), max(p.lens), lse=other, seq_len_q=SQ,
        mask_type="causal")
    check_out(out, plain.double().cpu().numpy())
    check_lse(lse, other.double().cpu().numpy(), 1e-4)


@pytest.mark.parametrize("Hq,SQ", [(8, 1), (16, 3)])
def test_pages_past_32_bits(Hq, SQ):
    """A cache of 2.5e9 elements, its last pages in use."""
    p = Problem(19, [(300, [9, 30, 4]), (64, [100, 5])], Hq, 1, SQ)
    small, P = p.cache, 600_000
    p.cache = torch.empty(P, 2, 1, 16, 128, dtype=torch.bfloat16, device=DEV)
    p.cache[P - small.shape[0]:] = small
    p.tables = [[t + P - small.shape[0] if t >= 0 else t for t in r] for r in p.tables]
    p.check()


def test_graphs_that_share_a_workspace_and_streams_that_do_not():
    """Two captured steps of different sizes replayed in turn on one workspace; calls on two streams
    at once."""
    problems = [Problem(20, [(900, [9, 30, 4]), (64, [100, 1])], 8, 2),
                Problem(21, [(333, [40] * 9)], 32, 2, 2, ps=32)]
    calls, graphs, need = [], [], 0
    for p in problems:
        C = len(p.tables[0])
        rest = (i32([C * b for b in range(len(p.tables) + 1)]), i32(sum(p.tables, [])),
                i32(p.lens), max(p.lens), i32(p.first), i32(p.prefixes))
        calls.append((p.q.to(DEV), p.cache, rest, torch.empty_like(p.q, device=DEV), p.SQ))
        need = max(need, pkb.shared_prefix_workspace_size(
            calls[-1][0], p.cache, max(p.lens), len(p.prefixes), seq_len_q=p.SQ))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def call(c, ws=None, out=None, stream=None):
        return pkb.batch_decode_with_shared_prefix(*c[:2], ws, *c[2], seq_len_q=c[4], out=out,
                                                   mask_type="causal", stream=stream)[0]
    want = [call(c) for c in calls]
    for p, w in zip(problems, want):
        check_out(w, p.reference()[0])
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(c, ws, c[3])
    for i in (0, 1, 1, 0, 1, 0):
        calls[i][3].zero_()
        graphs[i].replay()
        assert torch.equal(calls[i][3], want[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[call(c, stream=s) for c, s in zip(calls, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(a, b) for a, b in zip(pair, want))


@pytest.mark.parametrize("Hq", [4, 16])
def test_queries_before_the_first_key(Hq):
    """Requests of fewer tokens than queries: the first queries see nothing."""
    p = Problem(22, [(0, [2, 5]), (1, [1, 40]), (3, [1])], Hq, 2, SQ=4)
    out, lse = p.check()
    assert not out[0, :2].any() and torch.isneginf(lse[0, :2]).all()
    p.check(causal=False)
