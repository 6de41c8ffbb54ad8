"""Freeing, extending, forking, compacting and copying pages on the GPU: every integer and every
moved byte equals the sequential oracle's."""
import random

import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import cache as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Both:
    """The same state on the GPU and in the oracle, and the calls on both."""

    def __init__(self, seed, R, C, P, ps, *, layers=1, Hkv=2, D=8, combined=True, offset=0):
        g = torch.Generator().manual_seed(seed)
        self.ps, self.combined = ps, combined
        shape = (P, 2, Hkv, ps, D) if combined else (P, Hkv, ps, D)
        n = layers if combined else 2 * layers
        self.pools = [torch.randint(-32768, 32767, shape, generator=g, dtype=torch.int16).to(DEV)
                      .view(torch.bfloat16) for _ in range(n)]
        self.handle = pkb.cache_pools(self.pools if combined else
                                      list(zip(self.pools[::2], self.pools[1::2])))
        # counts that start `offset` elements into their storage (4-byte alignment)
        store = torch.zeros(P + offset, dtype=torch.int32, device=DEV)
        self.refs = store[offset:]
        self.tables = torch.full((R, C), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(R, dtype=torch.int32, device=DEV)
        self.o = O.State(self.tables.tolist(), self.lens.tolist(), self.refs.tolist(), ps,
                         [self.bits(p) for p in self.pools])
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.full((max(pkb.fork_cache_workspace_size(4096),
                                  pkb.compact_cache_workspace_size(P)),), 0xAB,
                             dtype=torch.uint8, device=DEV)

    def bits(self, pool):
        a = pool.view(torch.int16).cpu().numpy()
        return a.reshape(a.shape[0], -1, self.ps, a.shape[-1]).copy()

    def set(self, tables=None, lens=None, refs=None):
        for name, value in (("tables", tables), ("lens", lens), ("refs", refs)):
            if value is not None:
                getattr(self, name).copy_(i32(value))
        o = self.o
        self.o = O.State(self.tables.tolist(), self.lens.tolist(), self.refs.tolist(), self.ps,
                         o.pools)

    def _ws_status(self):
        return pkb.paged_attn_workspace_status(self.ws)[1]

    def free(self, rows):
        self.o.status = 0
        self.status.zero_()
        pkb.free_cache_rows(i32(rows), self.tables, self.lens, self.refs, self.ps,
                            status=self.status)
        self.o.free(rows)
        assert self.status.item() == self.o.status
        self.same()

    def extend(self, rows, new):
        self.o.status = 0
        pkb.extend_cache_rows(i32(rows), i32(new), self.tables, self.lens, self.refs, self.ps,
                              workspace=self.ws)
        self.o.extend(rows, new)
        assert self._ws_status() == self.o.status
        self.same()

    def fork(self, parents, children):
        self.o.status = 0
        pkb.fork_cache_rows(self.handle, i32(parents), i32(children), self.tables, self.lens,
                            self.refs, workspace=self.ws)
        self.o.fork(parents, children)
        assert self._ws_status() == self.o.status
        self.same()

    def compact(self, in_place=True):
        self.o.status = 0
        kw = {}
        if not in_place:
            kw = dict(block_tables_out=torch.full_like(self.tables, 99),
                      page_refs_out=torch.full_like(self.refs, 99))
            kept = self.tables.clone(), self.refs.clone()
        t, r, live = pkb.compact_cache(self.handle, self.tables, self.lens, self.refs,
                                       workspace=self.ws, **kw)
        assert live.item() == self.o.compact()
        assert self._ws_status() == self.o.status
        if not in_place:
            assert torch.equal(self.tables, kept[0]) and torch.equal(self.refs, kept[1])
            self.tables.copy_(t)
            self.refs.copy_(r)
        self.same()

    def same(self):
        assert self.lens.tolist() == self.o.lens
        assert self.refs.tolist() == self.o.refs
        assert self.tables.tolist() == self.o.tables
        for p, q in zip(self.pools, self.o.pools):
            assert np.array_equal(self.bits(p), q)


@pytest.mark.parametrize("seed", range(6))
def test_random_calls(seed):
    """Long random runs of every call, lists with empty rows, repeats and bad ids among them."""
    rng = random.Random(seed)
    ps = rng.choice([8, 16, 24])
    R, C, P = rng.randint(3, 12), rng.randint(2, 9), rng.randint(20, 70)
    b = Both(seed, R, C, P, ps, layers=rng.randint(1, 3), combined=seed % 2 == 0, offset=seed % 3)
    for step in range(40):
        op = rng.choice(["extend", "extend", "free", "fork", "fork", "compact"])
        n = rng.randint(1, R)
        rows = [rng.randint(-1, R) if rng.random() < 0.05 else rng.randrange(R) for _ in range(n)]
        if op == "extend":
            b.extend(rows, [rng.choice([0, 1, rng.randint(0, 3 * ps), -1 if rng.random() < 0.05 else 2])
                            for _ in range(n)])
        elif op == "free":
            b.free(rows)
        elif op == "fork":
            b.fork([rng.randrange(R) for _ in range(n)], rows)
        else:
            b.compact(in_place=rng.random() < 0.5)


@pytest.mark.parametrize("P", [1, 5, 4096, 4097, 8192, 8193, 40000])
def test_lowest_pages_first_in_small_and_large_pools(P):
    """One CTA plans small pools, a cluster large ones; counts in use are scattered."""
    rng = np.random.RandomState(P)
    R = 9
    C = max(1, P // 4)
    b = Both(P, R, C, P, 8, Hkv=1, combined=True)
    used = (rng.rand(P) < 0.6).astype(np.int32)
    used[rng.permutation(P)[:max(1, P // 3)]] = 0
    b.set(refs=(used * 3).tolist())
    free = int((used == 0).sum())
    want = [0, 1, 7 * C, 8, 9, 0, min(free, C) * 8, 5, 3]
    b.extend(list(range(R))[::-1], want)
    b.free([0, 3, 3])
    b.extend([3, 0], [1, 2])


def test_pools_of_many_pages():
    """More steps of pages than a warp has lanes and than a thread keeps masks for."""
    P, R = 300001, 40
    rng = np.random.RandomState(1)
    b = Both(9, R, 9000, P, 8, Hkv=1, combined=False)
    used = (rng.rand(P) < 0.9).astype(np.int32)
    used[:200000] = 1
    b.set(refs=used.tolist())
    free = int((used == 0).sum())
    b.extend(list(range(R)), [rng.randint(0, 2 * 8 * free // R) for _ in range(R)])
    b.free([3, 5])
    b.fork([7, 8, 9], [3, 5, 5])
    b.compact(in_place=False)


def test_the_largest_pool():
    """2^24 pages; one more is refused."""
    P = 1 << 24
    refs = torch.ones(P, dtype=torch.int32, device=DEV)
    free = i32([5, 4_000_000, P - 9, P - 1])
    refs[free.long()] = 0
    tables, lens = torch.full((2, 4), -1, dtype=torch.int32, device=DEV), i32([0, 0])
    ws = torch.empty(pkb.extend_cache_workspace_size(2), dtype=torch.uint8, device=DEV)
    pkb.extend_cache_rows(i32([1, 0]), i32([24, 17]), tables, lens, refs, 16, workspace=ws)
    assert tables.tolist() == [[P - 9, P - 1, -1, -1], [5, 4_000_000, -1, -1]]
    assert lens.tolist() == [17, 24] and refs.eq(1).all()
    assert pkb.paged_attn_workspace_status(ws)[0] == pkb.OK
    with pytest.raises(pkb.PagedAttnError):
        more = torch.ones(P + 1, dtype=torch.int32, device=DEV)
        pkb.extend_cache_rows(i32([1]), i32([1]), tables, lens, more, 16, workspace=ws)


def test_many_rows():
    """More items than a CTA has threads, in one CTA and in clusters of 2 to 8."""
    for P, R in ((6000, 1500), (9000, 1500), (20000, 4096), (50000, 1500)):
        b = Both(P, R, 4, P, 8, Hkv=1, D=8)
        rng = random.Random(P)
        rows = list(range(R))
        rng.shuffle(rows)
        b.extend(rows, [rng.randint(0, 24) for _ in rows])
        b.free(rows[:700])
        b.extend(rows[::-1], [rng.choice([0, 1, 9]) for _ in rows])
        b.free(rows[300:900])
        b.fork([rng.choice(rows[900:]) for _ in range(600)], rows[300:900])
        b.compact(in_place=False)


def test_running_out_of_pages():
    """Items are served in order while the total fits; those that need no page always are."""
    b = Both(1, 6, 8, 10, 16)
    b.extend([0, 1, 2, 3], [64, 64, 64, 16])          # 4 + 4, then 12 > 10, and 13
    assert b.lens.tolist() == [64, 64, 0, 0, 0, 0]
    b.extend([0, 4, 5], [1, 17, 0])                   # the 5th page, then 1 + 2 > 2
    b.extend([0, 5, 4], [15, 16, 1])                  # row 0 needs none; row 5 takes the last
    b.fork([0, 1], [2, 3])                            # row 0 and 1 end with a page: shared whole
    b.extend([4], [1])
    b.free([0])
    b.extend([4], [1 << 30])                          # more than the table holds
    b.extend([0, 2], [2 ** 31 - 1, 2 ** 31 - 1])


def test_absurd_demands_do_not_wrap():
    """Demands whose sum passes 2^31 pages are refused, not wrapped into served ones."""
    P, n = 64, 300
    C = 1 << 23                                       # 300 x 2^23 pages pass 2^31; 10 GB of table
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    lens = torch.zeros(n, dtype=torch.int32, device=DEV)
    tables = torch.full((n, C), -1, dtype=torch.int32, device=DEV)
    rows = torch.arange(n, dtype=torch.int32, device=DEV)
    new = torch.full((n,), C * 8, dtype=torch.int32, device=DEV)
    ws = torch.empty(pkb.extend_cache_workspace_size(n), dtype=torch.uint8, device=DEV)
    pkb.extend_cache_rows(rows, new, tables, lens, refs, 8, workspace=ws)
    assert pkb.paged_attn_workspace_status(ws) == (pkb.ERR_CAPACITY, 2)
    assert not lens.any() and not refs.any() and tables.eq(-1).all()


def test_fork_contract():
    """Repeated children, children in use, a row that is its own parent, empty parents, a parent
    that is a child of the same call: what breaks the contract is left out, the rest is done."""
    b = Both(2, 8, 6, 40, 16, layers=2)
    b.extend([0, 1, 2], [40, 33, 16])
    b.fork([0, 1, 0, 2, 3, 5, 9, 0], [3, 3, 4, 1, 5, 5, 6, -1])
    b.fork([0, 6, 4], [6, 7, 7])
    b.extend([3, 4, 6], [1, 1, 20])                  # forks write their own tails
    b.free([0, 1, 2])
    b.compact()


def test_bad_pages_are_left_out():
    b = Both(3, 5, 4, 20, 16)
    b.extend([0, 1], [60, 30])
    t = b.tables.tolist()
    t[0][1], t[1][0], t[1][1] = 20, -5, 99
    b.set(tables=t)
    b.fork([0, 1], [2, 3])
    b.compact()
    b.free([0, 1, 2, 3, 4, 7, -1])
    b.set(lens=[1000, 0, 0, 0, 0])                   # longer than its table row
    b.compact()
    b.free([0])
    b.set(lens=[30, 0, 0, 0, 0], refs=[0] * 20)      # counts already 0
    b.free([0])


@pytest.mark.parametrize("P,density", [(7, 0.5), (300, 0.0), (300, 1.0), (300, 0.1), (5000, 0.5),
                                       (20000, 0.5), (20001, 0.97), (9000, 0.02)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(P, density, in_place):
    rng = np.random.RandomState(P)
    R = 11
    n = int(P * density)
    ids = rng.permutation(P)[:n]
    need = np.bincount(rng.randint(0, R, n), minlength=R)
    C = int(need.max(initial=0)) + 3
    tables = np.full((R, C), P + 5, np.int64)         # dead entries keep whatever they hold
    at = 0
    for r in range(R):
        tables[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
    refs = np.zeros(P, np.int64)
    refs[ids] = 1
    b = Both(P, R, C, P, 8, Hkv=1, layers=2)
    b.set(tables=tables.tolist(), lens=(need * 8 - (need > 0) * 3).tolist(), refs=refs.tolist())
    b.compact(in_place)
    b.compact(in_place)                               # nothing left to move


@pytest.mark.parametrize("combined", [True, False])
@pytest.mark.parametrize("Hkv,ps,D", [(8, 16, 128), (1, 8, 8), (2, 24, 40), (3, 128, 256)])
def test_copy(combined, Hkv, ps, D):
    """Within the pools and to others of another page count; bad ids are reported."""
    g = torch.Generator().manual_seed(ps)

    def pools(P, n):
        shape = (P, 2, Hkv, ps, D) if combined else (P, Hkv, ps, D)
        flat = [torch.randint(-32768, 32767, shape, generator=g, dtype=torch.int16).to(DEV)
                .view(torch.bfloat16) for _ in range(n if combined else 2 * n)]
        return flat, pkb.cache_pools(flat if combined else list(zip(flat[::2], flat[1::2])))

    def bits(flat):
        return [p.view(torch.int16).cpu().numpy().copy() for p in flat]
    a, ha = pools(30, 3)
    c, hc = pools(17, 3)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for flat, handle, src, dst in ((a, None, [3, 3, 29, 7], [0, 5, 1, 7]),
                                   (c, hc, [29, 0, 30, 4, -1, 2], [16, 3, 1, 17, 2, 0])):
        want, source = bits(flat), bits(a)
        expect = O.copy_pages(source if handle else want, want, src, dst)
        status.zero_()
        pkb.copy_cache_pages(ha, i32(src), i32(dst), dst_pools=handle, status=status)
        assert status.item() == expect
        for x, y in zip(bits(flat), want):
            assert np.array_equal(x, y)
    pkb.copy_cache_pages(ha, i32([]), i32([]))


def test_pools_past_4_gb():
    """Pages whose bytes lie past 2^32 in their pool."""
    P, Hkv, ps, D = 40000, 2, 128, 256
    pool = torch.zeros(P, 2, Hkv, ps, D, dtype=torch.bfloat16, device=DEV)     # 10.5 GB
    g = torch.Generator().manual_seed(0)
    page = torch.randn(2, Hkv, ps, D, generator=g).to(torch.bfloat16).to(DEV)
    pool[7] = page
    h = pkb.cache_pools([pool])
    pkb.copy_cache_pages(h, i32([7]), i32([P - 1]))
    assert torch.equal(pool[P - 1], page)
    tables, lens = i32([[P - 1], [3]]), i32([100, 0])
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    refs[P - 1] = 1
    pkb.fork_cache_rows(h, i32([0]), i32([1]), tables, lens, refs)
    assert tables.tolist() == [[P - 1], [0]] and torch.equal(pool[0, :, :, :100], page[:, :, :100])
    assert pool[0, :, :, 100:].eq(0).all()
    _, _, live = pkb.compact_cache(h, tables, lens, refs)
    assert tables.tolist() == [[1], [0]] and live.item() == 2 and torch.equal(pool[1], page)


def test_graph_and_shared_workspace():
    """free + extend + fork + compact captured once and replayed; the calls of one stream share a
    workspace."""
    b = Both(4, 6, 8, 50, 16, layers=2)
    b.extend([0, 1], [50, 70])
    rows, new = i32([2, 3]), i32([33, 20])
    parents, children = i32([0, 1]), i32([4, 5])
    live = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        pkb.free_cache_rows(rows, b.tables, b.lens, b.refs, b.ps)
        pkb.free_cache_rows(children, b.tables, b.lens, b.refs, b.ps)
        pkb.extend_cache_rows(rows, new, b.tables, b.lens, b.refs, b.ps, workspace=b.ws)
        pkb.fork_cache_rows(b.handle, parents, children, b.tables, b.lens, b.refs, workspace=b.ws)
        pkb.compact_cache(b.handle, b.tables, b.lens, b.refs, num_live=live, workspace=b.ws)

    def oracle():
        b.o.free([2, 3])
        b.o.free([4, 5])
        b.o.extend([2, 3], [33, 20])
        b.o.fork([0, 1], [4, 5])
        return b.o.compact()
    step()
    n = oracle()
    torch.cuda.synchronize()
    b.same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
        n = oracle()
    b.same()
    assert live.item() == n


def test_two_graphs_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn on one stream, and a call between."""
    b = Both(6, 6, 8, 60, 16, layers=1)
    b.extend([0, 1], [50, 70])
    one, two = (i32([2]), i32([40])), (i32([0]), i32([3]))

    def first():
        pkb.free_cache_rows(one[0], b.tables, b.lens, b.refs, b.ps)
        pkb.extend_cache_rows(*one, b.tables, b.lens, b.refs, b.ps, workspace=b.ws)

    def second():
        pkb.free_cache_rows(two[1], b.tables, b.lens, b.refs, b.ps)
        pkb.fork_cache_rows(b.handle, *two, b.tables, b.lens, b.refs, workspace=b.ws)
    first()
    second()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for graph, call in zip(graphs, (first, second)):
        with torch.cuda.graph(graph):
            call()
    for _ in range(4):
        graphs[0].replay()
        graphs[1].replay()
        pkb.extend_cache_rows(i32([0]), i32([7]), b.tables, b.lens, b.refs, b.ps, workspace=b.ws)
    b.o.free([2])
    b.o.extend([2], [40])
    b.o.free([3])
    b.o.fork([0], [3])
    for _ in range(4):
        b.o.free([2])
        b.o.extend([2], [40])
        b.o.free([3])
        b.o.fork([0], [3])
        b.o.extend([0], [7])
    b.same()


def test_two_streams_at_once():
    """Two states with workspaces of their own, driven by interleaved calls on two streams."""
    both = [Both(20 + k, 8, 9, 9000, 8, Hkv=1, layers=2) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in both]
    lists = [(i32(list(range(6))), i32([3 + k, 40, 9, 1, 8, 70]), i32([0, 1]), i32([6, 7]))
             for k in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, st, (rows, new, parents, children) in zip(both, streams, lists):
            with torch.cuda.stream(st):
                pkb.free_cache_rows(rows, b.tables, b.lens, b.refs, b.ps)
                pkb.free_cache_rows(children, b.tables, b.lens, b.refs, b.ps)
                pkb.extend_cache_rows(rows, new, b.tables, b.lens, b.refs, b.ps, workspace=b.ws)
                pkb.fork_cache_rows(b.handle, parents, children, b.tables, b.lens, b.refs,
                                    workspace=b.ws)
                pkb.compact_cache(b.handle, b.tables, b.lens, b.refs, workspace=b.ws)
    torch.cuda.synchronize()
    for k, b in enumerate(both):
        for _ in range(5):
            b.o.free(list(range(6)) + [6, 7])
            b.o.extend(list(range(6)), [3 + k, 40, 9, 1, 8, 70])
            b.o.fork([0, 1], [6, 7])
            b.o.compact()
        b.same()


def test_other_stream_without_a_workspace():
    # the workspaces are freed while their kernels run; what the current stream allocates next
    # must not be that memory
    b, side = Both(23, 8, 9, 9000, 8, Hkv=1, layers=2), torch.cuda.Stream()
    rows, new = i32([0, 1, 2]), i32([30, 5, 60])
    parents, children = i32([0, 1]), i32([6, 7])
    refs_out, tables_out = torch.empty_like(b.refs), torch.empty_like(b.tables)
    torch.cuda.synchronize()

    def churn():
        for n in (pkb.extend_cache_workspace_size(3), pkb.fork_cache_workspace_size(2),
                  pkb.compact_cache_workspace_size(9000)):
            torch.full((n,), 255, dtype=torch.uint8, device=DEV)

    pkb.extend_cache_rows(rows, new, b.tables, b.lens, b.refs, b.ps, stream=side)
    churn()
    pkb.fork_cache_rows(b.handle, parents, children, b.tables, b.lens, b.refs, stream=side)
    churn()
    pkb.free_cache_rows(rows[:1], b.tables, b.lens, b.refs, b.ps, stream=side)
    _, _, live = pkb.compact_cache(b.handle, b.tables, b.lens, b.refs, stream=side,
                                   block_tables_out=tables_out, page_refs_out=refs_out)
    churn()
    torch.cuda.synchronize()
    b.tables.copy_(tables_out)
    b.refs.copy_(refs_out)
    b.o.extend([0, 1, 2], [30, 5, 60])
    b.o.fork([0, 1], [6, 7])
    b.o.free([0])
    assert live.item() == b.o.compact()
    b.same()


def test_refusals():
    b = Both(5, 3, 4, 10, 16)
    one = i32([0])
    bad = [lambda: pkb.free_cache_rows(one.long(), b.tables, b.lens, b.refs, 16),
           lambda: pkb.free_cache_rows(one, b.tables, b.lens[:2], b.refs, 16),
           lambda: pkb.free_cache_rows(one, b.tables[0], b.lens, b.refs, 16),
           lambda: pkb.free_cache_rows(one, b.tables[:, :2], b.lens, b.refs, 16),
           lambda: pkb.extend_cache_rows(one, i32([1, 2]), b.tables, b.lens, b.refs, 16),
           lambda: pkb.fork_cache_rows(b.handle, i32([0, 1]), one, b.tables, b.lens, b.refs),
           lambda: pkb.compact_cache(b.handle, b.tables, b.lens, b.refs,
                                     block_tables_out=b.tables[:2]),
           lambda: pkb.copy_cache_pages(b.handle, one, i32([1, 2])),
           lambda: pkb.cache_pools([b.pools[0], b.pools[0][:5]]),
           lambda: pkb.cache_pools([b.pools[0].float()])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    for call in (lambda: pkb.extend_cache_rows(one, one, b.tables, b.lens, b.refs, 16, workspace=small),
                 lambda: pkb.fork_cache_rows(b.handle, one, one, b.tables, b.lens, b.refs,
                                             workspace=small),
                 lambda: pkb.compact_cache(b.handle, b.tables, b.lens, b.refs, workspace=small)):
        with pytest.raises(pkb.PagedAttnError):
            call()
    with pytest.raises(pkb.PagedAttnError):           # counts of another pool
        pkb.compact_cache(b.handle, b.tables, b.lens, b.refs[:9].clone())
    empty = i32([])
    pkb.free_cache_rows(empty, b.tables, b.lens, b.refs, 16)
    pkb.extend_cache_rows(empty, empty, b.tables, b.lens, b.refs, 16, workspace=b.ws)
    assert pkb.paged_attn_workspace_status(b.ws)[0] == pkb.OK
    pkb.fork_cache_rows(b.handle, empty, empty, b.tables, b.lens, b.refs, workspace=b.ws)
    b.same()
