"""Cutting rows back to their kept tokens on the GPU: tables, lengths, counts, weights and every
byte of the pools equal the sequential oracle's."""
import random

import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import eviction as O
from tests.test_gpu_cache_pages import Both, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Rows(Both):
    """Adds weights and the call to the pages' state."""

    def __init__(self, seed, R, C, P, ps, *, layers=1, Hkv=2, **kw):
        super().__init__(seed, R, C, P, ps, layers=layers, Hkv=Hkv, **kw)
        self.w = torch.rand(layers, R, Hkv, C * ps, generator=torch.Generator().manual_seed(seed))
        self.ow, self.w = self.w.numpy().copy(), self.w.to(DEV)

    def evict(self, rows, kept, sink=0, weights=True, status=None):
        self.o.status = 0
        n, K = kept.shape[1], kept.shape[3]
        ws = torch.full((pkb.evict_cache_workspace_size(n, K, self.ps),), 0xAB, dtype=torch.uint8,
                        device=DEV)
        word = i32([0])
        lists = torch.from_numpy(kept.astype(np.int32)).to(DEV)
        pkb.evict_cache_rows(self.handle, i32(rows), lists, self.tables, self.lens, self.refs,
                             weights=self.w if weights else None, sink=sink, workspace=ws,
                             status=word)
        O.evict(self.o, rows, kept, sink, self.ow if weights else None, self.combined)
        self.same()
        assert np.array_equal(self.w.cpu().numpy(), self.ow)
        assert word.item() == self.o.status == pkb.paged_attn_workspace_status(ws)[1]

    def lists(self, rng, rows, K, sink=0, N=None, Hkv=2):
        """Random ascending lists for the rows' present lengths that start with 0 .. sink - 1."""
        N = N or self.w.shape[0]
        kept = np.full((N, len(rows), Hkv, K), -1, np.int64)
        for i, r in enumerate(rows):
            L = self.o.lens[r] if 0 <= r < self.o.R else 0
            for layer in range(N):
                for h in range(Hkv):
                    if L > K:
                        kept[layer, i, h] = list(range(sink)) + sorted(
                            rng.sample(range(sink, L), K - sink))
                    elif L > 0:
                        kept[layer, i, h, :L] = np.arange(L)
        return kept


@pytest.mark.parametrize("seed", range(8))
def test_random_calls(seed):
    """Long runs of extending, forking, freeing and evicting, so that pages are shared."""
    rng = random.Random(seed)
    ps = rng.choice([8, 16, 24])
    R, C, P = rng.randint(3, 9), rng.randint(3, 9), rng.randint(30, 80)
    b = Rows(seed, R, C, P, ps, layers=rng.randint(1, 3), combined=seed % 2 == 0, offset=seed % 3,
             D=rng.choice([8, 24, 80, 128]))
    for step in range(30):
        op = rng.choice(["extend", "extend", "free", "fork", "evict", "evict"])
        n = rng.randint(1, R)
        rows = rng.sample(range(R), n)
        if op == "extend":
            b.extend(rows, [rng.randint(0, 3 * ps) for _ in rows])
        elif op == "free":
            b.free(rows[:1])
        elif op == "fork":
            b.fork([rng.randrange(R) for _ in rows], rows)
        else:
            K = rng.randint(1, 2 * ps)
            sink = rng.randint(0, K)
            b.evict(rows, b.lists(rng, rows, K, sink), sink, weights=rng.random() < 0.8)


@pytest.mark.parametrize("combined", [True, False])
@pytest.mark.parametrize("D", [8, 64, 128, 256, 512])
def test_long_rows(combined, D):
    """Lists of many tiles, few units (column slices) and many."""
    rng = random.Random(D)
    for R, K in ((1, 700), (6, 333)):
        b = Rows(D + R, R, 70, 71 * R, 16, D=D, combined=combined)
        rows = list(range(R))
        b.extend(rows, [1100 - 7 * r for r in rows])
        b.evict(rows, b.lists(rng, rows, K))
        b.extend(rows, [100] * R)
        b.evict(rows, b.lists(rng, rows, K, 40), 40)


def test_pages_that_others_share():
    """Forked rows: pages inside the sink stay shared, the rest is copied before it changes."""
    rng = random.Random(1)
    b = Rows(7, 4, 8, 60, 16, layers=2)
    b.extend([0], [100])
    b.fork([0, 0, 0], [1, 2, 3])
    shared = b.tables[0, :2].tolist()
    b.evict([2, 0], b.lists(rng, [2, 0], 50, 36), 36)
    assert b.tables[0, :2].tolist() == b.tables[2, :2].tolist() == shared
    assert b.refs[shared[0]].item() == 4
    b.evict([1, 3], b.lists(rng, [1, 3], 90, 0), 0)
    b.evict([1, 0], b.lists(rng, [1, 0], 16, 16), 16)       # nothing moves, pages go back
    b.free([0, 1, 2, 3])
    assert b.refs.sum().item() == 0


def test_too_few_free_pages():
    """Items are served in order while the pages last; the others keep everything."""
    rng = random.Random(2)
    b = Rows(8, 4, 6, 12, 8)
    b.extend([0], [40])
    b.fork([0, 0], [1, 2])
    b.extend([3], [40])                      # 10 pages in use, 2 free
    rows = [1, 3, 0, 2]
    b.evict(rows, b.lists(rng, rows, 12))    # 2 pages for row 1, none for row 3, none left
    assert b.lens.tolist() == [40, 12, 40, 12]
    b.evict([0], b.lists(rng, [0], 12))


def test_items_that_are_left_out():
    rng = random.Random(3)
    b = Rows(9, 5, 4, 24, 8)
    b.extend([0, 1, 2, 3, 4], [30, 30, 30, 30, 8])
    good = b.lists(rng, [0, 1, 2, 3, 4], 10)
    for change in ((0, 0, 0, 0, -1), (0, 1, 1, 9, 30), (0, 2, 0, 9, 8)):
        kept = good.copy()
        kept[change[:4]] = change[4]
        state = b.lens.tolist()
        b.evict([0, 1, 2, 3, 4][change[1]:change[1] + 1], kept[:, change[1]:change[1] + 1])
        assert b.lens.tolist() == state
    b.evict([5, -1, 3, 3, 4], b.lists(rng, [5, -1, 3, 3, 4], 10))
    tables = b.tables.tolist()
    tables[1][3], tables[2][1] = 24, -1
    lens = b.lens.tolist()
    lens[0] = 33
    b.set(tables=tables, lens=lens)
    b.evict([0, 1, 2], np.repeat(good[:, 1:2], 3, axis=1))
    assert b.lens.tolist()[:3] == [33, 30, 30]


def test_weights_narrower_than_a_row():
    b = Rows(10, 2, 4, 9, 8)
    b.extend([0, 1], [30, 20])
    b.w = b.w[..., :24].contiguous()
    b.ow = b.ow[..., :24].copy()
    b.evict([0, 1], b.lists(random.Random(4), [0, 1], 9))
    assert b.lens.tolist() == [30, 9]


def test_bad_entries_touch_nothing_else():
    """A slot whose entry lies before it or past the row keeps what it holds; the row's neighbours
    and the pages of the sink are not written."""
    b = Rows(11, 2, 4, 9, 8)
    b.extend([0, 1], [32, 32])
    kept = b.lists(random.Random(5), [0], 16, 8)
    kept[0, 0, 0, 3], kept[0, 0, 1, 12], kept[0, 0, 0, 13] = 20, 2, 32
    before = [p.clone() for p in b.pools]
    word = i32([0])
    pages = b.tables.tolist()
    pkb.evict_cache_rows(b.handle, i32([0]), i32(kept.tolist()), b.tables, b.lens, b.refs, sink=8,
                         status=word)
    assert word.item() == O.METADATA and b.lens.tolist() == [16, 32]
    free = set(range(9)) - set(pages[0]) - set(pages[1])
    for p, q in zip(b.pools, before):
        x, y = (t.view(torch.int16) for t in (p, q))
        for page in list(free) + pages[1] + pages[0][:1] + pages[0][2:]:
            assert torch.equal(x[page], y[page])
        at = pages[0][1]
        for h, j in ((1, 12), (0, 13)):
            for kv in range(2):
                assert torch.equal(x[at, kv, h, j - 8], y[at, kv, h, j - 8])


def test_large_pools_and_many_items():
    """More items than a planning CTA's threads, pages that a cluster hands out."""
    rng = random.Random(6)
    R, ps = 300, 8
    b = Rows(12, R, 3, 9000, ps, Hkv=1)
    b.extend([0], [20])
    b.fork([0] * (R - 1), list(range(1, R)))
    rows = rng.sample(range(R), R)
    b.evict(rows, b.lists(rng, rows, 10, Hkv=1))
    assert b.refs.max().item() == 1


def test_captured_calls_share_a_workspace():
    """Two captured evictions of different rows, replayed in turn, and one on another stream."""
    rng = random.Random(7)
    b, c = Rows(13, 3, 6, 30, 8), Rows(14, 3, 6, 30, 8)
    ws = torch.empty(pkb.evict_cache_workspace_size(3, 20, 8), dtype=torch.uint8, device=DEV)
    graphs = []
    for x in (b, c):
        x.extend([0, 1, 2], [40, 30, 44])
        x.kept = x.lists(rng, [2, 0, 1], 20)
        x.rows, x.dev = i32([2, 0, 1]), i32(x.kept.tolist())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkb.evict_cache_rows(x.handle, x.rows, x.dev, x.tables, x.lens, x.refs, weights=x.w,
                                 workspace=ws)
        graphs.append(g)
    for x, g in zip((b, c), graphs):
        g.replay()
        O.evict(x.o, [2, 0, 1], x.kept, 0, x.ow)
        x.same()
        assert np.array_equal(x.w.cpu().numpy(), x.ow)
    b.extend([0, 1, 2], [20, 20, 20])
    kept = b.lists(rng, [0, 1], 33)
    side = torch.cuda.Stream()
    rows, dev = i32([0, 1]), i32(kept.tolist())
    side.wait_stream(torch.cuda.current_stream())
    pkb.evict_cache_rows(b.handle, rows, dev, b.tables, b.lens, b.refs, stream=side)
    side.synchronize()
    O.evict(b.o, [0, 1], kept)
    b.same()


def test_empty_calls():
    b = Rows(15, 2, 2, 4, 8)
    b.evict([], np.zeros((1, 0, 2, 5), np.int64))
    b.evict([0, 1], np.zeros((1, 2, 2, 5), np.int64))       # empty rows


def test_pages_past_32_bits():
    """A pool of 2.5e9 elements: the tokens of its last pages move within them."""
    P, ps, L, K = 600_000, 16, 120, 40
    pool = torch.empty(P, 2, 1, ps, 128, dtype=torch.bfloat16, device=DEV)
    pages = [P - 1 - 3 * j for j in range(8)]
    pool[pages] = torch.randn(8, 2, 1, ps, 128, device=DEV).to(torch.bfloat16)
    held = pool[pages].transpose(0, 1).reshape(2, -1, 128).clone()
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    refs[pages] = 1
    tables, lens, word = i32([pages]), i32([L]), i32([0])
    kept = sorted(random.Random(15).sample(range(L), K))
    pkb.evict_cache_rows(pkb.cache_pools([pool]), i32([0]), i32([[[kept]]]), tables, lens, refs,
                         status=word)
    assert word.item() == 0 and lens.item() == K and tables.tolist() == [pages]
    now = pool[pages[:3]].transpose(0, 1).reshape(2, -1, 128)[:, :K]
    assert torch.equal(now, held[:, kept])
    assert refs[pages].tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
