"""What extend, fork and compact report to a caller who keeps no workspace: shortages and items that
broke their contract, in a status word that is OR-ed into."""
import pytest
import torch

import paged_kv_block_gb300 as pkb
from tests.test_gpu_cache_pages import Both, i32

pytestmark = pytest.mark.gpu
CAPACITY, METADATA = 2, 4


def state(b):
    return b.tables, b.lens, b.refs


@pytest.mark.parametrize("P", [10, 9000])
def test_shortages_are_reported_without_a_workspace(P):
    """One CTA plans the small pool, a cluster the large one (all but ten of its pages in use)."""
    b = Both(50, 6, 8, P, 16)
    b.set(refs=[0] * 10 + [1] * (P - 10))
    word = i32([0])
    pkb.extend_cache_rows(i32([0, 1]), i32([64, 50]), *state(b), 16, status=word)
    assert word.item() == 0 and b.lens.tolist()[:2] == [64, 50]
    pkb.extend_cache_rows(i32([2]), i32([33]), *state(b), 16, status=word)      # 3 of 2 pages
    assert word.item() == CAPACITY and b.lens[2] == 0
    pkb.extend_cache_rows(i32([2]), i32([16]), *state(b), 16, status=word)      # kept, not cleared
    assert word.item() == CAPACITY and b.lens[2] == 16
    word.zero_()
    pkb.fork_cache_rows(b.handle, i32([1]), i32([3]), *state(b), status=word)   # the last page
    assert word.item() == 0 and b.lens[3] == 50
    pkb.fork_cache_rows(b.handle, i32([1]), i32([4]), *state(b), status=word)
    assert word.item() == CAPACITY and b.lens[4] == 0
    pkb.fork_cache_rows(b.handle, i32([0]), i32([4]), *state(b), status=word)   # needs none
    assert word.item() == CAPACITY and b.lens[4] == 64
    word.fill_(8)
    pkb.extend_cache_rows(i32([0, 9]), i32([1, 1]), *state(b), 16, status=word)
    assert word.item() == 8 | CAPACITY | METADATA


@pytest.mark.parametrize("P,n", [(40, 1), (9000, 1), (9000, 30)])
def test_bad_items_are_reported_without_a_workspace(P, n):
    """Forks of a few small pages are one kernel, others two: both report."""
    b = Both(51, 40, 8, P, 16, layers=2)
    b.extend([0, 1], [40, 50])
    word = i32([0])
    children = list(range(2, 2 + n))
    pkb.fork_cache_rows(b.handle, i32([0] * n), i32(children), *state(b), status=word)
    assert word.item() == 0
    pkb.free_cache_rows(i32(children), *state(b), 16)
    pkb.fork_cache_rows(b.handle, i32([0] * n), i32([0] * n), *state(b), status=word)
    assert word.item() == METADATA
    word.zero_()
    good = b.tables[0, 1].clone()
    b.tables[0, 1] = P                               # a full page: found while the table is copied
    pkb.fork_cache_rows(b.handle, i32([0] * n), i32(children), *state(b), status=word)
    assert word.item() == METADATA
    pkb.free_cache_rows(i32(children), *state(b), 16)
    word.zero_()
    pkb.compact_cache(b.handle, *state(b), status=word)
    assert word.item() == METADATA
    b.tables[0, 1] = good
    word.zero_()
    pkb.compact_cache(b.handle, *state(b), status=word)
    assert word.item() == 0
    b.lens[1] = 1000                                 # longer than its table row
    pkb.compact_cache(b.handle, *state(b), status=word)
    assert word.item() == METADATA


def test_the_workspace_reports_as_before():
    """A status word beside a workspace: both say the same, only the workspace's is cleared."""
    b = Both(52, 4, 4, 5, 16)
    word = i32([0])
    pkb.extend_cache_rows(i32([0]), i32([100]), *state(b), 16, workspace=b.ws, status=word)
    assert word.item() == METADATA == b._ws_status()
    pkb.extend_cache_rows(i32([0]), i32([20]), *state(b), 16, workspace=b.ws, status=word)
    assert word.item() == METADATA and b._ws_status() == 0
    pkb.extend_cache_rows(i32([1]), i32([64]), *state(b), 16, workspace=b.ws, status=word)
    assert word.item() == METADATA | CAPACITY and b._ws_status() == CAPACITY
    none = i32([])
    pkb.extend_cache_rows(none, none, *state(b), 16, workspace=b.ws, status=word)
    pkb.fork_cache_rows(b.handle, none, none, *state(b), workspace=b.ws, status=word)
    assert word.item() == METADATA | CAPACITY and b._ws_status() == 0


def test_a_step_stops_before_it_overwrites_live_tokens():
    """A row that could not grow keeps its length, so appending to it would write over its last
    tokens, in a page that its fork shares: the status says so before the append is enqueued."""
    P, ps, D = 4, 16, 8
    cache = torch.zeros(P, 2, 1, ps, D, dtype=torch.bfloat16, device="cuda")
    pools = pkb.cache_pools([cache])
    tables, lens = torch.full((3, 4), -1, dtype=torch.int32, device="cuda"), i32([0, 0, 0])
    refs, word = i32([0] * P), i32([0])

    def step(rows, new):
        """The README's order: pages first, then, if all got theirs, the new rows."""
        word.zero_()
        pkb.extend_cache_rows(i32(rows), i32(new), tables, lens, refs, ps, status=word)
        if word.item():
            return False
        starts = [0]
        for r in range(3):
            starts.append(starts[-1] + (new[rows.index(r)] if r in rows else 0))
        k = torch.arange(1, 1 + starts[-1], device="cuda").view(-1, 1, 1).expand(-1, 1, D)
        k = k.to(torch.bfloat16).contiguous()
        pkb.append_paged_kv_cache(k, k, cache, lens, qo_indptr=i32(starts), block_tables=tables)
        return True

    assert step([0], [32])
    pkb.fork_cache_rows(pools, i32([0]), i32([1]), tables, lens, refs, status=word)
    assert word.item() == 0 and refs.tolist() == [2, 2, 0, 0]
    assert step([2], [32])
    before = cache.clone()
    assert not step([0], [3])
    assert torch.equal(cache, before) and lens.tolist() == [32, 32, 32]
    pkb.free_cache_rows(i32([2]), tables, lens, refs, ps)
    assert step([0], [3])
    shared = tables[1, :2].long()
    assert torch.equal(cache[shared], before[shared]) and lens.tolist() == [35, 32, 0]


def test_a_captured_call_reports_at_every_replay():
    b = Both(53, 3, 4, 5, 16)
    word, rows, new = i32([0]), i32([0]), i32([16])

    def grow():
        pkb.extend_cache_rows(rows, new, *state(b), 16, workspace=b.ws, status=word)
    grow()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grow()
    for want in (0, 0, 0, METADATA):                 # four pages fill the row
        graph.replay()
        assert word.item() == want
    b.lens.zero_()
    word.zero_()
    graph.replay()                                   # the fifth page
    assert word.item() == 0
    b.lens.zero_()
    graph.replay()
    assert word.item() == CAPACITY


def test_refusals():
    b = Both(54, 3, 4, 10, 16)
    one = i32([0])
    for word in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, device="cuda").double(),
                 i32([]), i32([0, 0, 0, 0])[::2]):
        for call in (lambda: pkb.extend_cache_rows(one, one, *state(b), 16, status=word),
                     lambda: pkb.fork_cache_rows(b.handle, one, one, *state(b), status=word),
                     lambda: pkb.compact_cache(b.handle, *state(b), status=word)):
            with pytest.raises(ValueError):
                call()
