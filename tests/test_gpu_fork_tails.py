"""Forks whose parent names a page outside the pool: nothing stale may become live."""
import pytest
import torch

import paged_kv_block_gb300 as pkb
from tests.test_gpu_cache_pages import Both

pytestmark = pytest.mark.gpu
METADATA = 4


@pytest.mark.parametrize("P", [30, 20000])
@pytest.mark.parametrize("bad", [-1, 1 << 30, "P"])
def test_a_bad_tail_leaves_the_item_out(P, bad):
    """The parent's partly filled page lies outside the pool: the child stays empty, takes no page
    and leaves the pages to the items behind it, the same child's next item among them."""
    b = Both(40, 8, 4, P, 16, Hkv=1, layers=2)
    b.extend([0, 1, 2], [40, 10, 33])
    t = b.tables.tolist()
    t[0][2] = P if bad == "P" else bad               # row 0: two full pages, then this one
    b.set(tables=t)
    before = [p.clone() for p in b.pools]
    b.fork([0, 1, 0], [3, 4, 5])
    lens, refs = b.lens.tolist(), b.refs.tolist()
    assert lens == [40, 10, 33, 0, 10, 0, 0, 0]
    assert refs[0] == refs[1] == 1 and b.tables[3].eq(-1).all() and b.tables[5].eq(-1).all()
    fresh = int(b.tables[4, 0])
    for now, old in zip(b.pools, before):
        keep = [p for p in range(P) if p != fresh]
        assert torch.equal(now.view(torch.int16)[keep], old.view(torch.int16)[keep])
    b.fork([0, 2], [6, 6])                           # the child belongs to its first item in order
    assert b.lens[6] == 33
    b.fork([0], [7])                                 # alone: the whole call does nothing
    assert b.lens[7] == 0


def test_a_bad_tail_takes_no_page_from_the_last_one():
    """One free page, wanted by a bad item and by a good one behind it."""
    b = Both(41, 4, 2, 3, 16, Hkv=1)
    b.extend([0, 1], [10, 10])
    t = b.tables.tolist()
    t[0][0] = 77
    b.set(tables=t)
    b.fork([0, 1], [2, 3])
    assert b.lens.tolist() == [10, 10, 0, 10] and b._ws_status() == METADATA


def test_many_bad_tails():
    """More items than a CTA has threads, every third of them with a bad tail."""
    R = 3000
    b = Both(42, R, 2, 9000, 8, Hkv=1)
    half = R // 2
    b.extend(list(range(half)), [1 + r % 16 for r in range(half)])
    t = b.tables.tolist()
    for r in range(0, half, 3):
        t[r][r % 16 // 8] = -7                       # the page of the row's last token
    b.set(tables=t)
    b.fork(list(range(half)), list(range(half, R)))
    for r in range(half):
        n = 1 + r % 16
        want = 0 if r % 3 == 0 and n % 8 else n
        assert int(b.o.lens[half + r]) == want


def test_bad_full_pages_are_copied_as_they_are():
    """An id outside the pool in the place of a full page: the child holds what its parent holds
    there, and no count changes for it."""
    b = Both(43, 3, 4, 12, 16, Hkv=1)
    b.extend([0, 1], [40, 32])
    t = b.tables.tolist()
    t[0][1], t[1][0] = 50, -3
    b.set(tables=t)
    b.fork([0], [2])
    assert b.lens[2] == 40 and b.tables[2, 1] == 50 and b.refs[t[0][0]] == 2
    status, _ = pkb.paged_attn_workspace_status(b.ws)
    assert status == pkb.ERR_METADATA
    b.free([2])
    b.fork([1], [2])
    assert b.lens[2] == 32 and b.tables[2, 0] == -3
