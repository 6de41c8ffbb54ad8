"""Attention weights of large calls, and of batches in which many requests sit the call out."""
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle.eviction import METADATA
from tests.test_gpu_weights import Problem

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_units_longer_than_a_wait():
    """A unit of 16.7 million rows takes 0.16 s, longer than the 0.1 s after which a wait without
    progress gives up; five of them for every SM.  Scores and LSEs of 0 make every weight the number
    of rows, exactly: all partial sums are whole numbers below 2^24."""
    Hq, ps, T = 64, 128, 262143
    pages = 5 * torch.cuda.get_device_properties(0).multi_processor_count * 256 // ps
    q = torch.zeros(T, Hq, 256, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(pages, 2, 1, ps, 256, dtype=torch.bfloat16, device=DEV)
    lse, status = torch.zeros(T, Hq, device=DEV), i32([0])
    w = torch.full((1, 1, pages * ps), 7.0, device=DEV)
    pkb.accumulate_attention_weights(
        q, lse, cache, i32([pages * ps]), w, qo_indptr=i32([0, T]), mask_type="dense", decay=0.0,
        block_tables=torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1), status=status)
    assert status.item() == 0
    assert (w == T * Hq).all()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("idle,heavy", [(1, 20), (62, 30), (200, 90), (700, 130)])
def test_a_prompt_among_idle_requests(D, idle, heavy):
    """No more queries than requests, most of them of one: as if that one were alone."""
    lens = [40 + b % 23 for b in range(idle)] + [333]
    new = [1 if b % 9 == 4 else 0 for b in range(idle)] + [heavy]
    p = Problem(idle, lens, new, 8, 2, D, 16)
    p.run(decay=0.5)
    p.run(csr=True, last=7)


def test_more_prompts_than_the_schedule_lists():
    """600 requests with units, beside idle ones and single tokens."""
    new = [3 + b % 12 if b % 3 else b % 2 for b in range(900)]
    Problem(41, [20 + b % 150 for b in range(900)], new, 24, 2, 128, 16).run()


def test_a_captured_call_reads_who_sits_out():
    """Replays go by the offsets of the moment: all of 60 queries in one request, spread, one each,
    and offsets that leave the batch."""
    B, total = 60, 60
    lens = [70 + b % 31 for b in range(B)]
    spreads = [[60 if b == 17 else 0 for b in range(B)], [1] * B,
               [20 if b % 20 == 3 else 0 for b in range(B)]]
    problems = [Problem(50 + i, lens, new, 8, 2, 128, 16) for i, new in enumerate(spreads)]
    p = problems[0]
    q, lse = torch.empty_like(p.q, device=DEV), torch.empty_like(p.lse, device=DEV)
    qo, device_lens = i32([0] * (B + 1)), i32(lens)
    cache, w = p.cache.clone(), torch.empty_like(p.w, device=DEV)
    tables, status = torch.empty_like(i32(p.tables)), i32([0])

    def load(p):
        assert p.starts[-1] == total and p.cache.shape == cache.shape
        for to, x in ((q, p.q), (lse, p.lse), (qo, i32(p.starts)), (cache, p.cache), (w, p.w),
                      (tables, i32(p.tables))):
            to.copy_(x)
    load(p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkb.accumulate_attention_weights(q, lse, cache, device_lens, w, qo_indptr=qo,
                                         block_tables=tables, status=status)
    for p in problems + problems[::-1]:
        load(p)
        graph.replay()
        p.check(w)
        assert status.item() == 0
    load(p)
    qo.copy_(i32([0] * 18 + [10 ** 9] * 43))
    graph.replay()
    assert status.item() == METADATA
    assert torch.equal(w.nan_to_num(-1), p.w.to(DEV).nan_to_num(-1))
