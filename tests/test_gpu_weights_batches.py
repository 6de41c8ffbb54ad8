"""Attention weights of large calls, and of batches in which many requests sit the call out."""
import pytest
import torch

import paged_kv_block_gb300 as pkb

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_units_longer_than_a_wait():
    """A unit of 16.7 million rows takes longer than the 0.1 s after which a wait without progress
    gives up; five of them for every SM.  Scores and LSEs of 0 make every weight the number of rows,
    exactly: all partial sums are whole numbers below 2^24."""
    Hq, ps, T = 64, 128, 262143
    pages = 5 * torch.cuda.get_device_properties(0).multi_processor_count * 256 // ps
    q = torch.zeros(T, Hq, 128, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(pages, 2, 1, ps, 128, dtype=torch.bfloat16, device=DEV)
    lse, status = torch.zeros(T, Hq, device=DEV), i32([0])
    w = torch.full((1, 1, pages * ps), 7.0, device=DEV)
    pkb.accumulate_attention_weights(
        q, lse, cache, i32([pages * ps]), w, qo_indptr=i32([0, T]), mask_type="dense", decay=0.0,
        block_tables=torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1), status=status)
    assert status.item() == 0
    assert (w == T * Hq).all()
