"""Decode behind a shared prefix of millions of tokens.

Tolerances.  |v| <= 1, so outputs are below 1.  A part of the prefix has at most 2^14 tiles of 128
keys, 2^17 additions into an accumulator that grows evenly and that the tensor core may truncate:
at worst 2^17 * 2^-23 / 2 = 7.8e-3.  The probabilities' rounding to bf16 is the same in every copy
of a page, at worst 2^-8, and the output's is 2^-8 again: 1.6e-2 in all, below the parity
contract's 2e-2.  The sum of a part's 2^14 tile sums in fp32 is off by 2^14 * 2^-24 = 1e-3 at
worst, sums inside a tile and the scores by some 1e-5 more, and so is its logarithm: 1.2e-3."""
import math

import pytest
import torch

import paged_kv_block_gb300 as pkb
from tests.gpu_util import check_lse, check_out

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_parts_end_long_before_a_wait_does():
    """1,240 requests of 64 rows are more tiles than the SMs need, so nothing but their length cuts
    the prefix of 8 million tokens into parts; as a single part it would take longer than the 0.1 s
    after which a wait gives up.  All of its pages are one page."""
    B, SQ, Hq, ps, copies, tail = 1240, 4, 16, 128, 62500, 5
    g = torch.Generator().manual_seed(31)
    pool = torch.randn(2, 2, 1, ps, 128, generator=g).to(torch.bfloat16)
    pool[:, 1].clamp_(-1, 1)
    pool[1, :, :, tail:] = math.nan
    q = torch.randn(B, SQ, Hq, 128, generator=g).to(torch.bfloat16)
    tables = torch.zeros(B, copies + 1, dtype=torch.int32, device=DEV)
    tables[:, copies] = 1
    n = copies * ps + tail
    kv, lse = pool.to(DEV), torch.empty(B, SQ, Hq, device=DEV)
    qd = q.to(DEV)
    ws = torch.empty(pkb.shared_prefix_workspace_size(qd, kv, n, 1, seq_len_q=SQ),
                     dtype=torch.uint8, device=DEV)
    out, _ = pkb.batch_decode_with_shared_prefix(
        qd, kv, ws, i32([b * (copies + 1) for b in range(B + 1)]), tables.view(-1), i32([n] * B), n,
        i32([0, B]), i32([copies * ps]), seq_len_q=SQ, lse=lse)
    assert pkb.paged_attn_workspace_status(ws)[1] == 0
    k, v = (torch.cat([pool[0, j, 0], pool[1, j, 0, :tail]]).double() for j in range(2))
    x = q.double() @ k.T * 128 ** -0.5
    x[..., :ps] += math.log(copies)
    check_out(out, (torch.softmax(x, -1) @ v).numpy())
    check_lse(lse, torch.logsumexp(x, -1).numpy(), 1.2e-3)
