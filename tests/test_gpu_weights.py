"""Attention weight per cached token on the GPU against the float64 oracle.

Tolerance.  A score is a sum of D products of bf16 values, exact in fp32, added in fp32.  Partial
sums stay below some 300 in magnitude for these inputs (|q.k| of 256 columns with deviations 1.5 and
1 is below 6 * 24), so the D / 16 additions of MMA steps and the 16 inside each are off by 256 *
2^-24 * 300 = 4.6e-3 at the very worst and, their signs being random, by a sixteenth of it; times
the scale (1/16, 1/11) and a Gaussian spread over steps that leaves 1e-5 to 3e-5 in the exponent.
With |scale q.k| and |lse| below 32 the products scale * score, log2(e) * lse and their difference
add 3 * 2^-24 * 47 = 8.4e-6, the exponential's approximation 2^-22.  Sums of up to 2^14 positive
terms in chains of at most 2^10 add 2^-14 = 6e-5 at the worst.  So RTOL = 1e-4 relative to the sum
of positive terms, which is the result itself."""
import math

import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import eviction as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
RTOL = 1e-4


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Problem:
    """Requests of `lens` tokens whose last `new` are queries; nothing unwritten may be read: the
    pools are NaN outside the live tokens, the weights past every length."""

    def __init__(self, seed, lens, new, Hq, Hkv, D, ps, *, combined=True, causal=True, W=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.ps, self.causal = lens, new, ps, causal
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        B, G = len(lens), Hq // Hkv
        need = [-(-n // ps) for n in lens]
        P = sum(need) + 3
        perm = torch.randperm(P, generator=g).tolist()
        C = max(need + [1])
        self.tables, at = [], 0
        pool = torch.full((P, 2, Hkv, ps, D), math.nan).to(torch.bfloat16)
        self.keys = []
        for b, n in enumerate(lens):
            row = perm[at:at + need[b]]
            at += need[b]
            self.tables.append(row + [-1] * (C - need[b]))
            k = torch.randn(n, Hkv, D, generator=g).to(torch.bfloat16)
            for j in range(n):
                pool[row[j // ps], 0, :, j % ps] = k[j]
            self.keys.append(k.double().numpy())
        self.starts = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.q = (1.5 * torch.randn(self.starts[-1], Hq, D, generator=g)).to(torch.bfloat16)
        self.lse = torch.empty(self.starts[-1], Hq)
        for b, n in enumerate(lens):
            for i in range(new[b]):
                r = self.starts[b] + i
                see = max(0, n - new[b] + i + 1) if causal else n
                for h in range(Hq):
                    x = self.keys[b][:see, h // G] @ self.q[r, h].double().numpy()
                    self.lse[r, h] = float(torch.logsumexp(torch.from_numpy(x) * D ** -0.5, 0))
        self.W = W or max(lens + [1]) + 5
        self.old = torch.rand(B, Hkv, self.W, generator=g)
        self.w = self.old.clone()
        for b, n in enumerate(lens):
            self.w[b, :, n:] = math.nan
        self.cache = pool.to(DEV) if combined else (pool[:, 0].contiguous().to(DEV),
                                                    torch.empty_like(pool[:, 1]).to(DEV))

    def run(self, *, csr=False, fixed=False, last=0, decay=1.0, **kw):
        w = self.w.to(DEV)
        q, lse = self.q.to(DEV), self.lse.to(DEV)
        if fixed:
            n = self.new[0]
            shape = (len(self.lens),) + ((n,) if n > 1 else ()) + (self.Hq,)
            q, lse = q.view(shape + (self.D,)), lse.view(shape)
        else:
            kw["qo_indptr"] = i32(self.starts)
        if csr:
            need = [-(-n // self.ps) for n in self.lens]
            kw["paged_kv_indices"] = i32([p for n, row in zip(need, self.tables) for p in row[:n]])
            kw["paged_kv_indptr"] = i32(np.concatenate([[0], np.cumsum(need)]).tolist())
        else:
            kw["block_tables"] = i32(self.tables)
        status = i32([0])
        got = pkb.accumulate_attention_weights(q, lse, self.cache, i32(self.lens), w, decay=decay,
                                               last_queries=last, status=status,
                                               mask_type="causal" if self.causal else "dense", **kw)
        assert got is w and status.item() == 0
        self.check(w, last, decay)
        return w

    def check(self, w, last=0, decay=1.0):
        want = O.weights(self.q.double().numpy(), self.lse.numpy(), self.keys, self.lens,
                         self.starts, self.old.numpy(), last=last, causal=self.causal, decay=decay)
        w = w.cpu().numpy()
        for b, n in enumerate(self.lens):
            np.testing.assert_allclose(w[b, :, :n], want[b], rtol=RTOL, atol=1e-7)
            assert np.array_equal(w[b, :, n:], self.w[b, :, n:].numpy(), equal_nan=True)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (5, 1), (24, 2), (16, 1), (64, 1)])
@pytest.mark.parametrize("D", [128, 256])
def test_one_query_per_request(Hq, Hkv, D):
    p = Problem(Hq + D, [1, 2, 15, 16, 17, 128, 129, 300], [1] * 8, Hq, Hkv, D, 16)
    p.run(fixed=True)
    p.run(csr=True, decay=0.5)


@pytest.mark.parametrize("ps,combined", [(8, True), (24, False), (64, True), (128, False)])
def test_page_sizes(ps, combined):
    p = Problem(ps, [500, 7, 129], [1, 1, 1], 8, 2, 128, ps, combined=combined)
    p.run()
    p.run(csr=True, fixed=True, decay=0.0)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new", [[2, 2, 2], [3, 1, 8], [40, 7, 0], [150, 300, 1], [300, 130, 257]])
@pytest.mark.parametrize("causal", [True, False])
def test_several_queries(D, new, causal):
    lens = [300, 300, 257]
    p = Problem(sum(new), lens, new, 8, 2, D, 16, causal=causal)
    p.run(fixed=len(set(new)) == 1, decay=0.75)
    p.run(last=5)
    if max(new) > 100:
        p.run(last=128)


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (5, 1), (24, 2), (7, 1), (64, 1), (48, 1)])
def test_head_groups_of_prompts(Hq, Hkv):
    p = Problem(Hq, [200, 131], [200, 60], Hq, Hkv, 128, 32, combined=False)
    p.run()
    p.run(csr=True, last=33)


def test_longer_prompt():
    p = Problem(5, [1500], [1400], 4, 1, 128, 16)
    p.run()
    p.run(last=1000)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (256, 8, 2), (128, 5, 1), (256, 24, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_wide_tiles(D, Hq, Hkv, causal):
    """Weights wide enough, by their shape, for key tiles of 256."""
    p = Problem(D + Hq, [700, 300, 513], [700, 251, 400], Hq, Hkv, D, 24, causal=causal, W=60000)
    p.run(decay=0.5)
    p.run(last=300)


@pytest.mark.parametrize("B", [31, 33, 140])
def test_many_prompts(B):
    """The order in which units are handed out goes over 32 requests at a time."""
    lens = [1 + (37 * b) % 290 for b in range(B)]
    Problem(B, lens, [max(1, n // 2) for n in lens], 8, 2, 128, 16).run()


def test_more_queries_than_keys():
    """Queries before the first key see nothing."""
    p = Problem(6, [3, 40], [10, 41], 8, 2, 128, 16)
    p.run()


def test_rows_that_see_nothing():
    """An LSE of -inf adds nothing, and +inf neither."""
    p = Problem(7, [100, 90], [1, 1], 8, 2, 128, 16)
    p.lse[0, ::2] = -math.inf
    p.lse[1, 1] = math.inf
    p.run()
    p = Problem(8, [200], [150], 8, 2, 128, 16)
    p.lse[::3, 1] = -math.inf
    p.run()


def test_a_nan_stays_with_its_request():
    """Padding rows and other requests' queries of NaN reach nobody else's weights."""
    for new in ([1, 1, 1], [140, 130, 9]):
        p = Problem(9, [300, 140, 60], new, 8, 2, 128, 16)
        clean = p.run().clone()
        p.q[p.starts[1]:p.starts[2]] = math.nan
        q = torch.cat([p.q, torch.full((5, 8, 128), math.nan).to(torch.bfloat16)]).to(DEV)
        lse = torch.cat([p.lse, torch.full((5, 8), math.nan)]).to(DEV)
        w = p.w.to(DEV)
        pkb.accumulate_attention_weights(q, lse, p.cache, i32(p.lens), w, qo_indptr=i32(p.starts),
                                         block_tables=i32(p.tables))
        for b in (0, 2):
            assert torch.equal(w[b].nan_to_num(-1), clean[b].nan_to_num(-1))


def test_bad_metadata():
    p = Problem(10, [100, 90, 80], [1, 1, 1], 8, 2, 128, 16, W=85)
    args = p.q.to(DEV), p.lse.to(DEV), p.cache
    tables = [list(r) for r in p.tables]
    tables[2][1], tables[2][3] = 999, -1
    w, status = p.old.to(DEV), i32([0])
    pkb.accumulate_attention_weights(*args, i32(p.lens), w, block_tables=i32(tables), status=status)
    assert status.item() == O.METADATA
    want = O.weights(p.q.double().numpy(), p.lse.numpy(), p.keys, p.lens, p.starts,
                     np.pad(p.old.numpy(), ((0, 0), (0, 0), (0, 50))))
    w = w.cpu().numpy()
    for b in (0, 1):                          # longer than W: the first W tokens
        np.testing.assert_allclose(w[b], want[b][:, :85], rtol=RTOL, atol=1e-7)
    bad = np.zeros(80, bool)
    bad[16:32] = bad[48:64] = True
    np.testing.assert_allclose(w[2][:, :80][:, ~bad], want[2][:, ~bad], rtol=RTOL, atol=1e-7)
    assert np.array_equal(w[2][:, :80][:, bad], p.old.numpy()[2][:, :80][:, bad])
    # offsets that leave the batch: those requests are left out
    w, status = p.old.to(DEV), i32([0])
    pkb.accumulate_attention_weights(*args, i32([20, 20, 20]), w, block_tables=i32(p.tables),
                                     qo_indptr=i32([0, 1, 7, 3]), status=status)
    assert status.item() == O.METADATA
    assert torch.equal(w[1:].cpu(), p.old[1:])
    # a CSR row with fewer entries than its length needs
    w, status = p.old.to(DEV), i32([0])
    flat = i32(sum(p.tables, []))
    pkb.accumulate_attention_weights(*args, i32([60, 60, 60]), w, paged_kv_indices=flat,
                                     paged_kv_indptr=i32([0, 2, 2, 9]), status=status)
    assert status.item() == O.METADATA
    assert torch.equal(w[:, :, 60:].cpu(), p.old[:, :, 60:]) and torch.equal(w[1].cpu(), p.old[1])


@pytest.mark.parametrize("new", [1, 150])
def test_calls_repeat_bit_for_bit(new):
    """Also when captured, replayed and run on another stream."""
    p = Problem(11, [400, 333], [new, new], 8, 2, 128, 16)
    first = p.run()
    args = p.q.to(DEV), p.lse.to(DEV), p.cache, i32(p.lens)
    kw = dict(block_tables=i32(p.tables), qo_indptr=i32(p.starts))
    w = p.w.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkb.accumulate_attention_weights(*args, w, **kw)
    for _ in range(2):
        w.copy_(p.w)
        graph.replay()
        assert torch.equal(w.nan_to_num(-1), first.nan_to_num(-1))
    w.copy_(p.w)
    side.wait_stream(torch.cuda.current_stream())
    pkb.accumulate_attention_weights(*args, w, stream=side, **kw)
    side.synchronize()
    assert torch.equal(w.nan_to_num(-1), first.nan_to_num(-1))


def test_weights_of_a_step_sum_to_its_queries():
    """One step of each query head adds a total weight of G to its KV head."""
    p = Problem(12, [777, 65], [1, 1], 32, 8, 128, 16)
    p.old.zero_()
    p.w = torch.where(p.w.isnan(), p.w, torch.zeros_like(p.w))
    w = p.run(fixed=True)
    total = w.nan_to_num(0).sum(-1).cpu()
    assert torch.allclose(total, torch.full_like(total, 4.0), rtol=1e-4)


@pytest.mark.parametrize("busy", [1, 150])
def test_requests_without_queries_are_left_alone(busy):
    """Whatever their length: rows of a batch that sit a call out."""
    p = Problem(13, [200, 190, 64], [busy, 0, 2], 8, 2, 128, 16)
    w, status = p.w.to(DEV), i32([0])
    pkb.accumulate_attention_weights(p.q.to(DEV), p.lse.to(DEV), p.cache, i32([200, 10 ** 6, 64]),
                                     w, block_tables=i32(p.tables), qo_indptr=i32(p.starts),
                                     status=status)
    assert status.item() == 0
    p.check(w)


@pytest.mark.parametrize("new", [1, 150])
def test_pages_past_32_bits(new):
    """A cache of 2.5e9 elements, its last pages in use."""
    p = Problem(14, [400, 333], [new, new], 8, 1, 128, 16)
    small, P = p.cache, 600_000
    p.cache = torch.empty(P, 2, 1, 16, 128, dtype=torch.bfloat16, device=DEV)
    p.cache[P - small.shape[0]:] = small
    p.tables = [[t + P - small.shape[0] if t >= 0 else t for t in r] for r in p.tables]
    p.run()


def test_prompts_beside_single_tokens():
    """One request with many queries in a batch of few on average, and the other way round."""
    Problem(15, [300] + [40 + b for b in range(20)], [90] + [1] * 20, 4, 2, 128, 16).run()
    Problem(16, [700, 50, 20, 90], [300, 1, 0, 1], 8, 2, 256, 16).run(csr=True)


@pytest.mark.parametrize("D", [128, 256])
def test_a_prompt_in_a_large_batch_of_single_tokens(D):
    """Both kinds in one call, beyond the requests that the schedule keeps at hand; also with an
    invalid page in each."""
    new = [1] * 150
    new[140], new[7], new[60], new[61] = 70, 9, 0, 8
    p = Problem(17, [100 + b % 13 for b in range(150)], new, 4, 1, D, 16)
    p.run()
    p.run(last=3)
    p.run(csr=True, decay=0.5)
    tables = [list(r) for r in p.tables]
    tables[140][2] = tables[30][1] = 10 ** 6
    w, status = p.w.to(DEV), i32([0])
    pkb.accumulate_attention_weights(p.q.to(DEV), p.lse.to(DEV), p.cache, i32(p.lens), w,
                                     block_tables=i32(tables), qo_indptr=i32(p.starts),
                                     status=status)
    assert status.item() == O.METADATA
    clean = p.run()
    for b in range(150):
        skip = {140: slice(32, 48), 30: slice(16, 32)}.get(b, slice(0, 0))
        x, y = w[b, :, :p.lens[b]].clone(), clean[b, :, :p.lens[b]].clone()
        assert torch.equal(x[:, skip].cpu(), p.old[b][:, :p.lens[b]][:, skip])
        x[:, skip] = y[:, skip] = 0
        assert torch.equal(x, y)
