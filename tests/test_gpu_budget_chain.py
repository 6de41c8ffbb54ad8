"""Shared prompts and full rows, as a serving loop meets them: prompts are prefilled, forked into
samples that decode behind their common prefix, attention weights add up, and rows that outgrow
their budget are cut back, after which decoding goes on.  Every output against float64 over what
each row holds."""
import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import cache as OC
from oracle import eviction as O
from tests.gpu_util import LSE_ABS, OUT_MAX_ABS, OUT_MEAN_ABS

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D, PS, R, C, P, LAYERS = 8, 2, 128, 16, 6, 14, 70, 2
W = C * PS


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Loop:
    def __init__(self, combined):
        self.gen = torch.Generator().manual_seed(23)
        shape = (P, 2, HKV, PS, D) if combined else (P, HKV, PS, D)
        nan = float("nan")                   # nothing unwritten may be read

        def pool():
            return torch.full(shape, nan, dtype=torch.bfloat16, device=DEV)
        self.caches = [pool() if combined else (pool(), pool()) for _ in range(LAYERS)]
        self.pools = pkb.cache_pools(self.caches)
        self.tables = torch.full((R, C), -1, dtype=torch.int32, device=DEV)
        self.lens, self.refs, self.status = i32([0] * R), i32([0] * P), i32([0])
        self.weights = torch.full((LAYERS, R, HKV, W), nan, device=DEV)
        self.freqs, _ = pkb.rope_frequencies(D)
        self.f = OC.frequencies(D)[0]
        self.indptr = torch.arange(R + 1, dtype=torch.int32, device=DEV) * C
        self.position = [0] * R              # the next token's, whatever was evicted
        empty = np.zeros((HKV, 0, D)), np.zeros((HKV, 0, D)), np.zeros((HKV, 0))
        self.held = [[empty for _ in range(R)] for _ in range(LAYERS)]

    def attend(self, layer, r, q):
        """q [n, HQ, D], the last tokens of row r: outputs, LSEs, weights [HKV, L] of the row."""
        k, v, _ = self.held[layer][r]
        n, L = q.shape[0], k.shape[1]
        out, lse, w = np.empty(q.shape), np.empty((n, HQ)), np.zeros((HKV, L))
        for i in range(n):
            see = L - n + i + 1
            for h in range(HQ):
                g = h // (HQ // HKV)
                s = k[g, :see] @ q[i, h] / np.sqrt(D)
                lse[i, h] = np.log(np.exp(s - s.max()).sum()) + s.max()
                p = np.exp(s - lse[i, h])
                out[i, h] = p @ v[g, :see]
                w[g, :see] += p
        return out, lse, w

    def step(self, new, groups=None):
        """`new[r]` tokens for every row; groups: (group_indptr, prefix_lens) of a decode step."""
        starts = np.concatenate([[0], np.cumsum(new)]).tolist()
        rows = [r for r in range(R) if new[r]]
        pkb.extend_cache_rows(i32(rows), i32([new[r] for r in rows]), self.tables, self.lens,
                              self.refs, PS, status=self.status)
        pos = [p for r in range(R) for p in range(self.position[r], self.position[r] + new[r])]
        for layer, cache in enumerate(self.caches):
            qkv = torch.randn(starts[-1], HQ + 2 * HKV, D, generator=self.gen)
            q, k, v = (1.5 * qkv).to(torch.bfloat16).to(DEV).split([HQ, HKV, HKV], dim=1)
            qr, kr = pkb.rotary_embedding(q, i32(pos), self.freqs, k=k)
            packed = dict(qo_indptr=None if groups else i32(starts))
            pkb.append_paged_kv_cache(kr, v, cache, self.lens, block_tables=self.tables, **packed)
            lse = torch.empty(starts[-1], HQ, device=DEV)
            if groups:
                out, _ = pkb.batch_decode_with_shared_prefix(
                    qr, cache, None, self.indptr, self.tables.view(-1), self.lens, W,
                    i32(groups[0]), i32(groups[1]), mask_type="causal", lse=lse)
            else:
                kc, vc = ((cache[:, 0].contiguous(), cache[:, 1].contiguous())
                          if torch.is_tensor(cache) else cache)
                out, _ = pkb.batch_prefill_with_paged_kv_cache(
                    qr, kc, vc, i32(starts), self.tables, self.lens, page_size=PS,
                    mask_type="causal", lse=lse)
            pkb.accumulate_attention_weights(qr, lse, cache, self.lens, self.weights[layer],
                                             block_tables=self.tables, status=self.status,
                                             **packed)
            got = self.weights[layer].cpu().numpy()
            for r in rows:
                a, b = starts[r], starts[r + 1]
                grow = [np.concatenate([x, y.double().cpu().numpy().swapaxes(0, 1)], 1)
                        for x, y in zip(self.held[layer][r], (kr[a:b], v[a:b]))]
                w = np.concatenate([self.held[layer][r][2], np.zeros((HKV, b - a))], 1)
                self.held[layer][r] = (*grow, w)
                want, want_lse, add = self.attend(layer, r, qr[a:b].double().cpu().numpy())
                off = np.abs(out[a:b].double().cpu().numpy() - want)
                assert off.max() <= OUT_MAX_ABS and off.mean() <= OUT_MEAN_ABS, (r, off.max())
                assert np.abs(lse[a:b].cpu().numpy() - want_lse).max() <= LSE_ABS
                # weights: relative to LSEs that are off by LSE_ABS at most, step after step
                w += add
                np.testing.assert_allclose(got[r, :, :w.shape[1]], w, rtol=2 * LSE_ABS, atol=1e-5)
        for r in rows:
            self.position[r] += new[r]

    def cut(self, rows, keep, sink, recent):
        kept = pkb.select_cache_tokens(i32(rows), self.weights, self.lens, keep, sink=sink,
                                       recent=recent, status=self.status)
        lens = self.lens.tolist()
        want, _ = O.select(self.weights.cpu().numpy(), rows, lens, keep, sink, recent)
        assert np.array_equal(kept.cpu().numpy(), want)
        pkb.evict_cache_rows(self.pools, i32(rows), kept, self.tables, self.lens, self.refs,
                             weights=self.weights, sink=sink, status=self.status)
        for i, r in enumerate(rows):
            if lens[r] <= keep:
                continue
            for layer in range(LAYERS):
                x = self.held[layer][r]
                self.held[layer][r] = tuple(
                    np.stack([t[h][want[layer, i, h]] for h in range(HKV)]) for t in x)

    def invariant(self):
        assert self.status.item() == 0
        count = [0] * P
        for r in range(R):
            assert self.lens[r].item() == self.held[0][r][0].shape[1]
            for p in self.tables[r, :-(-int(self.lens[r]) // PS)].tolist():
                count[p] += 1
        assert self.refs.tolist() == count


@pytest.mark.parametrize("combined", [True, False])
def test_samples_of_shared_prompts_within_a_budget(combined):
    loop = Loop(combined)
    loop.step([100, 0, 0, 61, 0, 30])                # three prompts
    # samples: rows 0 to 2 of the first, 3 and 4 of the second
    pkb.fork_cache_rows(loop.pools, i32([0, 0, 3]), i32([1, 2, 4]), loop.tables, loop.lens,
                        loop.refs, status=loop.status)
    loop.weights[:, 1:3], loop.weights[:, 4] = loop.weights[:, :1], loop.weights[:, 3]
    for layer in loop.held:
        layer[1], layer[2], layer[4] = layer[0], layer[0], layer[3]
    for r, of in ((1, 0), (2, 0), (4, 3)):
        loop.position[r] = loop.position[of]
    loop.invariant()
    groups = [0, 3, 5, 6], [100, 61, 30]
    for _ in range(3):
        loop.step([1] * R, groups)
    # back to 48 tokens; the page of the first 16 stays shared, the others are taken out of sharing
    loop.cut([4, 1, 0, 2, 5], 48, 16, 8)
    loop.invariant()
    first = loop.tables[:3, 0].tolist()
    assert first == [first[0]] * 3 and loop.refs[first[0]].item() == 3
    groups = [0, 3, 5, 6], [16, 16, 0]
    for _ in range(2):
        loop.step([1] * R, groups)
    loop.step([20, 1, 0, 5, 33, 2])                  # chunks
    loop.cut(list(range(R)), 40, 16, 10)
    loop.step([1] * R, groups)
    loop.invariant()
