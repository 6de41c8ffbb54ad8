"""The cache calls together, as a serving loop makes them, ending in the library's own prefill and
decode attention: extend, append (two layers), prefill, fork, decode steps, free, compact, decode."""
import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import cache as O
from tests.gpu_util import OUT_MAX_ABS, OUT_MEAN_ABS

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D, PS, R, C, P, LAYERS = 8, 2, 128, 16, 7, 12, 60, 2


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def attention(q, keys, values, first):
    """q [n, Hq, D] at positions first.. over keys, values [L, Hkv, D]: causal, float64."""
    out = np.empty(q.shape)
    for i in range(q.shape[0]):
        for h in range(HQ):
            g = h // (HQ // HKV)
            s = keys[:first + i + 1, g] @ q[i, h] / np.sqrt(D)
            w = np.exp(s - s.max())
            out[i, h] = (w / w.sum()) @ values[:first + i + 1, g]
    return out


@pytest.mark.parametrize("combined", [True, False])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_serving_loop(combined, layout):
    gen = torch.Generator().manual_seed(17)
    shape = (P, 2, HKV, PS, D) if combined else (P, HKV, PS, D)
    nan = float("nan")                               # nothing unwritten may be read
    caches = [torch.full(shape, nan, dtype=torch.bfloat16, device=DEV) if combined else
              tuple(torch.full(shape, nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
              for _ in range(LAYERS)]
    pools = pkb.cache_pools(caches)
    tables, lens = torch.full((R, C), -1, dtype=torch.int32, device=DEV), i32([0] * R)
    refs = i32([0] * P)
    table, m = pkb.rope_frequencies(D, scaling="yarn", factor=4.0, original_max_position=64)
    f, wm = O.frequencies(D, scaling="yarn", factor=4.0, original=64.0)
    indptr = torch.arange(R + 1, dtype=torch.int32, device=DEV) * C
    ws = torch.empty(max(pkb.extend_cache_workspace_size(R), pkb.fork_cache_workspace_size(R),
                         pkb.compact_cache_workspace_size(P)), dtype=torch.uint8, device=DEV)
    status = i32([0])
    held = [[(np.zeros((0, HKV, D)),) * 2 for _ in range(R)] for _ in range(LAYERS)]

    def views(cache):
        return (cache[:, 0].contiguous(), cache[:, 1].contiguous()) if combined else cache

    def step(new):
        """`new[r]` tokens for every row: one launch per layer over the packed rows."""
        starts = np.concatenate([[0], np.cumsum(new)]).tolist()
        rows = [r for r in range(R) if new[r]]
        pkb.extend_cache_rows(i32(rows), i32([new[r] for r in rows]), tables, lens, refs, PS,
                              workspace=ws)
        assert pkb.paged_attn_workspace_status(ws)[0] == pkb.OK
        for layer, cache in enumerate(caches):
            qkv = torch.randn(starts[-1], HQ + 2 * HKV, D, generator=gen).to(torch.bfloat16).to(DEV)
            q, k, v = qkv.split([HQ, HKV, HKV], dim=1)
            decode = all(n == 1 for n in new)
            where = (dict(paged_kv_indptr=indptr, paged_kv_indices=tables.view(-1)) if decode
                     else dict(block_tables=tables))
            qr = pkb.append_paged_kv_cache(k, v, cache, lens, q=q, freqs=table, layout=layout,
                                           attention_factor=m, status=status,
                                           qo_indptr=None if decode else i32(starts), **where)
            if decode:
                out, _ = pkb.batch_decode_with_paged_kv_cache(
                    qr, cache, None, indptr, tables.view(-1), lens, C * PS)
            else:
                kc, vc = views(cache)
                out, _ = pkb.batch_prefill_with_paged_kv_cache(
                    qr, kc, vc, i32(starts), tables, lens, page_size=PS, mask_type="causal")
            for r in rows:
                a, b = starts[r], starts[r + 1]
                first = held[layer][r][0].shape[0]
                pos = list(range(first, first + b - a))
                bf = lambda x: torch.from_numpy(x).to(torch.bfloat16).double().numpy()  # noqa: E731
                kk = bf(O.rotate(k[a:b], pos, f, layout=layout, m=wm)[0])
                qq = bf(O.rotate(q[a:b], pos, f, layout=layout, m=wm)[0])
                old = held[layer][r]
                held[layer][r] = (np.concatenate([old[0], kk]),
                                  np.concatenate([old[1], v[a:b].double().cpu().numpy()]))
                want = attention(qq, *held[layer][r], first)
                off = np.abs(out[a:b].double().cpu().numpy() - want)
                assert off.max() <= OUT_MAX_ABS and off.mean() <= OUT_MEAN_ABS, (r, off.max())

    def invariant():
        count = [0] * P
        for r in range(R):
            for p in tables[r, :-(-int(lens[r]) // PS)].tolist():
                count[p] += 1
        assert refs.tolist() == count

    step([40, 33, 5, 16, 0, 0, 0])                   # prompts
    pkb.fork_cache_rows(pools, i32([0, 0, 3]), i32([4, 5, 6]), tables, lens, refs, workspace=ws)
    assert pkb.paged_attn_workspace_status(ws)[0] == pkb.OK
    for layer in held:
        layer[4], layer[5], layer[6] = layer[0], layer[0], layer[3]
    invariant()
    step([1] * R)                                    # every row goes its own way from here
    step([20, 0, 3, 0, 1, 2, 17])                    # chunks behind cached tokens
    pkb.free_cache_rows(i32([1, 0]), tables, lens, refs, PS, status=status)
    for layer in held:
        layer[0] = layer[1] = (np.zeros((0, HKV, D)),) * 2
    _, _, live = pkb.compact_cache(pools, tables, lens, refs, workspace=ws)
    invariant()
    assert refs[:live.item()].ne(0).all() and refs[live.item():].eq(0).all()
    # pages above are given back: nothing below may depend on them
    for cache in caches:
        for t in (cache if isinstance(cache, tuple) else (cache,)):
            t[live.item():] = nan
    step([50, 31, 1, 1, 1, 1, 1])                    # two new prompts among running rows
    step([1] * R)
    invariant()
    assert status.item() == 0
