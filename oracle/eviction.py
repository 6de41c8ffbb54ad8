"""Reference of the calls that keep rows within a budget of tokens: attention weights per token in
float64, and selection and eviction as sequential loops over whole numbers."""
import math

import numpy as np

from .cache import CAPACITY, METADATA


def weights(q, lse, keys, lens, starts, old, *, last=0, causal=True, scale=None, decay=1.0):
    """New weights [B][Hkv, L] from old ones [B][Hkv, >= L].  q [total, Hq, D], lse [total, Hq],
    keys [B] of [L, Hkv, D], starts [B + 1]."""
    out = []
    scale = scale or 1.0 / math.sqrt(q.shape[-1])
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        w = np.array(old[b], dtype=np.float64)[:, :L].copy()
        if n:
            before = max(L - n, 0)
            w[:, :before] = w[:, :before] * decay if decay else 0.0
            w[:, before:] = 0.0
        counted = min(n, last) if last else n
        G = q.shape[1] // keys[b].shape[1]
        for i in range(n - counted, n):
            row = starts[b] + i
            see = max(0, L - n + i + 1) if causal else L
            for h in range(q.shape[1]):
                if np.isneginf(lse[row, h]):
                    continue
                x = keys[b][:see, h // G].astype(np.float64) @ q[row, h].astype(np.float64)
                w[h // G, :see] += np.exp(x * scale - float(lse[row, h]))
        out.append(w)
    return out


def select(weights_, rows, lens, keep, sink=0, recent=0):
    """(kept [N, n, Hkv, keep], status) from weights [N, R, Hkv, W] fp32."""
    N, R, Hkv, W = weights_.shape
    kept = np.full((N, len(rows), Hkv, keep), -1, np.int64)
    status = 0
    for i, r in enumerate(rows):
        if not 0 <= r < R or not 0 <= lens[r] <= W:
            status |= METADATA
            continue
        L = int(lens[r])
        for layer in range(N):
            for h in range(Hkv):
                if L <= keep:
                    kept[layer, i, h, :L] = np.arange(L)
                    continue
                w = weights_[layer, r, h]
                must = [j for j in range(L) if j < sink or j >= L - recent]
                rest = [j for j in range(sink, L - recent)]
                rest.sort(key=lambda j: (math.isnan(w[j]), 0.0 if math.isnan(w[j]) else -w[j], j))
                kept[layer, i, h] = sorted(must + rest[:keep - len(must)])
    return kept, status


def evict(state, rows, kept, sink=0, weights_=None, combined=True):
    """Cuts rows of an oracle.cache.State back to the lists kept [N, n, Hkv, K]; weights [N, R, Hkv,
    W] move along.  The pools' heads are [2 Hkv] of a layer (combined) or K and V pools in turn."""
    N, _, Hkv, K = kept.shape
    items, seen = [], set()
    for i, r in enumerate(rows):
        listed = r in seen
        seen.add(r)
        ok = 0 <= r < state.R and not listed
        L = state.lens[r] if ok else -1
        pages = state.pages(L)
        ok = ok and L >= 0 and pages <= state.C
        if ok and L > K:
            ok = weights_ is None or L <= weights_.shape[-1]
            ok = ok and all(0 <= p < state.P for p in state.tables[r][:pages])
            ok = ok and bool((kept[:, i, :, 0] >= 0).all() and (kept[:, i, :, -1] >= K - 1).all()
                             and (kept[:, i, :, -1] < L).all())
        if not ok:
            state.status |= METADATA
            continue
        if L > K:
            shared = [j for j in range(sink // state.ps, state.pages(K))
                      if state.refs[state.tables[r][j]] > 1]
            items.append((i, r, L, shared))
    granted = state._grant([len(x[3]) for x in items])
    before = [p.copy() for p in state.pools]
    gone = []
    for (i, r, L, shared), pages in zip(items, granted):
        if pages is None:
            continue
        old = list(state.tables[r])
        gone += [old[j] for j in shared] + old[state.pages(K):state.pages(L)]
        for j, p in zip(shared, pages):
            state.tables[r][j] = p
            state.refs[p] = 1
        for layer in range(N):
            for h in range(Hkv):
                w = None if weights_ is None else weights_[layer, r, h].copy()
                for j, t in enumerate(kept[layer, i, h]):
                    src, dst = old[t // state.ps], state.tables[r][j // state.ps]
                    for kv in range(2):
                        pool = layer if combined else 2 * layer + kv
                        x = kv * Hkv + h if combined else h
                        state.pools[pool][dst, x, j % state.ps] = before[pool][src, x,
                                                                               t % state.ps]
                    if w is not None:
                        weights_[layer, r, h, j] = w[t]
        state.lens[r] = K
    for p in gone:
        state.refs[p] -= 1


__all__ = ["weights", "select", "evict", "CAPACITY", "METADATA"]
