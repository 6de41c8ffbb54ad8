"""Cases of the operators for caches that are shared or full: decode attention for requests with a
common prefix, and keeping a row within a budget of tokens by the attention that they received.

A prompt that is forked into many samples, or a long system prompt, sits once in the cache;
decode attention can read it once for all of its requests.  A row that outgrows its budget is
cut back: the attention weights of its tokens are added up as attention runs, the tokens to keep
are selected by them, and the kept keys and values move to the row's front.

`run` computes a case with plain torch operations, or, with `own` set, with the library.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"


def listed():
    return [
        # Eight samples of one prompt of a thousand tokens, a few tokens into their answers.
        # Latency counts.
        dict(name="shared_few", op="shared", groups=1, members=8, prefix_max=1000, tail_max=48,
             q_heads=32, kv_heads=8, queries=1, page_size=16, combined=True),
        # 64 requests behind one long system prompt, each with a question of its own.
        dict(name="shared_prompt", op="shared", groups=1, members=64, prefix_max=8192,
             tail_max=512, q_heads=32, kv_heads=8, queries=1, page_size=16, combined=True),
        # 13 prompts with 1 to 32 samples each, two queries per request (one of them drafted),
        # in separate pools.
        dict(name="shared_groups", op="shared", groups=13, members=32, prefix_max=4099,
             tail_max=301, q_heads=64, kv_heads=8, queries=2, page_size=32, combined=False),
        # The weights of one short request's tokens after a decode step.
        dict(name="weights_one", op="weights", batch=1, len_max=700, new_max=1, last=0,
             q_heads=8, kv_heads=2, head_dim=128, page_size=16, combined=True, decay=1.0),
        # The same for a decode batch of 64 requests, older weights fading.
        dict(name="weights_decode", op="weights", batch=64, len_max=8192, new_max=1, last=0,
             q_heads=32, kv_heads=8, head_dim=128, page_size=16, combined=True, decay=0.9375),
        # After a batch of prompts: what their last 32 queries look at (an observation window).
        dict(name="weights_window", op="weights", batch=16, len_max=4096, new_max=4096, last=32,
             q_heads=24, kv_heads=2, head_dim=256, page_size=32, combined=False, decay=1.0),
        # What all queries of four long prompts look at.
        dict(name="weights_prompt", op="weights", batch=4, len_max=8192, new_max=8192, last=0,
             q_heads=32, kv_heads=8, head_dim=128, page_size=32, combined=False, decay=1.0),
        # A row of two thousand tokens to be cut to 512.
        dict(name="select_one", op="select", layers=1, rows=1, kv_heads=8, len_max=2048,
             keep=512, sink=4, recent=64),
        # Every layer of 32 long rows.
        dict(name="select_many", op="select", layers=8, rows=32, kv_heads=8, len_max=8192,
             keep=2048, sink=4, recent=256),
        # One row with a very long context.
        dict(name="select_long", op="select", layers=1, rows=1, kv_heads=2, len_max=131072,
             keep=16384, sink=16, recent=1024),
        # One row of one layer gets room for 64 tokens and is cut back to its budget.
        dict(name="evict_one", op="evict", layers=1, rows=1, keep=509, new=64, sink=4,
             kv_heads=2, head_dim=128, page_size=16, combined=False, shared=0),
        # 32 rows of 8 layers get room for a chunk of 512 tokens each and are cut back; their
        # first pages were shared when they were forked.
        dict(name="evict_many", op="evict", layers=8, rows=32, keep=2048, new=512, sink=16,
             kv_heads=8, head_dim=128, page_size=16, combined=True, shared=512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "weights", "select", "evict"])
    page_size = rng.choice([16, 16, 32, 64, 128, 24])
    combined = rng.random() < 0.5
    if op == "shared":
        q_heads, kv_heads = rng.choice([(32, 8), (8, 2), (64, 8), (4, 4), (5, 1), (16, 1)])
        queries = rng.choice([1, 1, 1, 2, 4])
        groups = _log_int(rng, 1, 40)
        members = _log_int(rng, 1, max(1, 200 // groups))
        tail_max = _log_int(rng, queries, 700)
        prefix_max = _log_int(rng, 1, 16384 // groups + 300)
        return dict(op=op, groups=groups, members=members, prefix_max=prefix_max,
                    tail_max=tail_max, q_heads=q_heads, kv_heads=kv_heads, queries=queries,
                    page_size=page_size, combined=combined)
    if op == "weights":
        q_heads, kv_heads, head_dim = rng.choice([(32, 8, 128), (8, 2, 128), (64, 8, 128),
                                                  (24, 2, 256), (4, 4, 128), (7, 1, 128)])
        new_max = rng.choice([1, 1, 2, 4, _log_int(rng, 5, 6000)])
        len_max = max(new_max, _log_int(rng, 1, 8192))
        # no more pairs of a query and a key than the largest listed case
        pairs = 4e9 * 128 / (len_max * new_max * q_heads * head_dim)
        tokens = 2.5e9 / (len_max * kv_heads * head_dim * 4)
        batch = _log_int(rng, 1, max(1, min(128, int(pairs), int(tokens))))
        return dict(op=op, batch=batch, len_max=len_max, new_max=new_max,
                    last=rng.choice([0, 0, 16, 32]) if new_max > 4 else 0, q_heads=q_heads,
                    kv_heads=kv_heads, head_dim=head_dim, page_size=page_size, combined=combined,
                    decay=rng.choice([1.0, 1.0, 0.5, 0.0]))
    if op == "select":
        kv_heads = rng.choice([1, 2, 4, 8])
        len_max = _log_int(rng, 8, 131072)
        layers = _log_int(rng, 1, 16)
        rows = _log_int(rng, 1, max(1, min(64, (1 << 24) // (len_max * layers * kv_heads))))
        keep = _log_int(rng, 1, len_max)
        sink = rng.randint(0, min(keep, 16))
        return dict(op=op, layers=layers, rows=rows, kv_heads=kv_heads, len_max=len_max, keep=keep,
                    sink=sink, recent=rng.randint(0, keep - sink))
    kv_heads, head_dim = rng.choice([(8, 128), (2, 128), (2, 256), (4, 64), (1, 80)])
    layers = _log_int(rng, 1, 16)
    rows = _log_int(rng, 1, 64)
    most = 1e9 / (layers * rows * kv_heads * head_dim * 4)
    keep = _log_int(rng, 1, max(2, min(8192, int(most))))
    return dict(op=op, layers=layers, rows=rows, keep=keep,
                new=_log_int(rng, 1, max(2, min(1024, int(most) // 2))),
                sink=rng.randint(0, min(keep, 40)), kv_heads=kv_heads, head_dim=head_dim,
                page_size=page_size, combined=combined, shared=rng.choice([0, 0, keep // 2]))


# ---- inputs ---------------------------------------------------------------------------------

def _spread(lo, hi, n):
    """n whole numbers from hi down to lo: the same ones for every seed, so shapes are too."""
    return np.linspace(hi, lo, n).astype(np.int64)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def _i32(a):
    return _dev(np.asarray(a).astype(np.int32))


def _pools(case, P, gen):
    """The layers' caches: [N, P, 2, Hkv, ps, D], or K and V pools [N, P, Hkv, ps, D]."""
    shape = (case["kv_heads"], case["page_size"], case.get("head_dim", 128))
    n = case.get("layers", 1)

    def normal(*s):
        return torch.randn(s, generator=gen, device=DEVICE, dtype=torch.bfloat16)
    if case["combined"]:
        return dict(kv=normal(n, P, 2, *shape))
    return dict(k_pool=normal(n, P, *shape), v_pool=normal(n, P, *shape))


def _caches(s):
    return (s["kv"],) if "kv" in s else (s["k_pool"], s["v_pool"])


def _members(case):
    return _spread(max(1, case["members"] // 8), case["members"], case["groups"])


def _prefixes(case):
    return _spread(max(1, case["prefix_max"] // 4), case["prefix_max"], case["groups"])


def _tails(case):
    n = int(_members(case).sum())
    return _spread(max(case["queries"], case["tail_max"] // 8), case["tail_max"], n)


def _lens(case):
    """(lengths, new tokens) of a weights case; new tokens are the last ones of each length."""
    lens = _spread(max(case["new_max"], case["len_max"] // 4), case["len_max"], case["batch"])
    new = np.minimum(lens, case["new_max"])
    if case["new_max"] > 4:                  # prompts: all of their tokens are new
        new = np.minimum(new, _spread(case["new_max"] // 4 + 1, case["new_max"], case["batch"]))
    return lens, new


def _pages_of(lens, ps, rng, spare=1.05):
    """Rows of distinct pages drawn from one permutation; unused entries are -1."""
    need = -(-lens // ps)
    P = int(need.sum() * spare) + 1
    perm = rng.permutation(P)
    tables = np.full((len(lens), max(1, int(need.max()))), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        tables[r, :n] = perm[at:at + n]
        at += n
    return tables, P


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    s = dict(case=case)
    return {**s, **dict(shared=_prepare_shared, weights=_prepare_weights, select=_prepare_select,
                        evict=_prepare_evict)[case["op"]](case, gen, rng)}


def _queries(gen, *shape):
    """Queries that look at some keys far more than at others, as a model's do."""
    return (2.0 * torch.randn(shape, generator=gen, device=DEVICE)).to(torch.bfloat16)


def _prepare_shared(case, gen, rng):
    ps, SQ = case["page_size"], case["queries"]
    members, prefixes = _members(case), rng.permutation(_prefixes(case))
    tails = rng.permutation(_tails(case))
    B = len(tails)
    group = np.repeat(np.arange(case["groups"]), members)
    lens = prefixes[group] + tails
    # A prompt's full pages are shared; its partly filled one was copied for every sample.
    full = prefixes[group] // ps
    own_pages = -(-lens // ps) - full
    first = np.concatenate([[0], np.cumsum(members)])
    P = int((prefixes // ps).sum() + own_pages.sum()) + 7
    perm = rng.permutation(P)
    tables = np.full((B, int((-(-lens // ps)).max())), -1, np.int32)
    at = 0
    for g in range(case["groups"]):
        n = prefixes[g] // ps
        tables[first[g]:first[g + 1], :n] = perm[at:at + n]
        at += n
    for b in range(B):
        tables[b, full[b]:full[b] + own_pages[b]] = perm[at:at + own_pages[b]]
        at += own_pages[b]
    s = _pools(case, P, gen)
    for g in range(case["groups"]):
        left = prefixes[g] % ps
        if left:
            src = int(tables[first[g], prefixes[g] // ps])
            dst = _dev(tables[first[g]:first[g + 1], prefixes[g] // ps].astype(np.int64))
            for pool in _caches(s):
                pool[0][dst, ..., :left, :] = pool[0][src, ..., :left, :].clone()
    shape = (B, case["q_heads"], 128) if SQ == 1 else (B, SQ, case["q_heads"], 128)
    C = tables.shape[1]
    return dict(s, q=_queries(gen, *shape), lens=_i32(lens), group_indptr=_i32(first),
                prefix_lens=_i32(prefixes), indices=_dev(tables.reshape(-1)),
                indptr=_i32(np.arange(B + 1) * C), tables=_dev(tables), max_len=int(lens.max()))


def _prepare_weights(case, gen, rng):
    lens, new = _lens(case)
    order = rng.permutation(case["batch"])
    lens, new = lens[order], new[order]
    tables, P = _pages_of(lens, case["page_size"], rng)
    s = dict(_pools(case, P, gen), case=case)
    B, Hq = case["batch"], case["q_heads"]
    starts = np.concatenate([[0], np.cumsum(new)])
    s.update(q=_queries(gen, int(starts[-1]), Hq, case["head_dim"]), lens=_i32(lens),
             qo_indptr=_i32(starts), starts=starts.tolist(), host_lens=lens.tolist(),
             tables=_dev(tables),
             weights=torch.rand((B, case["kv_heads"], case["len_max"] + 64), generator=gen,
                                device=DEVICE))
    # what the attention call before it returned
    s["lse"] = torch.empty((int(starts[-1]), Hq), device=DEVICE)
    for b in range(B):
        _, n = _range(s, b)
        q0 = s["starts"][b + 1] - n
        s["lse"][s["starts"][b]:q0] = 0.0
        for g, scores, visible, q1, m in _scores(s, b, torch.float32):
            part = torch.logsumexp(scores.masked_fill(~visible[:, None], -math.inf), dim=-1)
            s["lse"][q1:q1 + m, g[0]:g[1]] = part
    if case["new_max"] == 1:                 # one query per request: [B, Hq, D]
        s["q_arg"], s["qo_arg"] = s["q"], None
    else:
        s["q_arg"], s["qo_arg"] = s["q"], s["qo_indptr"]
    return s


def _prepare_select(case, gen, rng):
    N, R, W = case["layers"], case["rows"], case["len_max"]
    w = torch.rand((N, R + 1, case["kv_heads"], W), generator=gen, device=DEVICE)
    w = w.pow(4)
    w = torch.where(w < 0.05, torch.zeros_like(w), w)      # tokens that nothing looked at
    lens = np.concatenate([rng.permutation(_spread(max(1, W // 2), W, R)), [W // 3]])
    return dict(weights=w, lens=_i32(lens), rows=_i32(rng.permutation(R)))


def _prepare_evict(case, gen, rng):
    N, R, ps, K, new = (case[k] for k in ("layers", "rows", "page_size", "keep", "new"))
    Hkv = case["kv_heads"]
    need, most = -(-K // ps), -(-(K + new) // ps)
    both = min(case["shared"], K) // ps if R > 1 else 0    # pages that all rows share
    P = both + R * (most + need - both) + 3
    perm = rng.permutation(P)
    tables = np.full((R, most), -1, np.int32)
    tables[:, :both] = perm[:both]
    refs = np.zeros(P, np.int32)
    refs[perm[:both]] = R
    at = both
    for r in range(R):
        tables[r, both:need] = perm[at:at + need - both]
        refs[perm[at:at + need - both]] = 1
        at += need - both
    s = _pools(case, P, gen)
    # any ascending choice that keeps the first `sink` tokens
    score = torch.rand((N, R, Hkv, K + new), generator=gen, device=DEVICE)
    score[..., :case["sink"]] = 2.0
    kept = score.topk(K, dim=-1).indices.sort(dim=-1).values.to(torch.int32)
    weights = torch.rand((N, R, Hkv, most * ps), generator=gen, device=DEVICE)
    return dict(s, kept=kept, weights=weights, tables=_dev(tables), refs=_dev(refs),
                lens=_i32(np.full(R, K)), rows=_i32(rng.permutation(R)),
                room=_i32(np.full(R, new)))


# ---- the plain forms ------------------------------------------------------------------------

def _keys(s, b, L, dtype, values=False):
    """Keys (or values) of request b, [L, Hkv, D]."""
    ps = s["case"]["page_size"]
    pages = s["tables"][b, :-(-L // ps)].long()
    if "kv" in s:
        x = s["kv"][0][pages, 1 if values else 0]
    else:
        x = s["v_pool" if values else "k_pool"][0][pages]
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:L].to(dtype)


def _plain_shared(s):
    case = s["case"]
    Hq, Hkv, SQ = case["q_heads"], case["kv_heads"], case["queries"]
    q = s["q"].view(-1, SQ, Hkv, Hq // Hkv, 128).float()
    out = torch.empty((q.shape[0], SQ, Hq, 128), device=DEVICE)
    lse = torch.empty((q.shape[0], SQ, Hq), device=DEVICE)
    members, lens = s["group_indptr"].tolist(), s["lens"].tolist()
    step = torch.arange(SQ, device=DEVICE)
    for g, pre in enumerate(s["prefix_lens"].tolist()):
        first, last = members[g], members[g + 1]
        k, v = (_keys(s, first, pre, torch.float32, values=x) for x in (False, True))
        head = torch.einsum("btgid,jgd->btgij", q[first:last], k) / math.sqrt(128)
        for b in range(first, last):
            L = lens[b]
            tail_k, tail_v = (_keys(s, b, L, torch.float32, values=x)[pre:] for x in (False, True))
            tail = torch.einsum("tgid,jgd->tgij", q[b], tail_k) / math.sqrt(128)
            scores = torch.cat([head[b - first], tail], dim=-1)
            late = torch.arange(L, device=DEVICE) > (L - SQ + step)[:, None]
            scores = scores.masked_fill(late[:, None, None], -math.inf)
            top = scores.amax(dim=-1, keepdim=True)
            e = torch.exp(scores - top)
            total = e.sum(dim=-1, keepdim=True)
            o = (torch.einsum("tgij,jgd->tgid", e[..., :pre], v)
                 + torch.einsum("tgij,jgd->tgid", e[..., pre:], tail_v)) / total
            out[b] = o.reshape(SQ, Hq, 128)
            lse[b] = (top + torch.log(total)).reshape(SQ, Hq)
    shape = s["q"].shape
    return out.view(shape).to(torch.bfloat16), lse.view(shape[:-1])


def _range(s, b):
    """(length, queries that count) of request b."""
    n = s["starts"][b + 1] - s["starts"][b]
    last = s["case"]["last"]
    return s["host_lens"][b], min(n, last) if last else n


def _scores(s, b, dtype):
    """Scores of the counted queries of request b, a KV head and some queries at a time:
    ((first, last query head), scores [m, heads, L], visible [m, L], first query row, m)."""
    case = s["case"]
    L, n = _range(s, b)
    G = case["q_heads"] // case["kv_heads"]
    k = _keys(s, b, L, dtype)
    row0 = s["starts"][b + 1] - n
    j = torch.arange(L, device=DEVICE)
    step = max(1, (1 << 28) // (L * G))
    for h in range(case["kv_heads"]):
        for i in range(0, n, step):
            m = min(step, n - i)
            q = s["q"][row0 + i:row0 + i + m, h * G:(h + 1) * G].to(dtype)
            scores = (q.reshape(m * G, -1) @ k[:, h].T).view(m, G, L) / math.sqrt(q.shape[-1])
            position = L - n + i + torch.arange(m, device=DEVICE)
            yield (h * G, (h + 1) * G), scores, j <= position[:, None], row0 + i, m


def _weights_of(s, b, dtype):
    """Attention weights of the tokens of request b, summed over its counted queries: [Hkv, L]."""
    case = s["case"]
    total = torch.zeros((case["kv_heads"], s["host_lens"][b]), dtype=dtype, device=DEVICE)
    G = case["q_heads"] // case["kv_heads"]
    for g, scores, visible, row, m in _scores(s, b, dtype):
        p = torch.exp(scores - s["lse"][row:row + m, g[0]:g[1], None].to(dtype))
        total[g[0] // G] += torch.where(visible[:, None], p, torch.zeros_like(p)).sum(dim=(0, 1))
    return total


def _plain_weights(s):
    w, decay = s["weights"], s["case"]["decay"]
    for b, L in enumerate(s["host_lens"]):
        old = L - (s["starts"][b + 1] - s["starts"][b])
        add = _weights_of(s, b, torch.float32)
        w[b, :, :old] = w[b, :, :old] * decay + add[:, :old]
        w[b, :, old:L] = add[:, old:]
    return w


def _plain_select(s):
    case = s["case"]
    N, Hkv, W = case["layers"], case["kv_heads"], case["len_max"]
    K, sink, recent = case["keep"], case["sink"], case["recent"]
    rows = s["rows"].long()
    w = s["weights"][:, rows]
    L = s["lens"][rows].long()[None, :, None, None]
    j = torch.arange(W, device=DEVICE)
    # rank: must-keep tokens first, then by weight, the lowest index first among equals
    key = torch.where((j < sink) | (j >= L - recent), torch.full_like(w, math.inf), w)
    key = torch.where(j < L, key, torch.full_like(w, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept = torch.sort(order[..., :K], dim=-1).values
    if kept.shape[-1] < K:
        kept = torch.nn.functional.pad(kept, (0, K - kept.shape[-1]))
    slot = torch.arange(K, device=DEVICE)
    whole = torch.where(slot < L, slot, torch.full_like(slot, -1)).expand(N, -1, Hkv, K)
    return torch.where(L > K, kept, whole).to(torch.int32)


def _plain_evict(s):
    case = s["case"]
    N, R, ps, K, Hkv = (case[k] for k in ("layers", "rows", "page_size", "keep", "kv_heads"))
    rows, tables, refs, lens = s["rows"].long(), s["tables"], s["refs"], s["lens"]
    slots = torch.arange(tables.shape[1], device=DEVICE)
    # room for the new tokens: the lowest free pages, in the order of the rows
    have, want = (lens[rows] + ps - 1) // ps, (lens[rows] + s["room"] + ps - 1) // ps
    free = torch.nonzero(refs == 0).flatten()
    first = torch.cumsum(want - have, 0) - (want - have)
    fresh = (slots >= have[:, None]) & (slots < want[:, None])
    pages = free[(first[:, None] + slots - have[:, None]).clamp(0, free.numel() - 1)]
    tables[rows] = torch.where(fresh, pages.int(), tables[rows])
    refs.index_add_(0, pages.flatten(), fresh.flatten().int())
    lens[rows] += s["room"]
    # pages whose contents change and that others share are replaced
    old = tables[rows]
    mine = (slots >= case["sink"] // ps) & (slots < -(-K // ps))
    shared = mine & (refs[old.clamp(min=0).long()] > 1)
    free = torch.nonzero(refs == 0).flatten()
    rank = torch.cumsum(shared.flatten(), 0).view(shared.shape) - 1
    pages = free[rank.clamp(0, free.numel() - 1)]
    now = torch.where(shared, pages.int(), old)
    # the kept tokens move
    kept = s["kept"].long()
    layer = torch.arange(N, device=DEVICE)[:, None, None, None]
    head = torch.arange(Hkv, device=DEVICE)[None, None, :, None]
    item = torch.arange(R, device=DEVICE)[None, :, None, None]
    to = torch.arange(K, device=DEVICE)
    src = layer, old[item, kept // ps].long(), head, kept % ps
    dst = layer, now[item, to // ps].long(), head, to % ps
    if "kv" in s:
        for j in range(2):
            pool = s["kv"][:, :, j]
            pool[dst] = pool[src]
    else:
        for pool in (s["k_pool"], s["v_pool"]):
            pool[dst] = pool[src]
    s["weights"][:, rows, :, :K] = s["weights"][:, rows].gather(-1, kept)
    # replaced pages and those past the new lengths go back
    gone = shared | ((slots >= -(-K // ps)) & (slots < -(-(K + case["new"]) // ps)))
    refs.index_add_(0, old.clamp(min=0).long().flatten(), -gone.flatten().int())
    refs.index_add_(0, pages.flatten(), shared.flatten().int())
    tables[rows] = now
    lens[rows] = K
    return (tables, lens, refs, s["weights"]) + _caches(s)


# ---- the library's calls --------------------------------------------------------------------

def _cache(s):
    return s["kv"][0] if "kv" in s else (s["k_pool"][0], s["v_pool"][0])


def _own_shared(s):
    import paged_kv_block_gb300 as pkb
    if "workspace" not in s:                 # a program keeps it from step to step
        s["workspace"] = torch.empty(pkb.shared_prefix_workspace_size(
            s["q"], _cache(s), s["max_len"], s["prefix_lens"].numel(),
            seq_len_q=s["case"]["queries"]), dtype=torch.uint8, device=DEVICE)
    lse = torch.empty(s["q"].shape[:-1], dtype=torch.float32, device=DEVICE)
    return pkb.batch_decode_with_shared_prefix(
        s["q"], _cache(s), s["workspace"], s["indptr"], s["indices"], s["lens"], s["max_len"],
        s["group_indptr"], s["prefix_lens"], seq_len_q=s["case"]["queries"], mask_type="causal",
        lse=lse)


def _own_weights(s):
    import paged_kv_block_gb300 as pkb
    return pkb.accumulate_attention_weights(
        s["q_arg"], s["lse"], _cache(s), s["lens"], s["weights"], block_tables=s["tables"],
        qo_indptr=s["qo_arg"], last_queries=s["case"]["last"], decay=s["case"]["decay"])


def _own_select(s):
    import paged_kv_block_gb300 as pkb
    case = s["case"]
    return pkb.select_cache_tokens(s["rows"], s["weights"], s["lens"], case["keep"],
                                   sink=case["sink"], recent=case["recent"])


def _own_evict(s):
    import paged_kv_block_gb300 as pkb
    case = s["case"]
    if "pools" not in s:
        s["pools"] = pkb.cache_pools(list(s["kv"]) if "kv" in s
                                     else list(zip(s["k_pool"], s["v_pool"])))
        s["workspace"] = torch.empty(
            max(pkb.extend_cache_workspace_size(case["rows"]),
                pkb.evict_cache_workspace_size(case["rows"], case["keep"], case["page_size"])),
            dtype=torch.uint8, device=DEVICE)
    pkb.extend_cache_rows(s["rows"], s["room"], s["tables"], s["lens"], s["refs"],
                          case["page_size"], workspace=s["workspace"])
    pkb.evict_cache_rows(s["pools"], s["rows"], s["kept"], s["tables"], s["lens"], s["refs"],
                         weights=s["weights"], sink=case["sink"], workspace=s["workspace"])
    return (s["tables"], s["lens"], s["refs"], s["weights"]) + _caches(s)


_PLAIN = dict(shared=_plain_shared, weights=_plain_weights, select=_plain_select,
              evict=_plain_evict)
_OWN = dict(shared=_own_shared, weights=_own_weights, select=_own_select, evict=_own_evict)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "shared":
        rows = int(_members(case).sum()) * case["queries"] * case["q_heads"]
        token = case["kv_heads"] * 128 * 4
        tails = int(_tails(case).sum())
        keys = float((_members(case) * _prefixes(case)).sum() + tails)
        return dict(bytes=(int(_prefixes(case).sum()) + tails) * token + rows * (128 * 4 + 4),
                    flops=4 * 128 * keys * case["queries"] * case["q_heads"])
    if op == "weights":
        lens, new = _lens(case)
        n = np.minimum(new, case["last"]) if case["last"] else new
        pairs = float((n * lens - n * (n - 1) / 2).sum())
        keys = int(lens.sum()) * case["kv_heads"]
        rows = int(n.sum()) * case["q_heads"]
        return dict(bytes=keys * (case["head_dim"] * 2 + 8) + rows * (case["head_dim"] * 2 + 4),
                    flops=2 * case["head_dim"] * pairs * case["q_heads"])
    if op == "select":
        lens = _spread(max(1, case["len_max"] // 2), case["len_max"], case["rows"])
        lists = case["layers"] * case["kv_heads"]
        return dict(bytes=4 * lists * (int(lens.sum()) + case["rows"] * case["keep"]), flops=0)
    # the kept tokens behind the first one that goes move: all but one part in new + 1 of them
    moved = (case["keep"] - case["sink"]) * case["new"] / (case["new"] + 1)
    heads = case["layers"] * case["rows"] * case["kv_heads"]
    return dict(bytes=heads * (moved * (2 * case["head_dim"] * 4 + 8) + 4 * case["keep"]), flops=0)


# ---- the definition in 64 bits --------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("select", "evict"):
        return None                          # indices and copies: exact by themselves
    s = prepare(case, seed)
    if case["op"] == "shared":
        return _exact_shared(s, case)
    return _exact_weights(s, case)


def _exact_shared(s, case):
    """Each request for itself over all of its own pages."""
    Hq, SQ, ps = case["q_heads"], case["queries"], case["page_size"]
    G = Hq // case["kv_heads"]
    q = s["q"].double().reshape(-1, SQ, Hq, 128)
    out = torch.empty(q.shape, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(q.shape[:-1], dtype=torch.float64, device=DEVICE)
    k_pool = s["kv"][0][:, 0] if "kv" in s else s["k_pool"][0]
    v_pool = s["kv"][0][:, 1] if "kv" in s else s["v_pool"][0]
    for b, L in enumerate(s["lens"].tolist()):
        at = torch.arange(L, device=DEVICE)
        page = s["tables"][b].long()[at // ps]
        k = k_pool[page, :, at % ps].double().repeat_interleave(G, dim=1)      # [L, Hq, D]
        v = v_pool[page, :, at % ps].double().repeat_interleave(G, dim=1)
        for t in range(SQ):
            n = L - SQ + t + 1
            x = (k[:n] * q[b, t]).sum(-1) * 128.0 ** -0.5                      # [n, Hq]
            lse[b, t] = torch.logsumexp(x, dim=0)
            out[b, t] = (torch.exp(x - lse[b, t])[..., None] * v[:n]).sum(0)
    return [out.reshape(s["q"].shape), lse.reshape(s["q"].shape[:-1])]


def _exact_weights(s, case):
    ps, D = case["page_size"], case["head_dim"]
    G = case["q_heads"] // case["kv_heads"]
    lens, starts = s["lens"].tolist(), s["qo_indptr"].tolist()
    rows = sum(starts[b + 1] - starts[b] for b in range(len(lens)))
    if rows * max(lens) * case["q_heads"] * D > 8e12:
        return None
    w = s["weights"].double()
    pool = s["kv"][0][:, 0] if "kv" in s else s["k_pool"][0]
    for b, L in enumerate(lens):
        at = torch.arange(L, device=DEVICE)
        k = pool[s["tables"][b].long()[at // ps], :, at % ps].double()         # [L, Hkv, D]
        n = starts[b + 1] - starts[b]
        counted = n if not case["last"] else min(n, case["last"])
        w[b, :, :L - n] *= case["decay"]
        w[b, :, L - n:L] = 0.0
        for i0 in range(0, counted, 1024):
            i1 = min(counted, i0 + 1024)
            r = starts[b + 1] - counted + torch.arange(i0, i1, device=DEVICE)
            last_key = L - counted + torch.arange(i0, i1, device=DEVICE)
            for h in range(case["q_heads"]):
                x = torch.mm(k[:, h // G], s["q"][r, h].double().T) / D ** 0.5  # [L, queries]
                e = torch.exp(x - s["lse"][r, h].double())
                e[at[:, None] > last_key] = 0.0
                w[b, h // G, :L] += e.sum(1)
    return w
