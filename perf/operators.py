"""Cases of the cache-side operators: rotary positions, appending new keys and values to the paged
cache, and copying, forking, recycling and compacting its pages.

A serving step that ends in this library's prefill or decode attention first rotates queries
and keys, writes the new K/V rows through the page table and keeps track of which request
owns which page.  Each case below is one such call (or the two calls that always come as a
pair: rows are freed before they are forked into or handed to a new request).

`run` computes a case with plain torch operations, or, with `own` set, with the library.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # One decode step of 64 requests: the queries and new keys of one layer.  Latency counts.
        dict(name="rope_decode", op="rope", tokens=64, q_heads=32, kv_heads=8, head_dim=128,
             rotary_dim=128, layout="half", scaling="none", factor=1.0, dtype="bf16",
             inverse=False, max_position=8192),
        # The gradient of a long fp32 batch whose heads rotate only their first 64 columns, in
        # the interleaved layout, with frequencies scaled for a long context and far positions.
        dict(name="rope_gradient_fp32", op="rope", tokens=32749, q_heads=24, kv_heads=2,
             head_dim=256, rotary_dim=64, layout="interleaved", scaling="yarn", factor=16.0,
             dtype="fp32", inverse=True, max_position=1000003),
        # One decode step of 64 requests: one token each, rotated and written into a combined
        # cache of 16-token pages through the CSR table that decode attention reads.
        dict(name="append_decode", op="append", batch=64, packed=False, new_max=1, prefix_max=4096,
             q_heads=32, kv_heads=8, head_dim=128, rotary_dim=128, layout="half",
             scaling="wavelength", factor=8.0, dtype="bf16", page_size=16, combined=True),
        # A batch of prompt chunks out of one fused projection (strided rows), 128 to 2048 tokens
        # each behind a cached prefix, into separate pools of 32-token pages.
        dict(name="append_prefill", op="append", batch=16, packed=True, new_max=2048,
             prefix_max=2048, q_heads=32, kv_heads=8, head_dim=128, rotary_dim=128, layout="half",
             scaling="none", factor=1.0, dtype="bf16", page_size=32, combined=False),
        # Duplicating a prompt's few pages in one layer's pool (copy on write of a shared page).
        dict(name="copy_few", op="copy", layers=1, pool_pages=512, pages=7, kv_heads=8,
             head_dim=128, page_size=16, combined=True),
        # Moving the pages of preempted requests aside in every layer.
        dict(name="copy_many", op="copy", layers=8, pool_pages=3000, pages=1201, kv_heads=8,
             head_dim=128, page_size=16, combined=True),
        # One request is forked once (a second sample of the same prompt).
        dict(name="fork_one", op="fork", layers=1, parents=1, children=1, max_len=1000,
             kv_heads=2, head_dim=128, page_size=16, combined=False),
        # Parallel samples: 32 prompts, about 8 samples of each, in 8 layers' caches.
        dict(name="fork_samples", op="fork", layers=8, parents=32, children=256, max_len=1500,
             kv_heads=8, head_dim=128, page_size=16, combined=True),
        # One finished request's row goes to a new prompt, in a small pool.
        dict(name="recycle_one", op="recycle", rows=16, pool_pages=1024, recycled=1,
             max_tokens=700, page_size=16),
        # Many rows change hands at once in a pool of 262,144 pages.
        dict(name="recycle_many", op="recycle", rows=512, pool_pages=262144, recycled=128,
             max_tokens=8192, page_size=16),
        # A small cache is compacted after a few requests have left.
        dict(name="compact_small", op="compact", layers=1, pool_pages=256, rows=8, live=0.5,
             kv_heads=2, head_dim=128, page_size=16, combined=False),
        # A large cache, half of it free, compacted so that its upper half can be given back.
        dict(name="compact_large", op="compact", layers=4, pool_pages=6007, rows=96, live=0.5,
             kv_heads=8, head_dim=128, page_size=16, combined=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "copy", "fork", "recycle", "compact"])
    q_heads, kv_heads, head_dim = rng.choice([(32, 8, 128), (8, 2, 128), (64, 8, 128), (24, 2, 256),
                                              (4, 4, 64), (5, 1, 80), (7, 1, 128)])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "wavelength"])
    factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 40.0])
    rotary_dim = rng.choice([head_dim, head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)])
    page_size = rng.choice([16, 16, 32, 64, 128, 24])
    combined = rng.random() < 0.5
    row = kv_heads * head_dim * 4                  # K and V bytes of one token in one layer
    if op == "rope":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = 1.5e9 / (2 * (q_heads + kv_heads) * head_dim * (4 if dtype == "fp32" else 2))
        return dict(op=op, tokens=_log_int(rng, 1, min(50000, int(most))), q_heads=q_heads,
                    kv_heads=rng.choice([kv_heads, kv_heads, 0]), head_dim=head_dim,
                    rotary_dim=rotary_dim, layout=layout, scaling=scaling, factor=factor,
                    dtype=dtype, inverse=rng.random() < 0.3,
                    max_position=_log_int(rng, 64, 1 << 20))
    if op == "append":
        packed = rng.random() < 0.6
        new_max = _log_int(rng, 1, 4000) if packed else rng.choice([1, 1, 2, 4])
        most = 24000 if packed else 600000
        batch = _log_int(rng, 1, max(1, min(256, most // new_max)))
        prefix_max = _log_int(rng, 1, 4096 if batch <= 64 else 1000)
        return dict(op=op, batch=batch, packed=packed, new_max=new_max, prefix_max=prefix_max,
                    q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, rotary_dim=rotary_dim,
                    layout=layout, scaling=scaling, factor=factor,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), page_size=page_size,
                    combined=combined)
    page = row * page_size
    if op == "copy":
        layers = _log_int(rng, 1, 24)
        pages = _log_int(rng, 1, max(1, min(5000, int(0.6e9 / (layers * page)))))
        return dict(op=op, layers=layers, pool_pages=2 * pages + rng.randint(1, pages), pages=pages,
                    kv_heads=kv_heads, head_dim=head_dim, page_size=page_size, combined=combined)
    if op == "fork":
        layers = _log_int(rng, 1, 16)
        parents = _log_int(rng, 1, 32)
        children = _log_int(rng, 1, max(1, min(200, int(0.3e9 / (layers * page)))))
        most = 1e9 / (layers * row * parents)
        return dict(op=op, layers=layers, parents=parents, children=children,
                    max_len=_log_int(rng, 1, max(2, min(4000, int(most)))),
                    kv_heads=kv_heads, head_dim=head_dim, page_size=page_size, combined=combined)
    if op == "recycle":
        pool_pages = _log_int(rng, 64, 262144)
        rows = _log_int(rng, 1, min(1000, pool_pages // 8))
        recycled = _log_int(rng, 1, rows)
        return dict(op=op, rows=rows, pool_pages=pool_pages, recycled=recycled,
                    max_tokens=max(1, pool_pages * page_size // (2 * rows)), page_size=page_size)
    layers = _log_int(rng, 1, 8)
    pool_pages = _log_int(rng, 8, max(16, min(20000, int(1.5e9 / (layers * page)))))
    return dict(op=op, layers=layers, pool_pages=pool_pages, rows=_log_int(rng, 1, 64),
                live=rng.choice([0.1, 0.3, 0.5, 0.8, 0.95]), kv_heads=kv_heads,
                head_dim=head_dim, page_size=page_size, combined=combined)


# ---- inputs ---------------------------------------------------------------------------------

BASE = 10000.0
ORIGINAL = 8192.0            # positions that the unscaled frequencies were made for


def _frequencies(rotary_dim, scaling, factor):
    """(angle per position of each column pair [rotary_dim / 2], magnitude), in 64 bits."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    base = BASE
    if scaling == "ntk" and rotary_dim > 2:
        base = BASE * factor ** (rotary_dim / (rotary_dim - 2.0))
    f = base ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        lo, hi = (rotary_dim * math.log(ORIGINAL / (2 * math.pi * beta)) / (2 * math.log(BASE))
                  for beta in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rotary_dim - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    if scaling == "wavelength":
        low, high = 1.0, 4.0
        turns = ORIGINAL * f / (2 * math.pi)       # turns over the original context
        t = ((turns - low) / (high - low)).clamp(0, 1)
        f = (1 - t) * f / factor + t * f
    return f, 1.0


def _rope_of(case):
    f, m = _frequencies(case["rotary_dim"], case["scaling"], case["factor"])
    return dict(frequencies=f.to(DEVICE), magnitude=m)


def _pools(case, P, gen):
    """The layers' caches: [N, P, 2, Hkv, ps, D], or K and V pools [N, P, Hkv, ps, D]."""
    shape = (case["kv_heads"], case["page_size"], case["head_dim"])
    n = case.get("layers", 1)
    if case["combined"]:
        return dict(kv=torch.randn((n, P, 2) + shape, generator=gen, device=DEVICE,
                                   dtype=torch.bfloat16))
    return {name: torch.randn((n, P) + shape, generator=gen, device=DEVICE, dtype=torch.bfloat16)
            for name in ("k_pool", "v_pool")}


def _own_pages(lens, page_size, P, C, rng):
    """Rows of distinct pages drawn from one permutation; unused entries are -1."""
    need = -(-lens // page_size)
    assert need.sum() <= P and need.max(initial=0) <= C
    perm = rng.permutation(P)
    tables = np.full((len(lens), C), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        tables[r, :n] = perm[at:at + n]
        at += n
    refs = np.zeros(P, np.int32)
    refs[perm[:at]] = 1
    return tables, refs


def _spread(lo, hi, n):
    """n whole numbers from hi down to lo: the same ones for every seed, so shapes are too."""
    return np.linspace(hi, lo, n).astype(np.int64)


def _new_tokens(case):
    lo = max(1, case["new_max"] // 16) if case["packed"] else case["new_max"]
    return _spread(lo, case["new_max"], case["batch"])


def _parent_lens(case):
    return _spread(max(1, case["max_len"] // 4), case["max_len"], case["parents"])


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    op = case["op"]
    s = dict(case=case)

    def normal(*shape, dtype):
        return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)

    if op == "rope":
        dt = DTYPES[case["dtype"]]
        T = case["tokens"]
        s["q"] = normal(T, case["q_heads"], case["head_dim"], dtype=dt)
        s["k"] = normal(T, case["kv_heads"], case["head_dim"], dtype=dt) if case["kv_heads"] else None
        s["positions"] = _dev(rng.randint(0, case["max_position"], T).astype(np.int32))
        return {**s, **_rope_of(case)}

    ps = case["page_size"]
    if op == "append":
        B, Hq, Hkv, D = (case[k] for k in ("batch", "q_heads", "kv_heads", "head_dim"))
        new = rng.permutation(_new_tokens(case))
        lens = new + rng.permutation(_spread(0, case["prefix_max"], B))
        C = -(-(case["new_max"] + case["prefix_max"]) // ps)
        P = int((lens.sum() // ps + B) * 1.1) + 1
        tables, _ = _own_pages(lens, ps, P, C, rng)
        total = int(new.sum())
        # one fused projection: q, k and v are slices of its rows
        qkv = normal(total, Hq + 2 * Hkv, D, dtype=DTYPES[case["dtype"]])
        if not case["packed"] and case["new_max"] > 1:
            qkv = qkv.view(B, case["new_max"], Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv.split([Hq, Hkv, Hkv], dim=-2)
        s["qo_indptr"] = _dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
        s["lens"] = _dev(lens.astype(np.int32))
        s["tables"] = _dev(tables)
        # the same rows as a CSR table (row b starts at b * C), as decode attention takes it
        s["kv_indptr"] = _dev((np.arange(B + 1) * C).astype(np.int32))
        return {**s, **_rope_of(case), **_pools(case, P, gen)}

    if op == "copy":
        ids = rng.permutation(case["pool_pages"])[:2 * case["pages"]].astype(np.int32)
        s["src"], s["dst"] = _dev(ids[::2]), _dev(ids[1::2])
        return {**s, **_pools(case, case["pool_pages"], gen)}

    if op == "fork":
        np_, nc = case["parents"], case["children"]
        # the children's rows still hold what the last samples left: a page or two each
        lens = np.concatenate([rng.permutation(_parent_lens(case)) - rng.randint(0, 2, np_),
                               rng.randint(1, min(case["max_len"], 2 * ps) + 1, nc)])
        lens = np.maximum(lens, 1)
        C = -(-case["max_len"] // ps) + 1
        P = int(_parent_lens(case).sum()) // ps + np_ + 3 * nc + 1
        tables, refs = _own_pages(lens, ps, P, C, rng)
        s["parents"] = _dev(rng.randint(0, np_, nc).astype(np.int32))
        s["children"] = _dev((np_ + rng.permutation(nc)).astype(np.int32))
        s["tables"], s["lens"], s["refs"] = _dev(tables), _dev(lens.astype(np.int32)), _dev(refs)
        return {**s, **_pools(case, P, gen)}

    if op == "recycle":
        R, P, most = case["rows"], case["pool_pages"], case["max_tokens"]
        most = max(1, min(most, (P // R) * ps))
        lens = rng.randint(1, most + 1, R)
        new = rng.randint(1, most + 1, case["recycled"])
        C = -(-most // ps)
        tables, refs = _own_pages(lens, ps, P, C, rng)
        s["rows"] = _dev(rng.permutation(R)[:case["recycled"]].astype(np.int32))
        s["new"] = _dev(new.astype(np.int32))
        s["tables"], s["lens"], s["refs"] = _dev(tables), _dev(lens.astype(np.int32)), _dev(refs)
        return s

    # compact: rows of random lengths; every second row shares its predecessor's first pages
    R, P = case["rows"], case["pool_pages"]
    need = _spread(0, 2 * P * case["live"] / R, R) if R > 1 else np.array([int(P * case["live"])])
    need = rng.permutation(need)
    lens = np.maximum(need * ps - rng.randint(0, ps, R), 0) * (need > 0)
    C = int(need.max(initial=0)) * 2 + 1
    tables, refs = _own_pages(lens, ps, P, C, rng)
    for r in range(1, R, 2):
        full = int(lens[r - 1] // ps)
        n = min(full, int(rng.randint(0, full + 1)))
        old = -(-int(lens[r]) // ps)
        if n and old + n <= C:
            tables[r, n:n + old] = tables[r, :old].copy()
            tables[r, :n] = tables[r - 1, :n]
            refs[tables[r - 1, :n]] += 1
            lens[r] += n * ps
    s["tables"], s["lens"], s["refs"] = _dev(tables), _dev(lens.astype(np.int32)), _dev(refs)
    return {**s, **_pools(case, P, gen)}


# ---- the plain forms ------------------------------------------------------------------------

def _cos_sin(s, positions, inverse=False):
    angle = positions.double()[:, None] * s["frequencies"]
    cos, sin = (torch.cos(angle) * s["magnitude"]).float(), (torch.sin(angle) * s["magnitude"]).float()
    return cos[:, None], (-sin if inverse else sin)[:, None]


def _rotate(x, cos, sin, layout):
    """x [T, H, D] rotated in 32 bits; the columns past the rotated ones as they are."""
    x = x.float()
    n = cos.shape[-1]
    if layout == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([y, x[..., 2 * n:]], dim=-1)


def _plain_rope(s):
    case = s["case"]
    cos, sin = _cos_sin(s, s["positions"], case["inverse"])
    q = _rotate(s["q"], cos, sin, case["layout"]).to(s["q"].dtype)
    if s["k"] is None:
        return q
    return q, _rotate(s["k"], cos, sin, case["layout"]).to(s["k"].dtype)


def _plain_append(s):
    case = s["case"]
    ps, D = case["page_size"], case["head_dim"]
    start = s["qo_indptr"]
    q, k, v = (s[n].reshape(-1, s[n].shape[-2], D) for n in ("q", "k", "v"))
    t = torch.arange(q.shape[0], device=DEVICE)
    b = torch.searchsorted(start, t, right=True) - 1
    position = s["lens"][b] - (start[b + 1] - t)
    page = s["tables"][b, position // ps].long()
    slot = position % ps
    cos, sin = _cos_sin(s, position)
    k = _rotate(k, cos, sin, case["layout"]).to(torch.bfloat16)
    v = v.to(torch.bfloat16)
    if case["combined"]:
        s["kv"][0][page, 0, :, slot] = k
        s["kv"][0][page, 1, :, slot] = v
    else:
        s["k_pool"][0][page, :, slot] = k
        s["v_pool"][0][page, :, slot] = v
    q = _rotate(q, cos, sin, case["layout"]).to(torch.bfloat16)
    return (q.reshape(s["q"].shape),) + _caches(s)


def _caches(s):
    return (s["kv"],) if "kv" in s else (s["k_pool"], s["v_pool"])


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    if "kv" in s:
        s["kv"][:, dst] = s["kv"][:, src]
    else:
        s["k_pool"][:, dst] = s["k_pool"][:, src]
        s["v_pool"][:, dst] = s["v_pool"][:, src]
    return _caches(s)


def _slots(s):
    return torch.arange(s["tables"].shape[1], device=DEVICE)


def _plain_free(s, rows):
    ps = s["case"]["page_size"]
    live = _slots(s) < ((s["lens"][rows] + ps - 1) // ps)[:, None]
    pages = s["tables"][rows].clamp(min=0).long()
    s["refs"].index_add_(0, pages.flatten(), -live.flatten().int())
    s["lens"][rows] = 0


def _plain_fork(s):
    ps = s["case"]["page_size"]
    parents, children = s["parents"].long(), s["children"].long()
    _plain_free(s, children)
    lens = s["lens"][parents]
    full, tail = lens // ps, lens % ps
    need = tail > 0
    free = torch.nonzero(s["refs"] == 0).flatten()
    fresh = free[(torch.cumsum(need, 0) - need.long()).clamp(max=free.numel() - 1)]
    slots = _slots(s)
    shared = slots < full[:, None]
    theirs = s["tables"][parents]
    mine = torch.where(shared, theirs, s["tables"][children])
    mine = torch.where((slots == full[:, None]) & need[:, None], fresh[:, None].int(), mine)
    s["tables"][children] = mine
    s["refs"].index_add_(0, theirs.clamp(min=0).flatten().long(), shared.flatten().int())
    s["refs"].index_add_(0, fresh, need.int())
    s["lens"][children] = lens
    last = theirs.gather(1, full.clamp(max=theirs.shape[1] - 1).long()[:, None]).flatten()
    src, dst, tail = last[need].long(), fresh[need], tail[need]
    token = (torch.arange(ps, device=DEVICE) < tail[:, None])[:, None, :, None]
    if "kv" in s:
        s["kv"][:, dst] = torch.where(token[:, None], s["kv"][:, src], s["kv"][:, dst])
    else:
        s["k_pool"][:, dst] = torch.where(token, s["k_pool"][:, src], s["k_pool"][:, dst])
        s["v_pool"][:, dst] = torch.where(token, s["v_pool"][:, src], s["v_pool"][:, dst])
    return (s["tables"], s["lens"], s["refs"]) + _caches(s)


def _plain_recycle(s):
    ps = s["case"]["page_size"]
    rows = s["rows"].long()
    _plain_free(s, rows)
    lens = s["lens"][rows]
    have, want = (lens + ps - 1) // ps, (lens + s["new"] + ps - 1) // ps
    free = torch.nonzero(s["refs"] == 0).flatten()
    first = torch.cumsum(want - have, 0) - (want - have)
    slots = _slots(s)
    fresh = (slots >= have[:, None]) & (slots < want[:, None])
    rank = (first[:, None] + slots - have[:, None]).clamp(0, free.numel() - 1)
    pages = free[rank]
    s["tables"][rows] = torch.where(fresh, pages.int(), s["tables"][rows])
    s["refs"].index_add_(0, pages.flatten(), fresh.flatten().int())
    s["lens"][rows] = lens + s["new"]
    return s["tables"], s["lens"], s["refs"]


def _plain_compact(s):
    ps = s["case"]["page_size"]
    refs = s["refs"]
    live = refs > 0
    n = live.sum()
    ids = torch.arange(refs.numel(), device=DEVICE)
    src = torch.nonzero(live & (ids >= n)).flatten()
    dst = torch.nonzero(~live & (ids < n)).flatten()
    if "kv" in s:
        s["kv"][:, dst] = s["kv"][:, src]
    else:
        s["k_pool"][:, dst] = s["k_pool"][:, src]
        s["v_pool"][:, dst] = s["v_pool"][:, src]
    to = ids.clone()
    to[src] = dst
    used = _slots(s) < ((s["lens"] + ps - 1) // ps)[:, None]
    tables = torch.where(used, to[s["tables"].clamp(min=0).long()].int(), s["tables"])
    after = refs.clone()
    after[dst] = refs[src]
    after[src] = 0
    return (tables, after, n.to(torch.int32).reshape(1)) + _caches(s)


# ---- the library's calls --------------------------------------------------------------------

def _own_table(s, pkb):
    """The rotary table and the pools' handle are made once, as a program makes them at start."""
    if "table" not in s:
        case = s["case"]
        s["table"], s["factor"] = pkb.rope_frequencies(
            case["rotary_dim"], base=BASE, scaling=case["scaling"], factor=case["factor"],
            original_max_position=ORIGINAL, device=DEVICE)
    return s["table"], s["factor"]


def _own_pools(s, pkb):
    if "pools" not in s:
        s["pools"] = pkb.cache_pools(list(s["kv"]) if "kv" in s
                                     else list(zip(s["k_pool"], s["v_pool"])))
    return s["pools"]


def _own_workspace(s, size, *args):
    if "workspace" not in s:
        s["workspace"] = torch.empty(size(*args), dtype=torch.uint8, device=DEVICE)
    return s["workspace"]


def _own_rope(s):
    import paged_kv_block_gb300 as pkb
    case = s["case"]
    table, factor = _own_table(s, pkb)
    return pkb.rotary_embedding(s["q"], s["positions"], table, k=s["k"], layout=case["layout"],
                                attention_factor=factor, inverse=case["inverse"])


def _own_append(s):
    import paged_kv_block_gb300 as pkb
    case = s["case"]
    table, factor = _own_table(s, pkb)
    cache = s["kv"][0] if "kv" in s else (s["k_pool"][0], s["v_pool"][0])
    pages = (dict(paged_kv_indptr=s["kv_indptr"], paged_kv_indices=s["tables"].view(-1))
             if case["combined"] else dict(block_tables=s["tables"]))
    q = pkb.append_paged_kv_cache(s["k"], s["v"], cache, s["lens"], q=s["q"], freqs=table,
                                  qo_indptr=s["qo_indptr"] if case["packed"] else None,
                                  layout=case["layout"], attention_factor=factor, **pages)
    return (q,) + _caches(s)


def _own_copy(s):
    import paged_kv_block_gb300 as pkb
    pkb.copy_cache_pages(_own_pools(s, pkb), s["src"], s["dst"])
    return _caches(s)


def _own_fork(s):
    import paged_kv_block_gb300 as pkb
    pools = _own_pools(s, pkb)
    n = s["children"].numel()
    ws = _own_workspace(s, pkb.fork_cache_workspace_size, n)
    ps = s["case"]["page_size"]
    pkb.free_cache_rows(s["children"], s["tables"], s["lens"], s["refs"], ps)
    pkb.fork_cache_rows(pools, s["parents"], s["children"], s["tables"], s["lens"], s["refs"],
                        workspace=ws)
    return (s["tables"], s["lens"], s["refs"]) + _caches(s)


def _own_recycle(s):
    import paged_kv_block_gb300 as pkb
    ps = s["case"]["page_size"]
    ws = _own_workspace(s, pkb.extend_cache_workspace_size, s["rows"].numel())
    pkb.free_cache_rows(s["rows"], s["tables"], s["lens"], s["refs"], ps)
    pkb.extend_cache_rows(s["rows"], s["new"], s["tables"], s["lens"], s["refs"], ps,
                          workspace=ws)
    return s["tables"], s["lens"], s["refs"]


def _own_compact(s):
    import paged_kv_block_gb300 as pkb
    pools = _own_pools(s, pkb)
    ws = _own_workspace(s, pkb.compact_cache_workspace_size, s["refs"].numel())
    tables, refs, live = pkb.compact_cache(
        pools, s["tables"], s["lens"], s["refs"], block_tables_out=torch.empty_like(s["tables"]),
        page_refs_out=torch.empty_like(s["refs"]), workspace=ws)
    return (tables, refs, live) + _caches(s)


_PLAIN = dict(rope=_plain_rope, append=_plain_append, copy=_plain_copy, fork=_plain_fork,
              recycle=_plain_recycle, compact=_plain_compact)
_OWN = dict(rope=_own_rope, append=_own_append, copy=_own_copy, fork=_own_fork,
            recycle=_own_recycle, compact=_own_compact)


def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rope":
        rows = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        e = 4 if case["dtype"] == "fp32" else 2
        return dict(bytes=2 * rows * case["head_dim"] * e + 4 * case["tokens"],
                    flops=3 * rows * case["rotary_dim"])
    if op == "recycle":
        # half of the longest, on average: the rows' entries, their old and new pages' counts
        pages = case["recycled"] * case["max_tokens"] / (2 * case["page_size"])
        return dict(bytes=4 * case["pool_pages"] + 4 * pages * 4, flops=0)
    row = case["kv_heads"] * case["head_dim"] * 4
    if op == "append":
        T = int(_new_tokens(case).sum())
        e = 4 if case["dtype"] == "fp32" else 2
        heads = case["q_heads"] + 2 * case["kv_heads"]
        return dict(bytes=T * heads * case["head_dim"] * (e + 2),
                    flops=3 * T * (case["q_heads"] + case["kv_heads"]) * case["rotary_dim"])
    if op == "copy":
        return dict(bytes=2 * case["pages"] * case["layers"] * row * case["page_size"], flops=0)
    if op == "fork":
        tail = case["children"] * case["page_size"] / 2
        entries = case["children"] * _parent_lens(case).mean() / case["page_size"]
        return dict(bytes=2 * tail * case["layers"] * row + 4 * entries * 4, flops=0)
    pages = case["pool_pages"]
    moved = pages * case["live"] * (1 - case["live"])
    return dict(bytes=2 * moved * case["layers"] * row * case["page_size"] + 4 * 2 * pages, flops=0)


# ---- the definition in 64 bits --------------------------------------------------------------

def _exact_turned(x, positions, case):
    """Rows x [T, H, D] rotated: every column pair is a complex number times m e^(i p f)."""
    f, m = _frequencies(case["rotary_dim"], case["scaling"], case["factor"])
    n = case["rotary_dim"] // 2
    y = x.double().clone()
    sign = -1.0 if case.get("inverse") else 1.0
    turn = torch.polar(torch.full((positions.numel(), n), m, dtype=torch.float64, device=x.device),
                       sign * positions.double()[:, None] * f.to(x.device)[None])
    if case["layout"] == "half":
        first, second = slice(0, n), slice(n, 2 * n)
    else:
        first, second = slice(0, 2 * n, 2), slice(1, 2 * n, 2)
    for h in range(x.shape[1]):
        z = torch.complex(x[:, h, first].double(), x[:, h, second].double()) * turn
        y[:, h, first], y[:, h, second] = z.real, z.imag
    return y


def exact(case, seed):
    if case["op"] not in ("rope", "append"):
        return None                                # copies and page tables: exact by themselves
    s = prepare(case, seed)
    if case["op"] == "rope":
        q = _exact_turned(s["q"], s["positions"], case)
        return q if s["k"] is None else (q, _exact_turned(s["k"], s["positions"], case))
    ps = case["page_size"]
    starts, lens, tables = (s[n].tolist() for n in ("qo_indptr", "lens", "tables"))
    page, slot, position = [], [], []
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        for p in range(L - n, L):
            position.append(p)
            page.append(tables[b][p // ps])
            slot.append(p % ps)
    page, slot, position = (torch.tensor(v, device=DEVICE) for v in (page, slot, position))
    q, k, v = (s[n].reshape(-1, s[n].shape[-2], s[n].shape[-1]) for n in ("q", "k", "v"))
    new = (_exact_turned(k, position, case), v.double())
    out = [_exact_turned(q, position, case).reshape(s["q"].shape)]
    if case["combined"]:
        kv = s["kv"].double()
        for j in range(2):
            kv[0, page, j, :, slot] = new[j]
        return out + [kv]
    for pool, rows in zip((s["k_pool"], s["v_pool"]), new):
        pool = pool.double()
        pool[0, page, :, slot] = rows
        out.append(pool)
    return out
