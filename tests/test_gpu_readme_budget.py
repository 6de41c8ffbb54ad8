"""The README's step within a budget, run as it stands there: outputs against float64, and what is
kept."""
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import cache as OC
from tests.gpu_util import OUT_MAX_ABS, OUT_MEAN_ABS
from tests.test_gpu_cache_chain import D, HKV, HQ, attention, i32
from tests.test_gpu_readme import ROOT, Layer

pytestmark = pytest.mark.gpu


def step():
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, flags=re.S)
    return next(b for b in blocks if "evict_cache_rows" in b)


def scene(pages):
    """Rows 0 and 1 share a prompt of 48 tokens and have 10 and 25 more, row 2 has 40."""
    gen = torch.Generator().manual_seed(3)
    before = [58, 73, 40]
    tables = [[0, 1, 2, 3, -1, -1], [0, 1, 2, 4, 5, -1], [6, 7, 8, -1, -1, -1]]

    def pool():
        return torch.randn(pages, HKV, 16, D, generator=gen).to(torch.bfloat16).cuda()
    caches = [tuple(pool() for _ in range(2)) for _ in range(2)]
    names = dict(x=0, layers=[Layer(gen, 3) for _ in range(2)], caches=caches,
                 pools=pkb.cache_pools(caches), tables=i32(tables),
                 lens=i32([n + 1 for n in before]),
                 refs=i32([2, 2, 2] + [1] * 6 + [0] * (pages - 9)), positions=i32([90, 91, 40]),
                 freqs=pkb.rope_frequencies(D)[0], kv_indptr=i32([0, 6, 12, 18]), max_len=96,
                 group_indptr=i32([0, 2, 3]), prefix_lens=i32([48, 0]), full=i32([1, 0]), budget=40,
                 weights=torch.rand(2, 3, HKV, 96, generator=gen).cuda(), status=i32([0]))
    return names, before, tables


def test_the_step_within_a_budget():
    names, before, tables = scene(14)
    old = [[c.double().cpu().numpy() for c in cache] for cache in names["caches"]]
    exec(step(), names)
    assert names["x"] == 2 and names["lens"].tolist() == [40, 40, 41]
    f = OC.frequencies(D)[0]
    for layer, cache in zip(names["layers"], old):
        q, k, v = layer.qkv.split([HQ, HKV, HKV], dim=1)
        for r, n in enumerate(before):
            rows = [np.stack([pool[tables[r][j // 16], :, j % 16] for j in range(n)])
                    for pool in cache]
            turned = [OC.rotate(t[r:r + 1], names["positions"].tolist()[r:r + 1], f)[0]
                      for t in (q, k)]
            bf = [torch.from_numpy(t).to(torch.bfloat16).double().numpy() for t in turned]
            want = attention(bf[0], np.concatenate([rows[0], bf[1]]),
                             np.concatenate([rows[1], v[r:r + 1].double().cpu().numpy()]), n)
            off = np.abs(layer.kept[r:r + 1] - want)
            assert off.max() <= OUT_MAX_ABS and off.mean() <= OUT_MEAN_ABS
    # the shared page of the sink stays, the next ones are copied for both rows
    assert names["tables"][:2, 0].tolist() == [0, 0] and names["refs"][0].item() == 2
    assert names["refs"].sum().item() == 3 + 3 + 3
    kept = names["kept"]
    assert (kept[..., :16].cpu() == torch.arange(16)).all()


def test_too_few_pages_are_noticed():
    names, *_ = scene(9)                             # none is free
    with pytest.raises(RuntimeError, match="keep all of their tokens"):
        exec(step(), names)
    assert names["lens"].tolist() == [59, 74, 41]
