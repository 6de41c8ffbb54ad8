"""The README's serving step, run as it stands there: every layer's attention against float64."""
import os
import re

import numpy as np
import pytest
import torch

from oracle import cache as O
from tests.gpu_util import OUT_MAX_ABS, OUT_MEAN_ABS
from tests.test_gpu_cache_chain import D, HKV, HQ, attention, i32

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def step():
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, flags=re.S)
    return next(b for b in blocks if "append_paged_kv_cache" in b)


class Layer:
    def __init__(self, gen, total):
        self.qkv = torch.randn(total, HQ + 2 * HKV, D, generator=gen).to(torch.bfloat16).cuda()
        self.kept = None

    def project(self, x):
        return self.qkv.split([HQ, HKV, HKV], dim=1)

    def finish(self, x, out):
        self.kept = out.double().cpu().numpy()
        return x + 1


def scene(pages):
    """Rows 0 and 1 hold 40 and 16 tokens, row 2 is done, row 3 becomes a fork of row 0."""
    gen = torch.Generator().manual_seed(2)
    lens, tables = [40, 16, 20, 0], [[0, 1, 2, -1, -1], [3, -1, -1, -1, -1], [4, 5, -1, -1, -1],
                                     [-1] * 5]
    new = [3, 30, 12, 1]

    def pool():
        return torch.randn(pages, HKV, 16, D, generator=gen).to(torch.bfloat16).cuda()
    names = dict(x=0, layers=[Layer(gen, sum(new)) for _ in range(2)],
                 caches=[tuple(pool() for _ in range(2)) for _ in range(2)],
                 done=i32([2]), parents=i32([0]), children=i32([3]), rows=i32([0, 1, 2, 3]),
                 new_tokens=i32(new), tables=i32(tables), lens=i32(lens),
                 refs=i32([1] * 6 + [0] * (pages - 6)), qo_indptr=i32([0, 3, 33, 45, 46]))
    return names, new


def test_the_serving_step():
    names, new = scene(12)
    old = [[[c[p].double().cpu().numpy() for p in (0, 1, 2)] + [c[3].double().cpu().numpy()]
            for c in cache] for cache in names["caches"]]
    exec(step(), names)
    assert names["x"] == 2 and names["lens"].tolist() == [43, 46, 12, 41]
    f, m = O.frequencies(D, scaling="yarn", factor=4.0, original=8192.0)

    def bf(a):
        return torch.from_numpy(a).to(torch.bfloat16).double().numpy()
    for layer, (K, V) in zip(names["layers"], old):
        def rows_of(pages, n):                       # [tokens, Hkv, D] of whole pages
            return np.concatenate([p.transpose(1, 0, 2) for p in pages])[:n]
        held = [(rows_of(c[:3], 40), rows_of(c[3:], 16), np.zeros((0, HKV, D)), rows_of(c[:3], 40))
                for c in (K, V)]
        q, k, v = (t.double().cpu().numpy() for t in layer.project(0))
        at = 0
        for r, n in enumerate(new):
            first, part = held[0][r].shape[0], slice(at, at + n)
            pos = list(range(first, first + n))
            qq, kk = (bf(O.rotate(t[part], pos, f, m=m)[0]) for t in (q, k))
            want = attention(qq, np.concatenate([held[0][r], kk]),
                             np.concatenate([held[1][r], v[part]]), first)
            off = np.abs(layer.kept[part] - want)
            assert off.max() <= OUT_MAX_ABS and off.mean() <= OUT_MEAN_ABS, (r, off.max())
            at += n


def test_the_serving_step_stops_without_pages():
    names, _ = scene(7)
    with pytest.raises(RuntimeError, match="without pages"):
        exec(step(), names)
    assert names["x"] == 0                           # nothing was appended
