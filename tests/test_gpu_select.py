"""Selecting the tokens to keep on the GPU: every list equals the oracle's sort."""
import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import eviction as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(seed, shape, kind):
    rng = np.random.RandomState(seed)
    w = rng.rand(*shape).astype(np.float32)
    if kind == "ties":                       # a handful of values
        w = np.floor(w * 4).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "zeros":                    # both zeros are equal
        w = np.where(w < 0.5, np.float32(-0.0), np.float32(0.0))
    elif kind == "signed":
        w = (w - 0.5) * np.float32(1e30)
    elif kind == "close":                    # differ in their last bits alone
        w = (np.float32(1.0) + rng.randint(0, 40, shape).astype(np.float32) * np.float32(2 ** -23))
    elif kind == "special":
        pick = rng.randint(0, 8, shape)
        w = np.select([pick == 0, pick == 1, pick == 2, pick == 3],
                      [np.float32(np.nan), np.float32(np.inf), np.float32(-np.inf),
                       np.float32(np.finfo(np.float32).min)], w).astype(np.float32)
    return w


def check(w, lens, rows, keep, sink=0, recent=0):
    """NaN past every length: nothing there may be read."""
    N, R, H, W = w.shape
    dirty = w.copy()
    for r in range(R):
        dirty[:, r, :, max(0, min(W, lens[r])):] = np.nan
    status = i32([0])
    lens_dev = i32(lens)
    got = pkb.select_cache_tokens(i32(rows), torch.from_numpy(dirty).to(DEV), lens_dev, keep,
                                  sink=sink, recent=recent, status=status)
    want, bits = O.select(w, rows, lens, keep, sink, recent)
    assert np.array_equal(got.cpu().numpy(), want)
    assert status.item() == bits


@pytest.mark.parametrize("kind", ["uniform", "ties", "equal", "zeros", "signed", "close",
                                  "special"])
@pytest.mark.parametrize("W,keep,sink,recent", [(1, 1, 0, 0), (33, 7, 0, 0), (300, 64, 4, 16),
                                                (300, 299, 5, 0), (2500, 512, 4, 508),
                                                (5000, 100, 0, 0)])
def test_lists(kind, W, keep, sink, recent):
    w = make(W, (2, 4, 2, W), kind)
    lens = [W, max(0, W - 31), W // 2, min(W, keep + 1)]
    check(w, lens, [2, 0, 3, 1], keep, sink, recent)


@pytest.mark.parametrize("lists", [1, 3, 40])
@pytest.mark.parametrize("W", [4097, 20011, 70001])
def test_clusters_and_long_lists(lists, W):
    w = make(W + lists, (1, 1, lists, W), "ties" if lists == 3 else "uniform")
    check(w, [W - 5], [0], W // 7, 2, 9)


def test_a_list_longer_than_shared_memory():
    """Over 8 CTAs' worth of keys in one list, and 160 lists without clusters."""
    W = 400003
    w = make(3, (1, 1, 1, W), "uniform")
    check(w, [W], [0], 50000, 4, 1000)
    w = make(4, (5, 1, 32, 41000), "ties")
    check(w, [41000], [0], 1000)


def test_rows_that_are_left_out():
    w = make(5, (1, 3, 2, 50), "uniform")
    check(w, [50, 51, -1], [0, 1, 2, 3, -1, 0], 8, 2, 2)


def test_one_layer_and_given_lists():
    w = torch.rand(3, 2, 90, device=DEV)
    lens, rows = i32([90, 40, 80]), i32([2, 1])
    four = pkb.select_cache_tokens(rows, w[None], lens, 41)
    kept = torch.full((2, 2, 41), 7, dtype=torch.int32, device=DEV)
    assert pkb.select_cache_tokens(rows, w, lens, 41, kept=kept) is kept
    assert torch.equal(four[0], kept)
    assert pkb.select_cache_tokens(i32([]), w, lens, 41).shape == (0, 2, 41)


def test_captured_and_on_another_stream():
    """A replayed capture reads the weights and lengths of the moment."""
    w, lens, rows = torch.rand(1, 2, 2, 700, device=DEV), i32([700, 600]), i32([0, 1])
    kept = torch.empty(1, 2, 2, 50, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkb.select_cache_tokens(rows, w, lens, 50, kept=kept)
    for seed in range(3):
        x = make(seed, (1, 2, 2, 700), "ties")
        w.copy_(torch.from_numpy(x))
        lens.copy_(i32([700 - seed, 40 + 10 * seed]))
        graph.replay()
        assert np.array_equal(kept.cpu().numpy(), O.select(x, [0, 1], lens.tolist(), 50)[0])
    other = pkb.select_cache_tokens(rows, w, lens, 50, stream=side)
    side.synchronize()
    assert torch.equal(other, kept)


@pytest.mark.parametrize("kind", ["uniform", "ties", "equal", "zeros", "special"])
@pytest.mark.parametrize("L", [2, 31, 64, 255, 256, 257, 700, 3000])
def test_all_but_one_and_only_one(kind, L):
    """The selection's ends, for short lists and longer ones, beside tokens that are kept anyway."""
    w = make(L, (2, 2, 3, L + 7), kind)
    for keep, sink, recent in ((1, 0, 0), (L - 1, 0, 0), (1, 1, 0), (L // 2, L // 4, L // 4),
                               (L // 2 + 1, 0, L // 2), (L - 1, 1, L - 2 - L // 3)):
        if keep >= 1 and sink >= 0 and recent >= 0 and sink + recent <= keep:
            check(w, [L, max(1, L - 1)], [1, 0], keep, sink, recent)


def test_short_rows_of_wide_lists():
    """Rows of 0 to 257 tokens where the width asks for a cluster."""
    w = make(6, (1, 6, 1, 50000), "ties")
    check(w, [0, 1, 40, 256, 257, 49999], [5, 4, 3, 2, 1, 0], 33, 3, 5)


def test_one_of_many():
    """The greatest, and the least left out, of long lists: far outside every sample."""
    for kind in ("uniform", "signed", "special"):
        w = make(7, (1, 3, 2, 60001), kind)
        check(w, [60001, 59000, 300], [0, 1, 2], 5, 3, 1)
        check(w, [60001, 59000, 300], [0, 1, 2], 58999, 3, 1)
