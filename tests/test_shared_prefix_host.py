"""CPU checks of decode with shared prefixes: what the C entry point and the binding refuse."""
import ctypes as C

import pytest
import torch

import paged_kv_block_gb300 as pkb
from paged_kv_block_gb300 import build as B
from paged_kv_block_gb300 import cache as K

A16 = 0x7F0000100000
BAD = pkb.ERR_INVALID_ARGUMENT
BASE = dict(batch=4, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=100,
            combined_cache=1, max_seq_len=512, mask_type=1, window_left=-1, bmm1_scale=0.0,
            bmm2_scale=1.0)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pkb.lib()


def test_workspace(lib):
    size = lambda groups, **kw: pkb.paged_decode_shared_workspace_size(  # noqa: E731
        pkb.DecodeParams(**{**BASE, **kw}), groups)
    assert 0 < size(0) < size(1) < size(2) == size(3) == size(10 ** 9)
    assert size(1, seq_len_q=4) > size(1)
    for kw in (dict(head_dim=64), dict(head_dim=256), dict(num_qo_heads=7), dict(page_size=12),
               dict(num_qo_heads=34), dict(window_left=5), dict(split_chunk=128), dict(batch=-1),
               dict(max_seq_len_q=2, total_q=4), dict(seq_len_q=17), dict(mask_type=2),
               dict(out_dtype=3), dict(max_seq_len=0), dict(batch=1 << 27), dict(num_pages=0)):
        assert size(1, **kw) == 0, kw
    assert size(-1) == 0


def test_c_refusals(lib):
    p = pkb.DecodeParams(**BASE)

    def run(params=p, groups=1, size=1 << 40, **kw):
        a = dict(q=A16, k=A16, v=None, indptr=A16, indices=A16, lens=A16, first=A16, prefix=A16,
                 out=A16, lse=None, ws=A16)
        a.update(kw)
        return lib.paged_decode_shared_run(C.byref(params), groups, *a.values(), size, None)
    for kw in (dict(groups=-1), dict(params=pkb.DecodeParams(**{**BASE, "window_left": 3})),
               dict(params=pkb.DecodeParams(**{**BASE, "combined_cache": 0})),
               *[{k: None} for k in ("q", "k", "indptr", "indices", "lens", "first", "prefix",
                                     "out")],
               *[{k: A16 + 8} for k in ("q", "k", "v", "out", "ws")],
               *[{k: A16 + 2} for k in ("indptr", "indices", "lens", "first", "prefix", "lse")]):
        assert run(**kw) == BAD, kw
    need = pkb.paged_decode_shared_workspace_size(p, 1)
    assert run(size=need - 1) == run(ws=None) == pkb.ERR_WORKSPACE


def test_binding_refusals(lib, monkeypatch):
    monkeypatch.setattr(K, "_device", lambda: -1)
    monkeypatch.setattr(K, "_stream", lambda stream, dev: 0)
    seen = []

    class Recorder:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 64
            return lambda *a: seen.append(a) or 0
    monkeypatch.setattr(K, "_call", Recorder())
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    bf16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    good = dict(query=bf16(4, 8, 128), kv_cache=bf16(9, 2, 2, 16, 128), workspace_buffer=None,
                paged_kv_indptr=i32(5), paged_kv_indices=i32(20), seq_lens=i32(4), max_seq_len=99,
                group_indptr=i32(3), prefix_lens=i32(2))
    out, lse = pkb.batch_decode_with_shared_prefix(**good)
    assert out.shape == (4, 8, 128) and lse is None and len(seen) == 1
    params = seen[0][0]._obj
    assert (params.batch, params.seq_len_q, params.window_left, params.split_chunk) == (4, 1, -1, 0)
    for bad in (dict(query=bf16(4, 8, 64)), dict(query=torch.zeros(4, 8, 128)),
                dict(kv_cache=bf16(9, 3, 2, 16, 128)), dict(kv_cache=torch.zeros(9, 2, 2, 16, 128)),
                dict(paged_kv_indptr=i32(4)), dict(seq_lens=i32(5)), dict(group_indptr=i32(2)),
                dict(prefix_lens=i32(3)), dict(prefix_lens=torch.zeros(2)), dict(kv_layout="NHD"),
                dict(seq_len_q=2), dict(out=bf16(4, 8, 64)), dict(out_dtype=torch.float64),
                dict(out=bf16(4, 8, 128), out_dtype=torch.float32), dict(lse=torch.zeros(4, 4)),
                dict(lse=torch.zeros(4, 8).double()), dict(mask_type="window"),
                dict(seq_lens=torch.zeros(4, dtype=torch.int64)), dict(group_indptr=i32(6)[::2]),
                dict(query=bf16(4, 128, 8).transpose(1, 2)),
                dict(out=bf16(4, 128, 8).transpose(1, 2)),
                dict(workspace_buffer=torch.zeros(99, 2)[:, 0])):
        with pytest.raises((ValueError, KeyError)):
            pkb.batch_decode_with_shared_prefix(**{**good, **bad})
    assert len(seen) == 1
    lse, out = torch.zeros(4, 8), bf16(4, 8, 128)
    versions = lse._version, out._version
    pkb.batch_decode_with_shared_prefix(**good, out=out, lse=lse)
    assert lse._version > versions[0] and out._version > versions[1]
    four = {**good, "query": bf16(4, 3, 8, 128)}
    pkb.batch_decode_with_shared_prefix(**four, seq_len_q=3, mask_type="causal", bmm2_scale=0.5,
                                        out_dtype=torch.float32)
    p = seen[-1][0]._obj
    assert (p.seq_len_q, p.mask_type, p.bmm2_scale, p.out_dtype) == (3, 1, 0.5, 2)
