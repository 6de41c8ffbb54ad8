"""Appended rows in every layout that the launch treats differently: slices of one projection,
tensors of their own, and mixtures.  Each starts from the same cache and has to leave the same bits
in all of it."""
import pytest
import torch

import paged_kv_block_gb300 as pkb
from tests.test_gpu_append import DEV, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("combined", [True, False])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,D,R", [(32, 8, 128, 128), (0, 1, 80, 40), (4, 2, 256, 64),
                                        (3, 3, 64, 20), (7, 1, 8, 0)])
@pytest.mark.parametrize("new", [[1300, 1, 0, 1250], [3, 1, 0, 2]])
def test_row_layouts_write_the_same_cache(new, combined, layout, dtype, Hq, Hkv, D, R):
    s = problem(D, new, [70, 3, 40, 0], Hq=max(Hq, 1), Hkv=Hkv, D=D, dtype=dtype, combined=combined)
    table = pkb.rope_frequencies(R)[0] if R else None
    k, v, q = s["k"], s["v"], s["q"] if Hq else None
    before = s["cache"].clone()

    def run(kk, vv, qq):
        cache = before.clone()
        out = pkb.append_paged_kv_cache(kk, vv, cache if combined else (cache[0], cache[1]),
                                        s["lens"], q=qq, qo_indptr=s["qo"], freqs=table,
                                        layout=layout, block_tables=s["tables"])
        return out, cache.view(torch.int16)
    out, cache = run(k, v, q)
    # every slot of a new token is written: none still holds all of its old row
    tokens = sum(new)
    rows = (cache != before.view(torch.int16)).any(-1)       # [.., Hkv, ps]
    assert rows.sum() == 2 * Hkv * tokens

    def wide(x):                                             # rows of their own, farther apart
        return torch.cat([x, x], dim=1)[:, :x.shape[1]]
    qc = None if q is None else q.contiguous()
    qw = None if q is None else wide(q)
    for kk, vv, qq in ((k.contiguous(), v.contiguous(), qc), (k.contiguous(), v, q),
                       (k, v.contiguous(), qc), (k, wide(v), q), (wide(k), v.contiguous(), qw)):
        o, c = run(kk, vv, qq)
        assert torch.equal(c, cache)
        assert out is None or torch.equal(o, out)
    # element-wise access: rows that start on an odd element
    odd = torch.zeros(tokens, Hkv * D + 1, dtype=dtype, device=DEV)[:, 1:].unflatten(1, (Hkv, D))
    odd.copy_(k)
    o, c = run(odd, v, q)
    assert torch.equal(c, cache) and (out is None or torch.equal(o, out))


@pytest.mark.parametrize("columns", [0, 3])
def test_a_batch_of_no_request_writes_nothing(columns):
    """All rows of the packed tensors are padding."""
    s = problem(9, [4, 5], [0, 2], Hq=2, Hkv=1, D=16)
    table, _ = pkb.rope_frequencies(16)
    before = s["cache"].clone()
    mark = torch.full(s["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV)
    q_out, word = mark.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    for pages in (dict(block_tables=none.new_zeros(0, columns)),
                  dict(paged_kv_indptr=none.new_zeros(1), paged_kv_indices=none)):
        pkb.append_paged_kv_cache(s["k"], s["v"], (s["cache"][0], s["cache"][1]), none, q=s["q"],
                                  q_out=q_out, qo_indptr=none.new_zeros(1), freqs=table,
                                  status=word, **pages)
        assert torch.equal(q_out, mark) and torch.equal(s["cache"], before) and word.item() == 0
