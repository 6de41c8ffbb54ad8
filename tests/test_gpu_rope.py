"""Rotary positions on the GPU against the float64 oracle.

Tolerance.  An output is one fp32 evaluation of m (x1 c - x2 s), rounded once to the output type.
The angle is off by at most 2^-24 of an eighth of a turn (0.79 rad) plus 2^-32 of a turn, sine
and cosine by 2 ulp (2^-23 of at most 1 each), the factor, the two products and the sum by half
a unit each: together below 8 * 2^-24 of m (|x1| + |x2|).  The final rounding adds half a step of
the type, and half its smallest step near zero."""
import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import cache as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def close(got, want, size, dtype=None):
    dtype = dtype or got.dtype
    got = got.double().cpu().numpy()
    bound = size * 8 * 2.0 ** -24
    bound = bound + HALF_STEP[dtype] * (np.abs(want) + bound) + TINY[dtype]
    off = np.abs(got - want) - bound
    assert (off <= 0).all(), f"{(off > 0).sum()} outside, worst by {off.max()}"


def rows(gen, *shape, dtype):
    return torch.randn(shape, generator=gen).to(dtype).to(DEV)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D,R", [(128, 128), (256, 64), (64, 20), (80, 80), (8, 2), (128, 30),
                                 (512, 512), (24, 24)])
def test_matches_oracle(layout, dtype, D, R):
    gen = torch.Generator().manual_seed(D * 1000 + R)
    T, Hq, Hk = 5, 3, 2
    q, k = rows(gen, T, Hq, D, dtype=dtype), rows(gen, T, Hk, D, dtype=dtype)
    pos = torch.tensor([0, 1, 4095, 1000003, 77], dtype=torch.int32)
    table, m = pkb.rope_frequencies(R)
    f, _ = O.frequencies(R)
    qo, ko = pkb.rotary_embedding(q, pos.to(DEV), table, k=k, layout=layout, attention_factor=m)
    for x, y in ((q, qo), (k, ko)):
        want, size = O.rotate(x, pos.tolist(), f, layout=layout)
        close(y, want, size)
        # columns past the rotated ones are copied bit for bit
        assert torch.equal(y[..., R:], x[..., R:])
    assert qo.dtype == dtype and qo.shape == q.shape


@pytest.mark.parametrize("T", [1, 2, 3, 63, 64, 65, 2435, 9731])
def test_token_counts(T):
    """Every token tile of the launch, the last one partly filled too."""
    gen = torch.Generator().manual_seed(T)
    q = rows(gen, T, 2, 64, dtype=torch.bfloat16)
    pos = torch.randint(0, 5000, (T,), generator=gen, dtype=torch.int32)
    table, _ = pkb.rope_frequencies(64)
    out = pkb.rotary_embedding(q, pos.to(DEV), table)
    a = pos.double()[:, None] * torch.from_numpy(O.frequencies(64)[0])
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    x = q.double().cpu()
    x1, x2 = x[..., :32], x[..., 32:]
    want = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1).numpy()
    size = (x1.abs() + x2.abs()).repeat(1, 1, 2).numpy()
    close(out, want, size)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("Hq,Hk,D,R", [(32, 8, 128, 128), (5, 0, 80, 80), (3, 2, 64, 32), (24, 2, 256, 64),
                                       (1, 1, 8, 8), (2, 1, 64, 20), (70, 9, 512, 512)])
def test_long_calls_equal_short_ones(layout, dtype, Hq, Hk, D, R):
    """The launch of a long call (several tokens per CTA, rows staged in shared memory) gives the
    bits of short calls on its parts; in place too."""
    gen = torch.Generator(device=DEV).manual_seed(D + R)
    T = 2600 if D < 512 else 2433
    fused = torch.randn(T, Hq + Hk, D, generator=gen, device=DEV).to(dtype)
    q, k = fused[:, :Hq], fused[:, Hq:] if Hk else None
    pos = torch.randint(-9, 1 << 20, (T,), generator=gen, device=DEV, dtype=torch.int32)
    table, _ = pkb.rope_frequencies(R)

    def both(x):
        return x if isinstance(x, tuple) else (x, x[:, :0])
    got = both(pkb.rotary_embedding(q, pos, table, k=k, layout=layout))
    for a in range(0, T, 500):
        part = slice(a, min(T, a + 500))
        want = both(pkb.rotary_embedding(q[part], pos[part], table, k=None if k is None else k[part],
                                         layout=layout))
        assert torch.equal(got[0][part], want[0]) and torch.equal(got[1][part], want[1])
    # rows that do not lie in one run: tensors of their own, and one of them a slice
    kc = None if k is None else k.contiguous()
    for qq, kk in ((q.contiguous(), kc), (q.contiguous(), k), (q, kc)):
        again = both(pkb.rotary_embedding(qq, pos, table, k=kk, layout=layout))
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    pkb.rotary_embedding(q, pos, table, k=k, layout=layout, q_out=q, k_out=k)
    assert torch.equal(q, got[0]) and (k is None or torch.equal(k, got[1]))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_and_negative_positions(layout):
    """Any int32 position: the angle of the last one is as exact as that of the first."""
    gen = torch.Generator().manual_seed(1)
    pos = [2 ** 31 - 1, -2 ** 31, -1, -8191, 1 << 30, 123456789]
    q = rows(gen, len(pos), 2, 16, dtype=torch.float32)
    table, _ = pkb.rope_frequencies(16)
    out = pkb.rotary_embedding(q, torch.tensor(pos, dtype=torch.int32, device=DEV), table,
                               layout=layout)
    want, size = O.rotate(q, pos, O.frequencies(16)[0], layout=layout)
    close(out, want, size)


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("ntk", 8.0), ("yarn", 40.0),
                                            ("wavelength", 8.0)])
def test_scaled_frequencies(scaling, factor):
    gen = torch.Generator().manual_seed(2)
    q = rows(gen, 3, 2, 128, dtype=torch.float32)
    pos = [3, 8191, 120000]
    table, m = pkb.rope_frequencies(128, scaling=scaling, factor=factor,
                                    original_max_position=4096)
    f, wm = O.frequencies(128, scaling=scaling, factor=factor, original=4096.0)
    out = pkb.rotary_embedding(q, torch.tensor(pos, dtype=torch.int32, device=DEV), table,
                               attention_factor=m)
    want, size = O.rotate(q, pos, f, m=wm)
    # the two evaluations of the frequencies differ by about 1e-13 relative: at position
    # 120000 that is 1.2e-8 rad
    close(out, want, size + size * 1.2e-8 / (8 * 2.0 ** -24))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("R", [32, 20])
def test_in_place_touches_the_rotated_columns_only(layout, R):
    gen = torch.Generator().manual_seed(4)
    q = rows(gen, 7, 3, 48, dtype=torch.bfloat16)
    k = rows(gen, 7, 2, 48, dtype=torch.bfloat16)
    pos = torch.arange(7, dtype=torch.int32, device=DEV) * 100
    table, _ = pkb.rope_frequencies(R)
    want = pkb.rotary_embedding(q, pos, table, k=k, layout=layout)
    q2, k2 = q.clone(), k.clone()
    got = pkb.rotary_embedding(q2, pos, table, k=k2, layout=layout, q_out=q2, k_out=k2)
    assert got[0].data_ptr() == q2.data_ptr()
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])


@pytest.mark.parametrize("D", [32, 512])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides_and_alignment(dtype, layout, D):
    """Slices of a fused projection, head-major storage, rows that start on odd elements, and a
    batch of sequences: all give what contiguous rows give."""
    gen = torch.Generator().manual_seed(6)
    T, Hq, Hk = 9, 4, 2
    table, _ = pkb.rope_frequencies(D)
    pos = torch.randint(0, 9999, (T,), generator=gen, dtype=torch.int32).to(DEV)
    fused = rows(gen, T, Hq + 2 * Hk, D, dtype=dtype)
    q, k = fused[:, :Hq], fused[:, Hq:Hq + Hk]
    want = pkb.rotary_embedding(q.contiguous(), pos, table, k=k.contiguous(), layout=layout)
    got = pkb.rotary_embedding(q, pos, table, k=k, layout=layout)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # in place inside the fused rows: the values' heads stay
    f2 = fused.clone()
    pkb.rotary_embedding(f2[:, :Hq], pos, table, k=f2[:, Hq:Hq + Hk], layout=layout,
                         q_out=f2[:, :Hq], k_out=f2[:, Hq:Hq + Hk])
    assert torch.equal(f2[:, :Hq], want[0]) and torch.equal(f2[:, Hq:Hq + Hk], want[1])
    assert torch.equal(f2[:, Hq + Hk:], fused[:, Hq + Hk:])
    # heads first in memory, in and out
    hq = q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(Hq, T, D, dtype=dtype, device=DEV).transpose(0, 1)
    assert torch.equal(pkb.rotary_embedding(hq, pos, table, layout=layout, q_out=out), want[0])
    # rows that start 1, 2 or 4 elements into their storage, and odd strides between tokens
    for off in (1, 2, 4):
        wide = torch.zeros(T, Hq * D + off, dtype=dtype, device=DEV)
        view = wide[:, off:].unflatten(1, (Hq, D))
        view.copy_(q)
        assert torch.equal(pkb.rotary_embedding(view, pos, table, layout=layout), want[0])
    q4 = q[:8].reshape(2, 4, Hq, D)
    got = pkb.rotary_embedding(q4, pos[:8].view(2, 4).contiguous(), table, layout=layout)
    assert torch.equal(got.view(8, Hq, D), want[0][:8])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient(layout):
    """inverse=True is the gradient: against the transposed map written out as a matrix in 64
    bits, and against differences of the forward call."""
    gen = torch.Generator().manual_seed(8)
    T, H, D, R, m = 4, 2, 24, 16, 1.375
    pos = [0, 5, 70000, 1000001]
    table, _ = pkb.rope_frequencies(R)
    dpos = torch.tensor(pos, dtype=torch.int32, device=DEV)
    f, _ = O.frequencies(R)
    g = rows(gen, T, H, D, dtype=torch.float32)
    grad = pkb.rotary_embedding(g, dpos, table, layout=layout, attention_factor=m, inverse=True)
    want, size = O.rotate(g, pos, f, layout=layout, m=m, inverse=True)
    eye = np.broadcast_to(np.eye(D)[:, None, :], (D, T, D)).reshape(D * T, 1, D)
    J = O.rotate(eye, pos * D, f, layout=layout, m=m)[0].reshape(D, T, D)     # J[i] = d y / d x_i
    byhand = np.einsum("itj,thj->thi", J, g.double().cpu().numpy())
    np.testing.assert_allclose(want, byhand, rtol=0, atol=1e-12)
    close(grad, want, size)
    # the map is linear: a difference over a step of 1 is exact but for the roundings of both
    # evaluations, each below 8 * 2^-24 of m (|x1| + |x2|) plus half a step of the output
    x = rows(gen, T, H, D, dtype=torch.float32)
    base = pkb.rotary_embedding(x, dpos, table, layout=layout, attention_factor=m)
    for i in range(D):
        x2 = x.clone()
        x2[..., i] += 1.0
        diff = (pkb.rotary_embedding(x2, dpos, table, layout=layout, attention_factor=m) - base)
        num = (diff.double() * g.double()).sum(-1).cpu().numpy()
        worst = (x.abs().max() * 2 + 2).item() * m * 9 * 2.0 ** -24 * 2
        tol = worst * g.abs().double().sum(-1).cpu().numpy() + 1e-6
        assert (np.abs(num - want[..., i]) <= tol).all()


def test_infinities_stay_in_their_pair():
    q = torch.zeros(2, 1, 16, device=DEV)
    q[0, 0, 3], q[1, 0, 12] = float("inf"), float("nan")
    table, _ = pkb.rope_frequencies(8)
    pos = torch.tensor([5, 5], dtype=torch.int32, device=DEV)
    out = pkb.rotary_embedding(q, pos, table)
    bad = ~torch.isfinite(out)
    assert bad[0, 0].nonzero().flatten().tolist() == [3, 7]
    assert bad[1, 0].nonzero().flatten().tolist() == [12]


def test_more_elements_than_31_bits():
    """Rows behind element 2^31 of their tensors, with and without staging."""
    T, H, D = 140000, 64, 256
    q = torch.zeros(T, H, D, dtype=torch.bfloat16, device=DEV)                  # 4.6 GB
    gen = torch.Generator().manual_seed(3)
    tail = rows(gen, 40, H, D, dtype=torch.bfloat16)
    q[-40:] = tail
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    table, _ = pkb.rope_frequencies(D)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pkb.rotary_embedding(q, pos, table, status=status)
    want = pkb.rotary_embedding(tail, pos[-40:], table)
    assert torch.equal(out[-40:], want) and not out[:-40].any() and status.item() == 0
    # heads first: a head stride that is no multiple of D rules staging out
    view = q.view(-1)[:(T - 1) * H * D].view(H, T - 1, D).transpose(0, 1)
    got = pkb.rotary_embedding(view[-3:], pos[-3:], table)
    assert torch.equal(got, pkb.rotary_embedding(view[-3:].contiguous(), pos[-3:], table))


@pytest.mark.parametrize("T", [1, 3, 700])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_broadcast_inputs(T, layout):
    # one row for all heads, or for all tokens: the same bits as from the repeated rows
    gen = torch.Generator().manual_seed(15)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    table, _ = pkb.rope_frequencies(64)
    by_head = rows(gen, T, 1, 64, dtype=torch.bfloat16).expand(T, 6, 64)
    by_token = rows(gen, 1, 2, 64, dtype=torch.bfloat16).expand(T, 2, 64)
    got = pkb.rotary_embedding(by_head, pos, table, k=by_token, layout=layout)
    want = pkb.rotary_embedding(by_head.contiguous(), pos, table, k=by_token.contiguous(),
                                layout=layout)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if T > 1:
        for out in (by_head, torch.zeros(1, 6, 64, device=DEV).bfloat16().expand(T, 6, 64)):
            with pytest.raises(pkb.PagedAttnError):
                pkb.rotary_embedding(by_head.contiguous(), pos, table, q_out=out, layout=layout)


def test_other_stream_and_graph():
    gen = torch.Generator().manual_seed(9)
    q = rows(gen, 33, 4, 64, dtype=torch.bfloat16)
    pos = torch.arange(33, dtype=torch.int32, device=DEV)
    table, _ = pkb.rope_frequencies(64)
    want = pkb.rotary_embedding(q, pos, table)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkb.rotary_embedding(q, pos, table, q_out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkb.rotary_embedding(q, pos, table, q_out=out)
    pos.add_(3)
    want = pkb.rotary_embedding(q, pos, table)
    graph.replay()
    assert torch.equal(out, want)


def test_graph_between_other_kernels():
    """Captured between kernels of another library, a memset and a copy, long and short calls: each
    waits for what precedes it and is waited for."""
    gen = torch.Generator().manual_seed(10)
    table, _ = pkb.rope_frequencies(64)
    for T in (40, 5000):
        q = rows(gen, T, 6, 64, dtype=torch.bfloat16)
        pos = torch.arange(T, dtype=torch.int32, device=DEV)
        buf = {n: torch.zeros_like(q) for n in ("in", "a", "b", "c")}

        def chain():
            buf["a"].zero_()
            buf["in"].mul_(2)
            pkb.rotary_embedding(buf["in"], pos, table, q_out=buf["a"])
            pkb.rotary_embedding(buf["a"], pos, table, q_out=buf["b"])
            buf["a"].add_(1)
            buf["c"].copy_(buf["b"])
            pkb.rotary_embedding(buf["c"], pos, table, q_out=buf["c"], inverse=True)
            buf["c"].add_(buf["a"])
        buf["in"].copy_(q)
        chain()
        torch.cuda.synchronize()
        want = {n: t.clone() for n, t in buf.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain()
        for t in buf.values():
            t.fill_(float("nan"))
        for _ in range(5):
            buf["in"].copy_(q)
            graph.replay()
        for n, t in buf.items():
            assert torch.equal(t, want[n]), (T, n)


def test_refusals():
    table, _ = pkb.rope_frequencies(32)
    q = torch.zeros(4, 2, 32, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    for kw in (dict(positions=pos[:3]), dict(positions=pos.long()), dict(freqs=table.float()),
               dict(q=q.double()), dict(k=q[:3]), dict(k=q.half()), dict(k=q[..., :16].contiguous()),
               dict(q=q.transpose(1, 2)), dict(q_out=q[:, :1]), dict(q_out=q.half()),
               dict(k_out=q), dict(q=q[0])):
        a = dict(q=q, positions=pos, freqs=table)
        a.update(kw)
        with pytest.raises(ValueError):
            pkb.rotary_embedding(**a)
    with pytest.raises(pkb.PagedAttnError):           # in place, but stepping differently
        fused = torch.zeros(4, 4, 32, device=DEV)
        pkb.rotary_embedding(fused[:, :2], pos, table, q_out=fused.view(8, 2, 32)[:4])
    with pytest.raises(pkb.PagedAttnError):           # more rotated columns than a head has
        pkb.rotary_embedding(q[..., :16].contiguous(), pos, table)
    assert pkb.rotary_embedding(q[:0], pos[:0], table).shape == (0, 2, 32)
