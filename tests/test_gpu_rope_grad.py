"""The rotation under autograd on the GPU: gradients against the transposed map in 64 bits."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import cache as O
from tests.test_gpu_rope import close, rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D,R", [(64, 64), (24, 16), (128, 30)])
def test_gradients_match_the_transposed_map(dtype, layout, inverse, D, R):
    gen = torch.Generator().manual_seed(D + R)
    T, Hq, Hk = 5, 3, 2
    table, m = pkb.rope_frequencies(R, scaling="yarn", factor=4.0, original_max_position=2048)
    f, wm = O.frequencies(R, scaling="yarn", factor=4.0, original=2048.0)
    pos = [0, 3, 70000, -5, 2047]
    dpos = torch.tensor(pos, dtype=torch.int32, device=DEV)
    q, k = (rows(gen, T, h, D, dtype=dtype).requires_grad_() for h in (Hq, Hk))
    outs = pkb.rotary_embedding(q, dpos, table, k=k, layout=layout, attention_factor=m,
                                inverse=inverse)
    with torch.no_grad():
        again = pkb.rotary_embedding(q, dpos, table, k=k, layout=layout, attention_factor=m,
                                     inverse=inverse)
    grads = [rows(gen, *y.shape, dtype=dtype) for y in outs]
    torch.autograd.backward(outs, grads)
    for x, y, z, g in zip((q, k), outs, again, grads):
        assert torch.equal(y, z)
        want, size = O.rotate(g, pos, f, layout=layout, m=wm, inverse=not inverse)
        # far positions: the two evaluations of the frequencies differ by about 1e-13 relative
        close(x.grad, want, size + size * 7e-9 / (8 * 2.0 ** -24))


def test_a_layer_and_its_differences():
    """Slices of one projection, rotated and multiplied: the projection's gradient against
    differences of the same layer in 64 bits."""
    gen = torch.Generator().manual_seed(3)
    T, H, D = 4, 2, 8
    table, _ = pkb.rope_frequencies(D)
    f, _ = O.frequencies(D)
    pos = [0, 1, 2, 3]
    dpos = torch.tensor(pos, dtype=torch.int32, device=DEV)
    fused = rows(gen, T, 2 * H, D, dtype=torch.float32).requires_grad_()
    weight = rows(gen, T, H, D, dtype=torch.float32)

    q, k = pkb.rotary_embedding(fused[:, :H], dpos, table, k=fused[:, H:])
    (q * k * weight).sum().backward()

    def loss(x):
        a, _ = O.rotate(x[:, :H], pos, f)
        b, _ = O.rotate(x[:, H:], pos, f)
        return (a * b * weight.double().cpu().numpy()).sum()
    x = fused.detach().double().cpu().numpy()
    # central differences of a quadratic are exact but for rounding (2^-52 of sums below 100, over
    # a step of 1/64); the fp32 layer: about 30 roundings of values below 8 * 8
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += 1 / 128
        down[i] -= 1 / 128
        want = (loss(up) - loss(down)) * 64
        assert abs(fused.grad[i].item() - want) <= 30 * 64 * 2.0 ** -24


def test_shared_rows_and_one_sided_gradients():
    """A row that all heads share gets the sum of their gradients; gradients that are one value for
    all elements, and of k alone."""
    gen = torch.Generator().manual_seed(4)
    T, H, D = 6, 4, 16
    table, _ = pkb.rope_frequencies(D)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    one = rows(gen, T, 1, D, dtype=torch.float32).requires_grad_()
    k = rows(gen, T, 2, D, dtype=torch.float32).requires_grad_()
    out, ko = pkb.rotary_embedding(one.expand(T, H, D), pos, table, k=k)
    out.sum().backward(retain_graph=True)
    ones = torch.ones(T, H, D, device=DEV)
    back = pkb.rotary_embedding(ones, pos, table, inverse=True)
    assert torch.equal(one.grad, back.sum(1, keepdim=True)) and k.grad is None
    g = rows(gen, T, 2, D, dtype=torch.float32)
    got, = torch.autograd.grad(ko, k, g)
    assert torch.equal(got, pkb.rotary_embedding(g, pos, table, inverse=True))
    # 4-dimensional rows, and a gradient whose heads come first in memory
    q4 = rows(gen, 2, 3, H, D, dtype=torch.float32).requires_grad_()
    p4 = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
    g4 = rows(gen, H, 2, 3, D, dtype=torch.float32).permute(1, 2, 0, 3)
    got, = torch.autograd.grad(pkb.rotary_embedding(q4, p4, table), q4, g4)
    assert torch.equal(got, pkb.rotary_embedding(g4.contiguous(), p4, table, inverse=True))


def test_the_gradient_has_a_gradient():
    gen = torch.Generator().manual_seed(5)
    table, _ = pkb.rope_frequencies(8)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    q = rows(gen, 3, 2, 8, dtype=torch.float32).requires_grad_()
    v = rows(gen, 3, 2, 8, dtype=torch.float32).requires_grad_()
    g, = torch.autograd.grad(pkb.rotary_embedding(q, pos, table), q, v, create_graph=True)
    w = rows(gen, 3, 2, 8, dtype=torch.float32)
    got, = torch.autograd.grad(g, v, w)
    assert torch.equal(got, pkb.rotary_embedding(w, pos, table))


def test_on_another_stream():
    gen = torch.Generator().manual_seed(6)
    table, _ = pkb.rope_frequencies(64)
    T = 5000
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    q = rows(gen, T, 4, 64, dtype=torch.float32).requires_grad_()
    g = rows(gen, T, 4, 64, dtype=torch.float32)
    want = pkb.rotary_embedding(g, pos, table, inverse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, = torch.autograd.grad(pkb.rotary_embedding(q, pos, table), q, g)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_a_captured_forward_and_a_refused_gradient():
    """A captured call runs with inputs that require a gradient; its gradient is refused while a
    graph is captured, and inverse=True, which is that gradient, is captured instead."""
    gen = torch.Generator().manual_seed(7)
    table, _ = pkb.rope_frequencies(16)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    q = rows(gen, 9, 2, 16, dtype=torch.float32).requires_grad_()
    g = rows(gen, 9, 2, 16, dtype=torch.float32)
    want = pkb.rotary_embedding(q, pos, table).detach(), pkb.rotary_embedding(g, pos, table,
                                                                              inverse=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkb.rotary_embedding(q, pos, table)
        with pytest.raises(ValueError):
            torch.autograd.grad(out, q, g)
        back = pkb.rotary_embedding(g, pos, table, inverse=True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(back, want[1])


def test_a_captured_gradient_beside_an_eager_graph():
    """A backward pass under capture while an eager graph of the same leaf lives: refused as an
    exception, and the process goes on.  In a process of its own."""
    code = """
import torch, paged_kv_block_gb300 as pkb
table, _ = pkb.rope_frequencies(16)
pos = torch.arange(9, dtype=torch.int32, device="cuda")
x = torch.randn(9, 2, 16, device="cuda", requires_grad=True)
eager = pkb.rotary_embedding(x, pos, table).sum()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    loss = pkb.rotary_embedding(x, pos, table).sum()
    try:
        loss.backward()
    except ValueError as e:
        print("refused:", "inverse=True" in str(e))
    kept = pkb.rotary_embedding(x.detach(), pos, table)
graph.replay()
eager.backward()
torch.cuda.synchronize()
want = pkb.rotary_embedding(torch.ones_like(x), pos, table, inverse=True)
print(torch.equal(x.grad, want), torch.equal(kept, pkb.rotary_embedding(x.detach(), pos, table)))
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    assert run.stdout.split("\n")[:2] == ["refused: True", "True True"], run.stdout
