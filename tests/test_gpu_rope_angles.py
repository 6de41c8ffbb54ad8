"""Small angles: the sine of a slow pair at a near position keeps its bits.

A row with x1 = 0 and x2 = 1 comes back as (-sin a, cos a), each one product by 1 and one sum with
0: exact.  So the output is the kernel's sine.  Its relative error: the angle less whole quarter
turns is rounded once (2^-24, and a sine below an eighth of a turn is off by no more than its angle
is), sine and cosine are within 2 ulp (2^-22): together below 5 * 2^-24.  The table's entries are
nearest to 2^-64 of a turn, so position p adds |p| 2^-65 of a turn; the oracle's angles are off by
2^-52 relative."""
import math

import numpy as np
import pytest
import torch

import paged_kv_block_gb300 as pkb
from oracle import cache as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def off(got, want, positions):
    bound = (5 * 2.0 ** -24 + 2.0 ** -51) * np.abs(want)
    bound = bound + np.abs(np.array(positions, np.float64))[:, None] * 2.0 ** -65 * 2 * math.pi
    return (np.abs(got - want) - bound).max()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("base,factor", [(1e4, 1.0), (1e4, 40.0), (5e5, 8.0), (1e6, 64.0)])
def test_sines_of_slow_pairs(base, factor, inverse, layout):
    R = 128
    freqs = [base ** (-2 * i / R) / factor for i in range(R // 2)]
    positions = [0, 1, -1, 2, 3, 17, 100, -4095, 70000, 2 ** 31 - 1]
    table, _ = pkb.rope_frequencies(R, inv_freq=freqs)
    q = torch.zeros(len(positions), 2, R, device=DEV)
    second = slice(R // 2, R) if layout == "half" else slice(1, R, 2)
    first = slice(0, R // 2) if layout == "half" else slice(0, R, 2)
    q[..., second] = 1.0
    pos = torch.tensor(positions, dtype=torch.int32, device=DEV)
    out = pkb.rotary_embedding(q, pos, table, layout=layout, inverse=inverse).double().cpu().numpy()
    a = O.angles(positions, freqs) * (-1.0 if inverse else 1.0)
    for h in range(2):
        assert off(out[:, h, first], -np.sin(a), positions) <= 0
        assert off(out[:, h, second], np.cos(a), positions) <= 0


def test_angles_on_both_sides_of_zero_are_mirror_images():
    """No direction is preferred: position -p gives the sine of p with its sign changed."""
    table, _ = pkb.rope_frequencies(128, base=1e6)
    p = torch.arange(1, 2001, dtype=torch.int32, device=DEV)
    q = torch.randn(2000, 1, 128, generator=torch.Generator().manual_seed(1)).to(DEV)
    ahead = pkb.rotary_embedding(q, p, table)
    back = pkb.rotary_embedding(q, -p, table, inverse=True)
    assert torch.equal(ahead, back)
