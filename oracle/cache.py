"""Float64 / integer reference of the cache-side operators (include/paged_cache.h), on the CPU.

Rotations use angles reduced in 50-digit decimals, so any int32 position is exact; the page
operations are sequential loops over Python integers.  Test infrastructure only: it shares no
code with the library.
"""
from __future__ import annotations

import math
from decimal import Decimal, getcontext

import numpy as np
import torch

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628621")

METADATA, CAPACITY = 4, 2        # status bits


def frequencies(rotary_dim, *, base=10000.0, scaling="none", factor=1.0, original=0.0,
                low=None, high=None):
    """(angles per position [rotary_dim / 2], attention factor), one pair at a time."""
    R, out = rotary_dim, []
    if scaling == "ntk" and R > 2:
        base = base * factor ** (R / (R - 2))
    if scaling == "yarn":
        low, high = low or 1.0, high or 32.0

        def pair_with(turns):
            return R * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(math.floor(pair_with(high)), 0), min(math.ceil(pair_with(low)), R - 1)
    if scaling == "wavelength":
        low, high = low or 1.0, high or 4.0
    for i in range(R // 2):
        f = 1.0 / base ** (2 * i / R)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            g = (i - first) / max(last - first, 0.001)
            g = 0.0 if g < 0 else 1.0 if g > 1 else g
            f = (1 - g) * f + g * (f / factor)
        elif scaling == "wavelength":
            wavelength = 2 * math.pi / f
            if wavelength > original / low:
                f = f / factor
            elif wavelength >= original / high:
                c = (original / wavelength - low) / (high - low)
                f = (1 - c) * f / factor + c * f
        out.append(f)
    m = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0
    return np.array(out), m


def angles(positions, freqs):
    """p * f modulo one turn, in radians [-pi, pi], exact to about 2^-52 for any int32 p."""
    turns = [Decimal(float(f)) / (2 * PI) for f in freqs]
    a = np.empty((len(positions), len(freqs)))
    for t, p in enumerate(positions):
        for i, f in enumerate(turns):
            x = int(p) * f
            a[t, i] = float((x - x.to_integral_value()) * 2 * PI)
    return a


def rotate(x, positions, freqs, *, layout="half", m=1.0, inverse=False):
    """x [T, H, D] (any float type) rotated; float64.  The second value bounds what an fp32
    evaluation may be off by: (|x1| + |x2|) m per pair (times the caller's unit)."""
    x = x.double().cpu().numpy() if isinstance(x, torch.Tensor) else np.asarray(x, np.float64)
    y, size = x.copy(), np.zeros_like(x)
    n = len(freqs)
    a = angles(positions, freqs)
    if inverse:
        a = -a
    for i in range(n):
        j, k = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = np.cos(a[:, i])[:, None], np.sin(a[:, i])[:, None]
        y[..., j] = m * (x[..., j] * c - x[..., k] * s)
        y[..., k] = m * (x[..., k] * c + x[..., j] * s)
        size[..., j] = size[..., k] = abs(m) * (np.abs(x[..., j]) + np.abs(x[..., k]))
    return y, size


def append(k, v, lens, tables, page_size, num_pages, *, starts, freqs=None, layout="half",
           m=1.0):
    """What an append writes: a list of (token, page, slot) and the positions of every token
    (None: no request owns it).  tables: one list of page ids per request."""
    total = k.shape[0]
    where, positions = [], [None] * total
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            t = starts[b] + i
            p = int(lens[b]) - n + i
            positions[t] = p
            j = p // page_size
            if p < 0 or j >= len(tables[b]) or not 0 <= tables[b][j] < num_pages:
                continue
            where.append((t, int(tables[b][j]), p % page_size))
    return where, positions


class State:
    """Tables [R][C], lengths, page counts and the layers' pools ([P, X, ps, D] arrays, X the
    heads of K and V together, as integers or floats: only moved, never computed with)."""

    def __init__(self, tables, lens, refs, page_size, pools=()):
        self.tables = [list(map(int, r)) for r in tables]
        self.lens = [int(x) for x in lens]
        self.refs = [int(x) for x in refs]
        self.ps, self.pools, self.status = page_size, [p.copy() for p in pools], 0
        self.R, self.C, self.P = len(self.lens), len(self.tables[0]), len(self.refs)

    def pages(self, n):
        return -(-n // self.ps)

    def free(self, rows):
        for r in rows:
            if not 0 <= r < self.R:
                self.status |= METADATA
                continue
            n, self.lens[r] = self.pages(self.lens[r]), 0
            if n > self.C:
                self.status |= METADATA
            for p in self.tables[r][:max(n, 0)]:
                if 0 <= p < self.P and self.refs[p] > 0:
                    self.refs[p] -= 1
                else:
                    self.status |= METADATA

    def _grant(self, needs):
        """(pages of each item, or None where the free pages do not suffice)."""
        free = [p for p in range(self.P) if self.refs[p] == 0]
        at, got = 0, []
        for n in needs:
            if n == 0:
                got.append([])
            elif at + n <= len(free):
                got.append(free[at:at + n])
            else:
                got.append(None)
                self.status |= CAPACITY
            at += n
        return got

    def extend(self, rows, new):
        items, seen = [], set()
        for r, m in zip(rows, new):
            ok = 0 <= r < self.R and m >= 0 and self.lens[r] >= 0
            ok = ok and self.lens[r] + m < 2 ** 31 and self.pages(self.lens[r] + m) <= self.C
            if not ok or r in seen:
                self.status |= METADATA
                continue
            seen.add(r)
            items.append((r, m, self.pages(self.lens[r] + m) - self.pages(self.lens[r])))
        for (r, m, n), pages in zip(items, self._grant([i[2] for i in items])):
            if pages is None:
                continue
            have = self.pages(self.lens[r])
            for j, p in enumerate(pages):
                self.tables[r][have + j] = p
                self.refs[p] = 1
            self.lens[r] += m

    def fork(self, parents, children):
        before, items, seen = list(self.lens), [], set()
        for a, c in zip(parents, children):
            ok = 0 <= a < self.R and 0 <= c < self.R and a != c and before[c] == 0
            ok = ok and before[a] >= 0 and self.pages(before[a]) <= self.C
            full, tail = divmod(before[a], self.ps) if ok else (0, 0)
            ok = ok and (tail == 0 or 0 <= self.tables[a][full] < self.P)
            if not ok or c in seen:
                self.status |= METADATA
                continue
            seen.add(c)
            items.append((a, c, int(tail > 0)))
        for (a, c, n), pages in zip(items, self._grant([i[2] for i in items])):
            if pages is None:
                continue
            full, tail = divmod(before[a], self.ps)
            for j in range(full):
                p = self.tables[a][j]
                self.tables[c][j] = p
                if 0 <= p < self.P:
                    self.refs[p] += 1
                else:
                    self.status |= METADATA
            for p in pages:
                self.tables[c][full] = p
                self.refs[p] = 1
                s = self.tables[a][full]
                for pool in self.pools:
                    pool[p, :, :tail] = pool[s, :, :tail]
            self.lens[c] = before[a]

    def compact(self):
        """Returns the number of live pages."""
        live = sum(r != 0 for r in self.refs)
        src = [p for p in range(live, self.P) if self.refs[p] != 0]
        dst = [p for p in range(live) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
            for pool in self.pools:
                pool[d] = pool[s]
        for r in range(self.R):
            n = self.pages(self.lens[r])
            if n > self.C:
                self.status |= METADATA
            for j in range(min(max(n, 0), self.C)):
                p = self.tables[r][j]
                if not 0 <= p < self.P:
                    self.status |= METADATA
                self.tables[r][j] = to.get(p, p)
        return live


def copy_pages(src_pools, dst_pools, src, dst):
    """Returns the status bits."""
    status = 0
    for s, d in zip(src, dst):
        if not (0 <= s < src_pools[0].shape[0] and 0 <= d < dst_pools[0].shape[0]):
            status |= METADATA
            continue
        for a, b in zip(src_pools, dst_pools):
            b[d] = a[s]
    return status
