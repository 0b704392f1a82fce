"""fp64 CPU oracle of the paged cache: rotary positions, page bookkeeping, and
attention over pages.

TEST INFRASTRUCTURE, NOT PRODUCT CODE: plain loops written from the definitions
in include/littlebit.h, sharing no code with the CUDA package.
"""
from __future__ import annotations

import math

import numpy as np

PAGES, INDEX = 1 << 8, 1 << 9   # status bits LB_ERR_PAGES and LB_ERR_INDEX


# ------------------------------------------------------------------ rotary positions
def frequencies(rotary_dim, base=10000.0, factor=1.0, bands=None, log_ramp=False):
    """Radians per token of every pair."""
    out = []
    for i in range(rotary_dim // 2):
        f = base ** (-2.0 * i / rotary_dim)
        keep = 0.0
        if bands is not None:
            original, slow, fast = bands
            turns = original * f / (2 * math.pi)
            if log_ramp:
                keep = (math.log(turns) - math.log(slow)) / (math.log(fast) - math.log(slow))
            else:
                keep = (turns - slow) / (fast - slow)
            keep = min(1.0, max(0.0, keep))
        out.append(f * keep + f / factor * (1 - keep))
    return np.array(out)


def rotate(x, positions, rotary_dim, interleaved=False, scale=1.0, inverse=False, **how):
    """x (tokens, heads, width) float64, each pair turned by its angle."""
    y = np.array(x, dtype=np.float64)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * frequencies(rotary_dim, **how)
    if inverse:
        angle = -angle
    for i in range(rotary_dim // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)
        c, s = np.cos(angle[:, i])[:, None], np.sin(angle[:, i])[:, None]
        p, q = x[..., a].astype(np.float64), x[..., b].astype(np.float64)
        y[..., a], y[..., b] = scale * (p * c - q * s), scale * (q * c + p * s)
    return y


# ------------------------------------------------------------------ bookkeeping
class Model:
    """A cache as Python sees it: the tables as numpy arrays, planes as numpy
    arrays (n_pages, heads, page_size, width) of any type, and the status word."""

    def __init__(self, n_pages, page_size, n_slots, max_pages, planes=()):
        self.ps, self.n_slots, self.max_pages, self.n_pages = page_size, n_slots, max_pages, n_pages
        self.table = np.full((n_slots, max_pages), -1, dtype=np.int32)
        self.length = np.zeros(n_slots, dtype=np.int32)
        self.refs = np.zeros(n_pages, dtype=np.int32)
        self.planes = list(planes)
        self.status = 0

    def pages(self, tokens):
        return -(-tokens // self.ps)

    def _free(self):
        return [int(p) for p in np.nonzero(self.refs == 0)[0]]

    def _slot(self, s):
        if s == -1:
            return False
        if not 0 <= s < self.n_slots:
            self.status |= INDEX
            return False
        return True

    def extend(self, slots, starts, tokens, prefix=-1):
        where = np.full(tokens, -1, dtype=np.int64)
        positions = np.full(tokens, -1, dtype=np.int32)
        free, taken, asked, done = self._free(), set(), 0, []
        for i, s in enumerate(slots):
            n = starts[i + 1] - starts[i]
            if not self._slot(s):
                continue
            if s in taken:
                self.status |= INDEX
                continue
            length = int(self.length[s])
            if n and length % self.ps and self.refs[self.table[s, length // self.ps]] != 1:
                self.status |= INDEX
                continue
            taken.add(s)
            if self.pages(length + n) > self.max_pages:
                self.status |= PAGES
                continue
            need = self.pages(length + n) - self.pages(length)
            if asked + need > len(free):   # asks for nothing then: those behind may still fit
                self.status |= PAGES
                continue
            asked += need
            for k in range(need):
                page = free[asked - need + k]
                self.table[s, self.pages(length) + k] = page
                self.refs[page] = 1
            done.append((i, s, length, n))
        for i, s, length, n in done:
            self.length[s] = length + n
        shift = int(self.length[prefix]) if prefix >= 0 else 0
        for i, s, length, n in done:
            for j in range(n):
                at = length + j
                where[starts[i] + j] = int(self.table[s, at // self.ps]) * self.ps + at % self.ps
                positions[starts[i] + j] = at + shift
        return where, positions

    def locate(self, slots, starts, tokens, first=None, prefix=-1):
        where = np.full(tokens, -1, dtype=np.int64)
        positions = np.full(tokens, -1, dtype=np.int32)
        shift = int(self.length[prefix]) if prefix >= 0 else 0
        for i, s in enumerate(slots):
            for j in range(starts[i + 1] - starts[i]):
                if s == -1:
                    continue
                at = j + (0 if first is None else int(first[i]))
                if not (0 <= s < self.n_slots and 0 <= at < self.length[s]):
                    self.status |= INDEX
                    continue
                where[starts[i] + j] = int(self.table[s, at // self.ps]) * self.ps + at % self.ps
                positions[starts[i] + j] = at + shift
        return where, positions

    def fork(self, parents, children):
        free, used, asked, taken, before = self._free(), 0, 0, set(), self.length.copy()
        for p, c in zip(parents, children):
            if p == -1 or c == -1:
                continue
            if not (0 <= p < self.n_slots and 0 <= c < self.n_slots) or p == c or before[c] or c in taken:
                self.status |= INDEX
                continue
            n = int(before[p])
            full, rest = n // self.ps, n % self.ps
            if rest and not 0 <= self.table[p, full] < self.n_pages:
                self.status |= INDEX
                continue
            taken.add(c)
            if rest:
                asked += 1
                if asked > len(free):
                    self.status |= PAGES
                    continue
                page = free[asked - 1]
                self.refs[page] = 1
                for plane in self.planes:
                    plane[page, :, :rest] = plane[self.table[p, full], :, :rest]
                self.table[c, full] = page
            for k in range(full):
                self.table[c, k] = self.table[p, k]
                self.refs[self.table[p, k]] += 1
            self.length[c] = n

    def free(self, slots):
        for s in slots:
            if self._slot(s):
                for k in range(self.pages(int(self.length[s]))):
                    self.refs[self.table[s, k]] -= 1
                    self.table[s, k] = -1
                self.length[s] = 0

    def compact(self):
        live = [int(p) for p in np.nonzero(self.refs > 0)[0]]
        n = len(live)
        movers, holes = [p for p in live if p >= n], [p for p in range(n) if self.refs[p] <= 0]
        to = {p: p for p in live}
        to.update(zip(movers, holes))
        for src, dst in zip(movers, holes):
            for plane in self.planes:
                plane[dst] = plane[src]
            self.refs[dst], self.refs[src] = self.refs[src], 0
        for s in range(self.n_slots):
            for k in range(self.pages(int(self.length[s]))):
                self.table[s, k] = to[int(self.table[s, k])]
        return n

    def rows(self, plane, slot, count=None):
        """The rows that a slot holds, (heads, tokens, width)."""
        n = int(self.length[slot]) if count is None else count
        parts = [plane[self.table[slot, k]] for k in range(self.pages(n))]
        joined = np.concatenate(parts, axis=1) if parts else plane[:1, :, :0][0]
        return joined[:, :n]


# ------------------------------------------------------------------ attention
def attend(q, keys, values, slots, starts, prefix=-1, scale=None):
    """q (tokens, query heads, width); keys, values: slot -> (heads, tokens, width).
    Returns (out, reach, size): the outputs, sum_j w_j |v_j| / sum_j w_j, and
    per (token, head) the number of keys and the largest scale * sum_d |q_d k_jd|."""
    T, Hq, D = q.shape
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, reach = np.zeros(q.shape), np.zeros(q.shape)
    size = np.zeros((T, Hq, 2))
    for i, s in enumerate(slots):
        n = int(starts[i + 1] - starts[i])
        for j in range(n):
            t = int(starts[i]) + j
            for h in range(Hq):
                k, v = [], []
                if prefix >= 0:
                    g = Hq // keys(prefix).shape[0]
                    k.append(keys(prefix)[h // g])
                    v.append(values(prefix)[h // g])
                if s >= 0:
                    g = Hq // keys(s).shape[0]
                    seen = max(0, keys(s).shape[1] - n + j + 1)
                    k.append(keys(s)[h // g, :seen])
                    v.append(values(s)[h // g, :seen])
                if not k or sum(len(x) for x in k) == 0:
                    continue
                k, v = np.concatenate(k).astype(np.float64), np.concatenate(v).astype(np.float64)
                x = q[t, h].astype(np.float64)
                score = scale * (k @ x)
                w = np.exp(score - score.max())
                out[t, h], reach[t, h] = w @ v / w.sum(), w @ np.abs(v) / w.sum()
                size[t, h] = len(k), abs(scale) * (np.abs(k) @ np.abs(x)).max()
    return out, reach, size


def attend_tolerance(out, reach, size, half_step, width):
    """How far an output may be off: the weights and the output are each rounded
    once to the type (half_step, relative), and what is summed in fp32 -- scores
    over the width, weights and products over the keys -- is off by at most
    2^-24 of the sum of magnitudes per addition; exp2 by 2^-21.  An error d of a
    score changes its weight by a factor within 1 +- 2 d, in the numerator and
    in the denominator; weights below the type's normal range are off by 2^-25
    of the largest at most (fp16)."""
    step = 2.0 ** -24
    d = (width + 4) * step * size[..., 1:] + 2 ** -21
    soft = 2 * (2 * d + step * size[..., :1])
    tiny = size[..., :1] * 2.0 ** -25 * np.abs(reach).max(-1, keepdims=True) if half_step < 2.0 ** -9 else 0.0
    return (half_step + soft) * reach + half_step * np.abs(out) + tiny + 2.0 ** -24
