"""Plain 64-bit forms of the window-plus-sinks attention, the page calls and
the multi-axis rotation, for their tests (numpy and torch on the CPU; none of
the library's code)."""
from __future__ import annotations

import math

import numpy as np
import torch

BF16_U = 2.0 ** -8  # half a bf16 step, relative


def turn64(x, angle):
    """Pairs (2i, 2i + 1), i < n, of x [..., D] turned by angle [..., n] (64 bits)."""
    y = x.double().clone()
    n = angle.shape[-1]
    a, b = x[..., 0:2 * n:2].double(), x[..., 1:2 * n:2].double()
    c, s = torch.cos(angle), torch.sin(angle)
    y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * c - b * s, a * s + b * c
    return y


def rope64(x, pos, frac, theta):
    """x [n, H, D] at positions pos (list of n)."""
    D = x.shape[-1]
    i = torch.arange(int(math.floor(frac * D / 2)), dtype=torch.float64)
    freq = theta ** (-2.0 * i / D)
    ang = torch.tensor(pos, dtype=torch.float64)[:, None, None] * freq
    return turn64(x, ang.expand(x.shape[0], x.shape[1], -1))


def axes64(x, positions, pairs, theta, interleaved=False, ladders=False, inverse=False):
    """x [tokens, H, D], positions [n_axes, tokens]."""
    D = x.shape[-1]
    order = [(a, r) for a, n in enumerate(pairs) for r in range(n)]
    if interleaved:
        order.sort(key=lambda ar: (ar[1], ar[0]))
    ang = torch.zeros(x.shape[0], 1, len(order), dtype=torch.float64)
    for i, (a, r) in enumerate(order):
        f = theta ** (-r / pairs[a]) if ladders else theta ** (-2.0 * i / D)
        ang[:, 0, i] = positions[a].double() * (-f if inverse else f)
    return turn64(x, ang.expand(x.shape[0], x.shape[1], -1))


def sees(j, p, window, sinks):
    return j <= p and (j > p - window or j < sinks)


def attend64(q, K, V, pos, window, sinks, scale):
    """q [n, Hq, D] at positions pos (list), K and V [m, Hkv, D] at positions
    0..m-1 -> (out [n, Hq, D], lse [n, Hq]). Keys that no query sees are dropped
    before any arithmetic, so NaN there does not matter."""
    n, Hq, D = q.shape
    G = Hq // K.shape[1]
    p = torch.tensor(pos)[:, None]
    j = torch.arange(max(pos) + 1)
    see = (j <= p) & ((j > p - window) | (j < sinks))
    keys = see.any(0).nonzero().flatten()
    see, k, v = see[:, keys], K[keys].double(), V[keys].double()
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    lse = torch.zeros(n, Hq, dtype=torch.float64)
    for h in range(Hq):
        s = (q[:, h].double() @ k[:, h // G].T * scale).masked_fill(~see, -math.inf)
        lse[:, h] = torch.logsumexp(s, 1)
        out[:, h] = torch.softmax(s, 1) @ v[:, h // G]
    return out, lse


def attention_bound(out64, v_absmax):
    """Largest error that the kernels' bf16 roundings allow on top of their
    rounded operands: each weight is rounded (relative half step u) and
    normalised by the unrounded sum, which moves an output by at most
    u * max|v|; the output is rounded (u * |o|). 2^-10 covers the 32-bit sums,
    the exp2 and a rotated operand that rounds to the other side."""
    return BF16_U * (v_absmax + float(out64.abs().max())) + 2.0 ** -10


def kept_pages(length, window, sinks, ps):
    keep = set()
    for j in range(length):
        if window == 0 or j > length - window or j < sinks:
            keep.add(j // ps)
    return keep


class Book:
    """The page calls one entry at a time, on lists."""

    def __init__(self, n_seqs, pps, n_pages, ps):
        self.table = [[-1] * pps for _ in range(n_seqs)]
        self.n_pages, self.ps = n_pages, ps

    @property
    def refs(self):
        r = [0] * self.n_pages
        for row in self.table:
            for e in row:
                if e >= 0:
                    r[e] += 1
        return r

    def fork(self, parents):
        old = [list(r) for r in self.table]
        self.table = [[-1] * len(old[0]) if p < 0 else list(old[p]) for p in parents]

    def reserve(self, lens, new):
        """-> (lacking, copies [(src, dst, rows)])"""
        left, free = self.refs, [p for p, r in enumerate(self.refs) if r == 0]
        grants = []
        for b, (n, add) in enumerate(zip(lens, new)):
            if add:
                for i in range(n // self.ps, (n + add - 1) // self.ps + 1):
                    e = self.table[b][i]
                    if e < 0 or left[e] > 1:
                        grants.append((b, i, e))
                        if e >= 0:
                            left[e] -= 1
        if len(grants) > len(free):
            return len(grants) - len(free), []
        copies = []
        for (b, i, e), f in zip(grants, free):
            if e >= 0 and i == lens[b] // self.ps and lens[b] % self.ps:
                copies.append((e, f, lens[b] % self.ps))
            self.table[b][i] = f
        return 0, copies

    def trim(self, lens, window, sinks):
        for b, n in enumerate(lens):
            if n >= 0:
                keep = kept_pages(n, window, sinks, self.ps)
                self.table[b] = [e if i in keep else -1 for i, e in enumerate(self.table[b])]

    def compact(self):
        """-> (n_live, page map)"""
        refs = self.refs
        n = sum(1 for r in refs if r)
        holes = [p for p in range(n) if not refs[p]]
        to = {p: p for p in range(n) if refs[p]}
        for p in range(n, self.n_pages):
            if refs[p]:
                to[p] = holes.pop(0)
        self.table = [[to.get(e, e) for e in r] for r in self.table]
        return n, [to.get(p, -1) for p in range(self.n_pages)]


def random_book(rng, n_seqs, pps, n_pages, ps, fill):
    """A book with some entries filled, some of them shared."""
    bk = Book(n_seqs, pps, n_pages, ps)
    pages = list(rng.permutation(n_pages))
    for b in range(n_seqs):
        for i in range(pps):
            if rng.random() < fill:
                if b and rng.random() < 0.3 and bk.table[b - 1][i] >= 0:
                    bk.table[b][i] = bk.table[b - 1][i]
                elif pages:
                    bk.table[b][i] = int(pages.pop())
    return bk


def as_np(t):
    return np.asarray(t.detach().cpu())
