"""Helpers of the tree-verify tests: random trees and caches, and the operators' definitions in 64 bits, row by row on
the CPU, without the library."""
from __future__ import annotations

import math
import random

import torch

U64 = (1 << 64) - 1
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # torch.finfo(t).eps / 2


def signed(m: int) -> int:
    return m - (1 << 64) if m >> 63 else m


def tree_masks(n: int, rng: random.Random, spread: int = 6):
    """Ancestors-or-self masks of a random tree of n nodes, parents first."""
    m = []
    for i in range(n):
        m.append((m[rng.randint(max(0, i - spread), i - 1)] if i else 0) | (1 << i))
    return m


def chain_mask(i: int) -> int:
    return (1 << (i + 1)) - 1


class Case:
    """A paged cache with sequences of given lengths and trees, on the CPU, and its copy on the GPU."""

    def __init__(self, lens, nodes, heads, kv, dim, page, dtype, seed=0, layers=1, layout="head", masks="tree", extra=3,
                 spare=2):
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.lens, self.nodes, self.H, self.K, self.D, self.page, self.dtype = lens, nodes, heads, kv, dim, page, dtype
        need = [-(-(a + n) // page) for a, n in zip(lens, nodes)]
        pages = sum(need) + extra
        order = list(range(pages))
        rng.shuffle(order)
        self.table = torch.full((len(lens), max(need) + spare), -1, dtype=torch.int32)
        at = 0
        for s, m in enumerate(need):
            self.table[s, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
            at += m
        shape = {"head": (2, layers, pages, kv, page, dim), "token": (2, layers, pages, page, kv, dim),
                 "mixed": (layers, pages, page, 2, kv, dim)}[layout]
        buf = torch.randn(shape, generator=g).to(dtype)
        self.layout, self.buf = layout, buf
        self.k, self.v = self._views(buf)
        self.rows = sum(nodes)
        off = [0]
        for n in nodes:
            off.append(off[-1] + n)
        self.off = off
        if masks == "tree":
            self.masks = [m for n in nodes for m in tree_masks(n, rng)]
        elif masks == "chain":
            self.masks = None
        else:  # any bits, some rows none
            self.masks = [rng.getrandbits(64) & ((1 << n) - 1) if rng.random() < 0.8 else 0 for n in nodes for _ in range(n)]
        self.q = torch.randn(self.rows, heads, dim, generator=g).to(dtype)

    def _views(self, buf):
        if self.layout == "head":
            return buf[0], buf[1]
        if self.layout == "token":
            return buf[0].permute(0, 1, 3, 2, 4), buf[1].permute(0, 1, 3, 2, 4)
        return buf[:, :, :, 0].permute(0, 1, 3, 2, 4), buf[:, :, :, 1].permute(0, 1, 3, 2, 4)

    def mask(self, s, i):
        return chain_mask(i) if self.masks is None else self.masks[self.off[s] + i]

    def gpu(self, dfv, refs=None):
        k, v = self._views(self.buf.cuda())
        cache = dfv.KVCache(k, v, self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(),
                            refs=None if refs is None else refs.cuda())
        return cache, self.tree(dfv)

    def tree(self, dfv, max_nodes=None, seq=None):
        m = None if self.masks is None else torch.tensor([signed(x) for x in self.masks], dtype=torch.int64).cuda()
        return dfv.TreeBatch(torch.tensor(self.off, dtype=torch.int32).cuda(), self.rows, max_nodes or max(max(self.nodes), 1),
                             mask=m, seq=seq)

    def keys(self, s, upto, layer=0):
        """k and v [kv heads, upto, dim] of sequence s in 64 bits."""
        n = -(-upto // self.page)
        pg = self.table[s, :n].long()
        take = lambda x: x[layer][pg].permute(1, 0, 2, 3).reshape(self.K, n * self.page, self.D)[:, :upto].double()  # noqa: E731
        return take(self.k), take(self.v)

    def attention(self, scale=None, layer=0):
        """(o, lse, weighted |v|, largest scale * sum |q k|, keys) by the definition; what a row does not attend to is
        left out of its sums."""
        scale = self.D ** -0.5 if scale is None else scale
        o = torch.zeros(self.rows, self.H, self.D, dtype=torch.float64)
        a = torch.zeros_like(o)
        lse = torch.full((self.rows, self.H), -math.inf, dtype=torch.float64)
        big = torch.zeros(self.rows, self.H, dtype=torch.float64)
        G = self.H // self.K
        for s, n in enumerate(self.nodes):
            k, v = self.keys(s, self.lens[s] + n, layer)
            for i in range(n):
                m = self.mask(s, i)
                at = list(range(self.lens[s])) + [self.lens[s] + j for j in range(n) if m >> j & 1]
                if not at:
                    continue
                at = torch.tensor(at)
                r = self.off[s] + i
                for h in range(self.H):
                    q, kk, vv = self.q[r, h].double(), k[h // G, at], v[h // G, at]
                    x = scale * (kk @ q)
                    lse[r, h] = torch.logsumexp(x, 0)
                    p = torch.softmax(x, 0)
                    o[r, h], a[r, h] = p @ vv, p @ vv.abs()
                    big[r, h] = (scale * (kk.abs() @ q.abs())).max()
        return o, lse, a, big, max(l + n for l, n in zip(self.lens, self.nodes))

    def tolerances(self, o, lse, a, big, keys):
        """Output: half a step of the type for its rounding and one for the rounding of p (weighted by |v|), plus twice
        the fp32 errors of p: the dot product's D + 2 roundings of at most `big`, 2^-21 for exp2 and its argument's
        rounding at |x| <= 2 big, one rounding per key in the sums.  lse: the same fp32 errors once."""
        u = 2.0 ** -24
        f = (self.D + 2) * u * big + 2.0 ** -21 + 4 * u * big + (keys + 16) * u
        half = HALF_STEP[self.dtype]
        to = half * o.abs() + (half + 2 * f[..., None]) * a * (1 + half) + 1e-30
        if self.dtype == torch.float16:  # its subnormals: spacing 2^-24, for p and for the output
            to = to + 2.0 ** -25 * (1 + a)
        tl = f + 4 * u * torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse)) + 4 * u
        return to, tl
