"""Norms per head, rotary positions and the append of any number of rows, to caches in 16 bits and in codes, against the
formulas in 64 bits; and what cache_read brings back."""
from __future__ import annotations

import math
import random

import pytest
import torch

from tests._prompt_util import E4M3, HALF_STEP, coded, offsets, valued

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """Sequences with lens[s] tokens that get rows[s] more, in a paged cache of `kind` (bf16, fp16 or codes)."""

    def __init__(self, lens, rows, heads, kv, dim, page, kind, seed=0, layers=1, layout="head", lead=0, tail=0, norm=True, size=1.0):
        rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.lens, self.rows, self.H, self.K, self.D, self.page, self.kind, self.layers = lens, rows, heads, kv, dim, page, kind, layers
        self.dt = BF if kind == E4M3 else kind
        need = [-(-(a + n) // page) for a, n in zip(lens, rows)]
        pages = sum(need) + 2
        order = list(range(pages))
        rng.shuffle(order)
        self.table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
        for s, m in enumerate(need):
            self.table[s, :m] = torch.tensor([order.pop() for _ in range(m)], dtype=torch.int32)
        shape = (layers, pages, kv, page, dim) if layout == "head" else (layers, pages, page, kv, dim)
        self.k, self.v = (torch.randn(shape, generator=g).to(kind) for _ in range(2))
        if layout != "head":
            self.k, self.v = self.k.transpose(2, 3), self.v.transpose(2, 3)
        self.exp = [torch.randint(100, 150, (layers, pages, kv, page), generator=g).to(torch.uint8) if kind == E4M3 else None for _ in range(2)]
        self.off = offsets(rows, lead)
        self.n = max(self.off[-1] + tail, 1)
        self.qkv = (size * torch.randn(self.n, heads + 2 * kv, dim, generator=g)).to(self.dt)
        self.gains = [(1 + 0.3 * torch.randn(dim, generator=g)).to(self.dt) if norm else None for _ in range(2)]
        self.positions = torch.zeros(self.n, dtype=torch.int32)
        for s, n in enumerate(rows):
            self.positions[self.off[s]:self.off[s + 1]] = torch.arange(lens[s], lens[s] + n, dtype=torch.int32)

    def cache(self, dfv):
        dev = [x if x is None else x.cuda() for x in self.exp]
        keep = lambda x: x.cuda() if x.is_contiguous() else x.transpose(2, 3).contiguous().cuda().transpose(2, 3)  # noqa: E731
        return dfv.KVCache(keep(self.k), keep(self.v), self.table.cuda(), i32(self.lens), k_exp=dev[0], v_exp=dev[1])

    def split(self, x):
        return x[:, :self.H], x[:, self.H:self.H + self.K], x[:, self.H + self.K:]

    def want(self, freqs, inter, scale=1.0, eps=EPS):
        """(y, t): every head normed and turned in 64 bits, and the fp32 error.  The norm: D + 2 roundings of the sum of
        squares, two of the mean and eps, halved by the root, 2^-22 for the root itself, two products.  The rotation: the
        angle off by 2 pi (2^-32 + 2^-25) and by position * 2^-50 for the table, sine and cosine by 2 units, three
        roundings."""
        x = self.qkv.double()
        off = torch.zeros_like(x)
        for heads, gain in ((slice(0, self.H), self.gains[0]), (slice(self.H, self.H + self.K), self.gains[1])):
            if gain is not None:
                z = x[:, heads]
                x[:, heads] = z / torch.sqrt(z.square().mean(-1, keepdim=True) + eps) * gain.double()
                off[:, heads] = x[:, heads].abs() * ((0.5 * (self.D + 4) + 3) * U + 2.0 ** -22)
        y, t = x.clone(), off.clone()
        r, HK = 2 * len(freqs), self.H + self.K
        for m, f in enumerate(freqs):
            a, b = (2 * m, 2 * m + 1) if inter else (m, m + r // 2)
            ang = self.positions.double() * f
            c, s = torch.cos(ang)[:, None] * scale, torch.sin(ang)[:, None] * scale
            u, w = x[:, :HK, a], x[:, :HK, b]
            y[:, :HK, a], y[:, :HK, b] = u * c - w * s, w * c + u * s
            far = self.positions.double().abs()[:, None] * 2.0 ** -50
            err = (u.abs() + w.abs()) * abs(scale) * (2 * math.pi * (2.0 ** -32 + 2.0 ** -25) + far + 8 * U) + (off[:, :HK, a] + off[:, :HK, b]) * abs(scale)
            t[:, :HK, a] = t[:, :HK, b] = err
        return y, t

    def run(self, dfv, cache, rot=None, theta=1e4, inter=False, layer=0, in_place=False, scale=None, eps=EPS, seq=None, most=None, **kw):
        rope = dfv.Rope(self.D, rot_dim=rot, theta=theta, interleaved=inter, scale=scale)
        rows = dfv.RowBatch(i32(self.off), self.n, most or max(max(self.rows), 1), seq=seq)
        dev = self.qkv.cuda()
        q, k, v = self.split(dev)
        g = [x if x is None else x.cuda() for x in self.gains]
        out = q if in_place else torch.full((self.n, self.H, self.D), 5.0, dtype=self.dt, device="cuda")
        dfv.norm_rope_append(cache, layer, rows, rope, q, k, v, self.positions.cuda(), q_gain=g[0], k_gain=g[1], eps=eps, out=out, **kw)
        r = rot or self.D
        return out, self.want([theta ** (-2 * i / r) for i in range(r // 2)], inter, scale or 1.0, eps)

    def check(self, cache, out, want, layer=0, stored=lambda s, i: True):
        y, t = want
        r0, r1 = self.off[0], self.off[-1]
        half = HALF_STEP[self.dt]
        small = 2.0 ** -25 if self.dt == HF else 1e-40
        d = (out.double().cpu() - y[:, :self.H]).abs()
        tol = t[:, :self.H] + half * (y[:, :self.H].abs() + t[:, :self.H]) + small
        assert bool((d <= tol)[r0:r1].all()), float((d / tol)[r0:r1].max())
        now = [(cache.k, cache.k_exp, self.k, self.exp[0], slice(self.H, self.H + self.K)),
               (cache.v, cache.v_exp, self.v, self.exp[1], slice(self.H + self.K, None))]
        for x, e, x0, e0, heads in now:
            x, x0 = x.cpu().clone(), x0.clone()
            raw = torch.uint8 if self.kind == E4M3 else torch.int16
            e = None if e is None else e.cpu().clone()
            e0 = None if e0 is None else e0.clone()
            for s, n in enumerate(self.rows):
                for i in range(n):
                    if not stored(s, i):
                        continue
                    r, at = self.off[s] + i, self.lens[s] + i
                    pg, tok = int(self.table[s, at // self.page]), at % self.page
                    w, tt = y[r, heads], t[r, heads]
                    got = x[layer, pg, :, tok]
                    if self.kind == E4M3:
                        b = e[layer, pg, :, tok].double() - 127
                        top, tops = w.abs().amax(-1), tt.amax(-1)
                        assert bool((448 * torch.exp2(b) >= top - tops).all())
                        assert bool(((448 * torch.exp2(b - 1) < top + tops) | (b == -100)).all())
                        z = (w.abs() + tt) * torch.exp2(-b)[:, None]
                        step = torch.exp2(torch.floor(torch.log2(z.clamp_min(2.0 ** -6))) - 3 + b[:, None])
                        assert bool(((valued(got, e[layer, pg, :, tok]) - w).abs() <= tt + step / 2).all())
                        e[layer, pg, :, tok] = e0[layer, pg, :, tok] = 0
                    else:
                        assert bool(((got.double() - w).abs() <= tt + half * (w.abs() + tt) + small).all())
                    x.view(raw)[layer, pg, :, tok] = 0
                    x0.view(raw)[layer, pg, :, tok] = 0
            assert torch.equal(x.view(raw), x0.view(raw)), "rows of the cache that nobody wrote"
            assert e is None or torch.equal(e, e0)


KINDS = [BF, HF, E4M3]


def same(a, b):
    """Equal values, NaN being equal to NaN."""
    return a.shape == b.shape and bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 96), (256, 256), (16, 16), (80, 48), (192, 64)])
@pytest.mark.parametrize("inter", [False, True])
def test_layouts_and_partial_heads(dfv, kind, dim, rot, inter):
    c = Case([30, 0, 16, 7], [5, 1, 0, 70], 6, 2, dim, 16, kind, seed=dim + rot)
    cache = c.cache(dfv)
    out, want = c.run(dfv, cache, rot=rot, inter=inter)
    c.check(cache, out, want)
    assert cache.errors() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gains", [(False, False), (True, False), (False, True)])
def test_gains_of_one_side_or_none(dfv, kind, gains):
    c = Case([3], [20], 4, 2, 128, 16, kind, seed=1)
    c.gains = [g if on else None for g, on in zip(c.gains, gains)]
    cache = c.cache(dfv)
    c.check(cache, *c.run(dfv, cache))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("page", [8, 64, 256])
def test_pages_and_strides(dfv, kind, layout, page):
    c = Case([page - 1, page, 0, 2 * page - 3], [2 * page + 5, 1, page, 0], 3, 3, 64, page, kind, seed=5, layers=2, layout=layout)
    cache = c.cache(dfv)
    c.check(cache, *c.run(dfv, cache, layer=1), layer=1)


@pytest.mark.parametrize("kind", KINDS)
def test_in_place_and_rows_of_nobody(dfv, kind):
    c = Case([7, 70], [90, 5], 8, 2, 128, 16, kind, seed=6, lead=3, tail=4)
    cache = c.cache(dfv)
    out, want = c.run(dfv, cache)
    assert bool((out[:3] == 5).all()) and bool((out[-4:] == 5).all())
    c.check(cache, out, want)
    again = c.cache(dfv)
    got, _ = c.run(dfv, again, in_place=True)
    assert torch.equal(got[3:-4], out[3:-4])
    assert torch.equal(got[:3].cpu(), c.qkv[:3, :8]) and torch.equal(got[-4:].cpu(), c.qkv[-4:, :8])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("inter", [False, True])
def test_turned_keys_as_rows(dfv, kind, inter):
    c = Case([7, 70], [90, 5], 4, 2, 128, 16, kind, seed=16, lead=3, tail=4)
    cache = c.cache(dfv)
    ko = torch.full((c.n, 3, 128), 5.0, dtype=c.dt, device="cuda")
    cache.page_table[0, 2] = -1  # tokens without a page have their rows all the same
    out, (y, t) = c.run(dfv, cache, inter=inter, k_out=ko[:, :2])
    got, want, t = ko[3:-4, :2].double().cpu(), y[3:-4, 4:6], t[3:-4, 4:6]
    assert bool(((got - want).abs() <= t + HALF_STEP[c.dt] * (want.abs() + t) + 2.0 ** -25).all())
    assert bool((ko[:3] == 5).all()) and bool((ko[-4:] == 5).all()) and bool((ko[:, 2] == 5).all())
    q, k, v = c.split(c.qkv.cuda())  # into k itself
    rows, g = dfv.RowBatch(i32(c.off), c.n, 90), [x.cuda() for x in c.gains]
    dfv.norm_rope_append(cache, 0, rows, dfv.Rope(128, interleaved=inter), q, k, v, c.positions.cuda(), q_gain=g[0], k_gain=g[1], k_out=k)
    assert torch.equal(k[3:-4], ko[3:-4, :2]) and torch.equal(k[:3].cpu(), c.qkv[:3, 4:6])


@pytest.mark.parametrize("kind", KINDS)
def test_many_rows_and_sequences(dfv, kind):
    c = Case([(5 * s) % 33 for s in range(400)], [(3 * s) % 7 for s in range(400)], 2, 1, 64, 8, kind, seed=7)
    cache = c.cache(dfv)
    c.check(cache, *c.run(dfv, cache, theta=1e6))
    c = Case([10], [1500], 5, 1, 64, 32, kind, seed=8, norm=False)
    cache = c.cache(dfv)
    c.check(cache, *c.run(dfv, cache, inter=True, rot=32))


@pytest.mark.parametrize("kind", KINDS)
def test_scale_eps_and_zero_rows(dfv, kind):
    c = Case([4], [6], 4, 2, 64, 16, kind, seed=9)
    c.qkv[2] = 0
    c.qkv[3] *= 1e-3
    cache = c.cache(dfv)
    c.check(cache, *c.run(dfv, cache, scale=1.25, eps=0.5, rot=32))


def test_codes_of_every_size(dfv):
    """Values from the smallest to the largest of bf16, rows of zeros, and maxima at and next to the borders of the powers."""
    c = Case([0], [300], 1, 1, 64, 16, E4M3, seed=10, norm=False)
    v = c.qkv[:, 2]
    v *= torch.exp2(torch.linspace(-133, 127, 300))[:, None].to(BF)
    v[0] = 0
    v[1], v[1, 5] = 0, 448.0
    v[2], v[2, 5] = 0, 450.0  # the next above in bf16
    v[3], v[3, 5] = 0, -3.389e38
    cache = c.cache(dfv)
    c.run(dfv, cache)
    val, code, e = coded(v.double())
    rows = dfv.RowBatch(i32([0, 300]), 300, 300)
    _, back = dfv.cache_read(cache, 0, rows)
    for i in range(300):
        pg = int(c.table[0, i // 16])
        assert int(cache.v_exp[0, pg, 0, i % 16]) == int(e[i]) + 127
        assert same(cache.v[0, pg, 0, i % 16].double().cpu(), code[i])
        assert same(back[i, 0].cpu(), val[i].to(BF))


def test_codes_of_what_is_not_finite(dfv):
    c = Case([0], [4], 1, 1, 64, 16, E4M3, seed=11, norm=False)
    v = c.qkv[:, 2]
    v[0, 3], v[1, 4], v[2, 5] = float("nan"), float("inf"), -float("inf")
    v[3] = float("inf")
    cache = c.cache(dfv)
    c.run(dfv, cache)
    _, back = dfv.cache_read(cache, 0, dfv.RowBatch(i32([0, 4]), 4, 4))
    back = back[:, 0].double().cpu()
    bad = ~torch.isfinite(v.double())
    assert torch.equal(torch.isnan(back), bad)
    want, _, _ = coded(torch.where(bad, torch.zeros(()).double(), v.double()))
    assert torch.equal(back[~bad], want[~bad])
    assert cache.errors() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_missing_pages_and_bad_lengths(dfv, kind):
    c = Case([14, 30], [40, 3], 2, 1, 64, 16, kind, seed=12)
    cache = c.cache(dfv)
    cache.page_table[0, 1] = -1  # tokens 16..31 of the first sequence
    c.check(cache, *c.run(dfv, cache), stored=lambda s, i: s == 1 or i < 2 or i >= 18)
    assert cache.errors() == dfv.KVERR_PAGE
    for bad in (-1, 1 << 20, 2 ** 31 - 1):
        cache = c.cache(dfv)
        cache.lens[0] = bad
        c.check(cache, *c.run(dfv, cache), stored=lambda s, i: s == 1)
        assert cache.errors() == dfv.KVERR_LEN
    cache = c.cache(dfv)
    c.check(cache, *c.run(dfv, cache, seq=i32([2, 1])), stored=lambda s, i: s == 1)
    assert cache.errors() == dfv.KVERR_SEQ
    # more rows than the call said: none of that sequence
    cache = c.cache(dfv)
    out, want = c.run(dfv, cache, most=39)
    assert cache.errors() == dfv.KVERR_LEN and bool((out[:40] == 5).all())
    assert torch.equal(out[40:], c.run(dfv, c.cache(dfv))[0][40:])


@pytest.mark.parametrize("dtype", [BF, HF, E4M3])
def test_rope_append_of_trees(dfv, dtype):
    """The drafted rows of a tree go into a cache in codes as the same rows do as a batch; into the others as before."""
    c = Case([30, 5], [7, 64], 4, 2, 64, 16, dtype, seed=13, norm=False)
    cache, other = c.cache(dfv), c.cache(dfv)
    out, _ = c.run(dfv, cache)
    q, k, v = c.split(c.qkv.cuda())
    tree = dfv.TreeBatch(i32(c.off), c.n, 64)
    got = dfv.rope_append(other, 0, tree, dfv.Rope(64), q, k, v, c.positions.cuda())
    if dtype == E4M3:
        assert torch.equal(got, out)
        assert torch.equal(cache.k.view(torch.uint8), other.k.view(torch.uint8)) and torch.equal(cache.k_exp, other.k_exp)
        assert torch.equal(cache.v.view(torch.uint8), other.v.view(torch.uint8)) and torch.equal(cache.v_exp, other.v_exp)
    else:
        assert float((got.double() - out.double()).abs().max()) <= 2 * HALF_STEP[dtype] * float(out.double().abs().max())


def test_a_captured_call(dfv):
    c = Case([9, 100], [50, 3], 8, 2, 128, 16, E4M3, seed=14)
    cache = c.cache(dfv)
    out, want = c.run(dfv, cache)
    k, e = cache.k.view(torch.uint8).clone(), cache.k_exp.clone()
    other = c.cache(dfv)
    rope, rows = dfv.Rope(128), dfv.RowBatch(i32(c.off), c.n, 50)
    dev, pos, g = c.qkv.cuda(), c.positions.cuda(), [x.cuda() for x in c.gains]
    q, kk, v = c.split(dev)
    got = torch.zeros_like(out)
    dfv.norm_rope_append(c.cache(dfv), 0, rows, rope, q, kk, v, pos, q_gain=g[0], k_gain=g[1], out=got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dfv.norm_rope_append(other, 0, rows, rope, q, kk, v, pos, q_gain=g[0], k_gain=g[1], out=got)
    got.zero_()
    graph.replay()
    assert torch.equal(got, out) and torch.equal(other.k.view(torch.uint8), k) and torch.equal(other.k_exp, e)


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,kv,page,layout", [(128, 4, 16, "head"), (64, 8, 64, "token"), (16, 1, 8, "head"), (80, 3, 32, "head"), (256, 2, 256, "token")])
def test_read(dfv, kind, dim, kv, page, layout):
    c = Case([90, 0, page, 300], [0, 0, 0, 0], 1, kv, dim, page, kind, seed=dim, layers=2, layout=layout)
    cache = c.cache(dfv)
    seqs, counts = [3, 0, 1, 2], [299, 90, 0, 1]
    off = offsets(counts, 2)
    n = off[-1] + 3
    k, v = (torch.full((n, kv, dim), 5.0, dtype=c.dt, device="cuda") for _ in range(2))
    dfv.cache_read(cache, 1, dfv.RowBatch(i32(off), n, 299, seq=i32(seqs)), k=k, v=v)
    for got, x, e in ((k, c.k, c.exp[0]), (v, c.v, c.exp[1])):
        got = got.cpu()
        assert bool((got[:2] == 5).all()) and bool((got[-3:] == 5).all())
        for b, s in enumerate(seqs):
            at = torch.arange(counts[b])
            pg, tok = c.table[s, at // page].long(), at % page
            want = x[1].double()[pg, :, tok] if e is None else valued(x[1].double()[pg, :, tok], e[1][pg, :, tok])
            assert torch.equal(got[off[b]:off[b + 1]].double(), want.to(c.dt).double())
    assert cache.errors() == 0


def test_read_strided_rows_missing_pages_and_bad_offsets(dfv):
    c = Case([60, 20], [0, 0], 1, 2, 64, 16, E4M3, seed=2)
    cache = c.cache(dfv)
    rows = dfv.RowBatch(i32([0, 60, 80]), 80, 60)
    k, v = dfv.cache_read(cache, 0, rows)
    both = torch.zeros(80, 2, 2, 64, dtype=BF, device="cuda")
    dfv.cache_read(cache, 0, rows, k=both[:, 0], v=both[:, 1])
    assert torch.equal(both[:, 0], k) and torch.equal(both[:, 1], v)
    cache.page_table[0, 1] = -1
    k2, v2 = dfv.cache_read(cache, 0, rows)
    assert cache.errors() == dfv.KVERR_PAGE
    assert not bool(k2[16:32].any()) and not bool(v2[16:32].any())
    k[16:32], v[16:32] = 0, 0
    assert torch.equal(k2, k) and torch.equal(v2, v)
    cache.err.zero_()
    width = cache.page_table.shape[1] * 16  # tokens that the table has room for
    long = dfv.RowBatch(i32([0, width + 7]), width + 7, width + 7, seq=i32([1]))
    k3, _ = dfv.cache_read(cache, 0, long)
    assert cache.errors() & dfv.KVERR_LEN and not bool(k3[32:].any())
    for off in ([0, 90, 80], [-1, 60, 80], [0, 61, 80]):
        cache.err.zero_()
        dfv.cache_read(cache, 0, dfv.RowBatch(i32(off), 80, 60))
        assert cache.errors() & dfv.KVERR_LEN
    cache.err.zero_()
    k4, _ = dfv.cache_read(cache, 0, dfv.RowBatch(i32([0, 60, 80]), 80, 60, seq=i32([0, 2])))
    assert cache.errors() & dfv.KVERR_SEQ and not bool(k4[60:].any())
