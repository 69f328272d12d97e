"""Tree attention over a cache in e4m3 codes against the definition in 64 bits."""
from __future__ import annotations

import math
import random

import pytest
import torch

from tests._prompt_util import E4M3, coded, offsets, valued
from tests._tree_util import chain_mask, signed, tree_masks

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


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
    def __init__(self, lens, nodes, heads, kv, dim, page, seed=0, layers=1, layout="head", masks="tree", spread=0.5, extra=2, junk=None):
        """spread: how far tokens' sizes are apart (factors of e); junk: the byte of every code and exponent outside the tokens."""
        rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.lens, self.nodes, self.H, self.K, self.D, self.page, self.layout = lens, nodes, heads, kv, dim, page, layout
        need = [-(-(a + n) // page) for a, n in zip(lens, nodes)]
        pages = sum(need) + extra
        order = list(range(pages))
        rng.shuffle(order)
        self.table = torch.full((len(lens), max(need) + 2), -1, dtype=torch.int32)
        for s, m in enumerate(need):
            self.table[s, :m] = torch.tensor([order.pop() for _ in range(m)], dtype=torch.int32)
        self.raw, self.exp = [], []
        for _ in range(2):
            x = torch.randn(layers, pages, kv, page, dim, generator=g) * torch.exp(spread * torch.randn(layers, pages, kv, page, 1, generator=g))
            _, code, e = coded(x.double())
            self.raw.append(code.float().to(E4M3).view(torch.uint8))
            self.exp.append((e + 127).to(torch.uint8))
        if junk is not None:
            used = torch.zeros(pages, page, dtype=torch.bool)
            for s, (a, n) in enumerate(zip(lens, nodes)):
                at = torch.arange(a + n)
                used[self.table[s, at // page].long(), at % page] = True
            for x, e in zip(self.raw, self.exp):
                x[~used[None, :, None].expand(layers, pages, kv, page)] = junk
                e[~used[None, :, None].expand(layers, pages, kv, page)] = junk
        self.off = offsets(nodes)
        self.rows = max(self.off[-1], 1)
        if masks == "tree":
            self.masks = [m for n in nodes for m in tree_masks(n, rng)]
        elif masks == "chain":
            self.masks = None
        else:  # any bits, some rows none
            self.masks = [rng.getrandbits(64) & ((1 << n) - 1) if rng.random() < 0.8 else 0 for n in nodes for _ in range(n)]
        self.q = torch.randn(self.rows, heads, dim, generator=g).to(BF)

    def cache(self, dfv, raw=None):
        k, v = (x.cuda().view(E4M3) if self.layout == "head" else x.transpose(2, 3).contiguous().cuda().view(E4M3).transpose(2, 3) for x in (raw or self.raw))
        return dfv.KVCache(k, v, self.table.cuda(), i32(self.lens), k_exp=self.exp[0].cuda(), v_exp=self.exp[1].cuda())

    def tree(self, dfv, most=None):
        m = None if self.masks is None else torch.tensor([signed(x) for x in self.masks], dtype=torch.int64, device="cuda")
        return dfv.TreeBatch(i32(self.off), self.rows, most or max(max(self.nodes), 1), mask=m)

    def run(self, dfv, cache=None, layer=0, scale=None, q=None, most=None):
        cache, tree = cache or self.cache(dfv), self.tree(dfv, most)
        ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, self.H))
        lse = torch.full((self.rows, self.H), 7.0, device="cuda")
        out = dfv.tree_attention(cache, layer, tree, self.q.cuda() if q is None else q, ws, scale=scale, lse=lse)
        assert dfv.read_device_error(ws) == 0
        return out, lse, cache.errors()

    def want(self, layer=0, scale=None):
        """(o, lse, tolerance of o, of lse).  The output: half a step of bf16 for its rounding, half a step of fp16 for the
        weights' (weighted by |v|; the weights are at most 2^6, their subnormals' spacing 2^-24), and twice the fp32 errors:
        D + 2 roundings of the dot product of at most `big`, 2^-21 for exp2, four roundings of the score and the power at
        their sizes, one per key in the sums; q as fp16 is off by 2^-25 of its row's largest element at most."""
        scale = scale or self.D ** -0.5
        u, G = 2.0 ** -24, self.H // self.K
        o = torch.zeros(self.rows, self.H, self.D, dtype=torch.float64)
        to, lse, tl = o.clone(), torch.full((self.rows, self.H), -math.inf, dtype=torch.float64), torch.zeros(self.rows, self.H, dtype=torch.float64)
        for s, n in enumerate(self.nodes):
            T = self.lens[s] + n
            at = torch.arange(T)
            pg, tok = self.table[s, at // self.page].long(), at % self.page
            (k, kb), (v, vb) = ((x[layer, pg, :, tok].view(E4M3), e[layer, pg, :, tok]) for x, e in zip(self.raw, self.exp))
            vc = v.double()
            k, v = valued(k, kb), valued(v, vb)
            for i in range(n):
                m = chain_mask(i) if self.masks is None else self.masks[self.off[s] + i]
                see = torch.tensor([j for j in range(T) if j < self.lens[s] or m >> (j - self.lens[s]) & 1], dtype=torch.long)
                r = self.off[s] + i
                if not len(see):
                    continue
                for h in range(self.K):
                    q = self.q[r, h * G:(h + 1) * G].double()
                    x = scale * q @ k[see, h].T
                    lse[r, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                    p = torch.softmax(x, -1)
                    o[r, h * G:(h + 1) * G] = p @ v[see, h]
                    a = p @ v[see, h].abs()
                    big = (scale * q.abs() @ k[see, h].abs().T).amax(-1)
                    low = scale * 2.0 ** -25 * q.abs().amax(-1) * k[see, h].abs().sum(-1).amax()
                    b = vb[see, h].double() - 127
                    f = (self.D + 2) * u * big + 2.0 ** -21 + 4 * u * (2 * big + b.abs().amax()) + (len(see) + 16) * u + low
                    w = x / math.log(2) + b
                    w = torch.exp2(w - w.amax(-1, keepdim=True))
                    small = 2.0 ** -31 * vc[see, h].abs().sum(0)[None] / (w * torch.exp2(-b)).sum(-1)[:, None]
                    to[r, h * G:(h + 1) * G] = 2.0 ** -8 * o[r, h * G:(h + 1) * G].abs() + (2.0 ** -11 + 2 * f[:, None]) * a * (1 + 2.0 ** -8) + small + 1e-30
                    tl[r, h * G:(h + 1) * G] = f + 4 * u * lse[r, h * G:(h + 1) * G].abs() + 4 * u
        return o, lse, to, tl

    def check(self, dfv, **kw):
        out, lse, err = self.run(dfv, **kw)
        assert err == 0
        n = self.off[-1]
        o, L, to, tl = self.want(**{k: v for k, v in kw.items() if k in ("layer", "scale")})
        d = (out.double().cpu() - o).abs()[:n]
        assert bool((d <= to[:n]).all()), "output off by %g of its tolerance" % float((d / to[:n]).max())
        lse = lse.double().cpu()[:n]
        none = torch.isinf(L[:n])
        assert bool((lse[none] == -math.inf).all())
        d = (lse - L[:n]).abs()[~none]
        assert bool((d <= tl[:n][~none]).all()), "lse off by %g of its tolerance" % float((d / tl[:n][~none]).max())


LENGTHS = [([0], [1]), ([1], [1]), ([63], [1]), ([64], [1]), ([127], [2]), ([128], [1]), ([1000], [1]), ([5, 0, 300, 64], [1, 2, 0, 2]), ([9000], [2])]


@pytest.mark.parametrize("heads,kv,dim,page", [(8, 1, 128, 16), (8, 4, 64, 64), (7, 1, 128, 8), (3, 3, 64, 256), (4, 2, 64, 8), (10, 2, 128, 128)])
@pytest.mark.parametrize("lens,nodes", LENGTHS)
def test_few_rows(dfv, lens, nodes, heads, kv, dim, page):
    Case(lens, nodes, heads, kv, dim, page, seed=len(lens) + heads).check(dfv)


# rows per kv head from 17 (one row tile) to 64 x 16 (several CTAs a range)
@pytest.mark.parametrize("heads,kv,dim,page", [(8, 1, 128, 16), (4, 2, 64, 8), (7, 1, 128, 64), (16, 1, 64, 256), (2, 1, 128, 8)])
@pytest.mark.parametrize("lens,nodes", [([0], [17]), ([100], [16]), ([127, 0, 64], [33, 40, 1]), ([700], [64]), ([3000, 5], [20, 64]), ([129], [18])])
def test_many_rows(dfv, lens, nodes, heads, kv, dim, page):
    Case(lens, nodes, heads, kv, dim, page, seed=len(lens) + heads).check(dfv)


def test_many_rows_of_many_sequences(dfv):
    Case([(37 * s) % 300 for s in range(60)], [s % 33 for s in range(60)], 4, 2, 64, 16, seed=7).check(dfv)
    Case([(37 * s) % 300 for s in range(30)], [s % 65 for s in range(30)], 5, 1, 128, 32, seed=8).check(dfv)


@pytest.mark.parametrize("masks", ["chain", "any"])
@pytest.mark.parametrize("dim,heads,nodes", [(64, 4, 30), (128, 8, 40)])
def test_masks_of_many_rows(dfv, masks, dim, heads, nodes):
    Case([0, 70, 200, 13], [nodes, 5, 20, nodes], heads, 1, dim, 16, seed=4, masks=masks).check(dfv)


@pytest.mark.parametrize("masks", ["tree", "chain", "any"])
@pytest.mark.parametrize("dim", [64, 128])
def test_masks(dfv, masks, dim):
    Case([0, 70, 200, 13], [16, 5, 16, 7], 2, 2, dim, 16, seed=4, masks=masks).check(dfv)
    Case([0, 70, 200, 13], [2, 1, 2, 0], 8, 1, dim, 16, seed=5, masks=masks).check(dfv)


@pytest.mark.parametrize("layout", ["head", "token"])
def test_layouts_and_layers(dfv, layout):
    Case([100, 31], [3, 4], 8, 2, 128, 32, seed=6, layers=3, layout=layout).check(dfv, layer=2)
    Case([100, 31], [3, 4], 8, 2, 64, 8, seed=6, layers=2, layout=layout).check(dfv, layer=1)


def test_many_sequences(dfv):
    Case([(37 * s) % 300 for s in range(200)], [s % 3 for s in range(200)], 4, 2, 64, 16, seed=7).check(dfv)


@pytest.mark.parametrize("spread,size,scale", [(3.0, 1.0, None), (8.0, 1.0, 1e-4), (0.5, 30.0, None), (0.5, 1e-20, None), (0.1, 1.0, 1.0)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nodes", [2, 16, 40])
def test_sizes_far_apart(dfv, dim, spread, size, scale, nodes):
    """Tokens whose powers differ by a lot, large and tiny queries: the weights of the product follow p times the power."""
    c = Case([700], [nodes], 8, 1, dim, 16, seed=8, spread=spread)
    c.q = (c.q.float() * size).to(BF)
    c.check(dfv, scale=scale)


@pytest.mark.parametrize("nodes", [2, 9, 50])
def test_a_query_of_zeros_and_one_large_element(dfv, nodes):
    c = Case([300], [nodes], 4, 1, 128, 16, seed=9)
    c.q[0] = 0
    c.q[1, :, 5] = 300.0
    c.check(dfv)


@pytest.mark.parametrize("heads,nodes", [(8, 2), (8, 9), (8, 40)])
@pytest.mark.parametrize("dim", [64, 128])
def test_what_is_masked_does_not_count(dfv, dim, heads, nodes):
    """Codes of NaN and exponent bytes of any value outside the tokens, and NaN in nodes that a row does not see."""
    lens = [200, 61]
    was = None
    for junk in (0, 255, 127, 128):
        c = Case(lens, [nodes, nodes], heads, 1, dim, 16, seed=10, junk=junk)
        out, lse, err = c.run(dfv)
        assert err == 0 and bool(torch.isfinite(out).all())
        assert was is None or (torch.equal(out, was[0]) and torch.equal(lse, was[1]))
        was = (out, lse)
    c = Case(lens, [nodes, nodes], heads, 1, dim, 16, seed=10, junk=0, masks="chain")
    out, lse, _ = c.run(dfv)
    raw = [x.clone() for x in c.raw]
    at = lens[0] + nodes - 1  # the last node of the first tree: seen by its own row only
    for x in raw:
        x[0, int(c.table[0, at // 16]), 0, at % 16, 3] = 0x7f
    got, lse2, _ = c.run(dfv, cache=c.cache(dfv, raw))
    keep = torch.ones(c.rows, dtype=torch.bool)
    keep[nodes - 1] = False
    assert torch.equal(got[keep.cuda()], out[keep.cuda()]) and torch.equal(lse2[keep.cuda()], lse[keep.cuda()])
    assert bool(torch.isnan(got[nodes - 1]).all())  # its key is NaN
    raw[0] = c.raw[0]
    got, lse2, _ = c.run(dfv, cache=c.cache(dfv, raw))
    assert torch.equal(got[keep.cuda()], out[keep.cuda()]) and torch.equal(lse2, lse)
    bad = torch.isnan(got[nodes - 1])
    assert bool(bad[:, 3].all()) and int(bad.sum()) == heads


@pytest.mark.parametrize("nodes", [2, 12, 64])
def test_nan_in_a_committed_token(dfv, nodes):
    c = Case([200], [nodes], 4, 2, 64, 16, seed=11)
    c.raw[1][0, int(c.table[0, 3]), 1, 7, 9] = 0xff
    out, _, err = c.run(dfv)
    bad = torch.isnan(out)
    assert err == 0 and bool(bad[:, 2:, 9].all()) and int(bad.sum()) == 2 * nodes


@pytest.mark.parametrize("nodes", [2, 20])
def test_missing_pages_and_bad_lengths(dfv, nodes):
    c = Case([100, 50], [nodes, 2], 4, 2, 64, 16, seed=12)
    was, _, _ = c.run(dfv)
    cache = c.cache(dfv)
    cache.page_table[0, 2] = -1
    out, _, err = c.run(dfv, cache=cache)
    assert err == dfv.KVERR_PAGE and torch.equal(out[nodes:], was[nodes:])
    cache = c.cache(dfv)
    cache.lens[0] = 1 << 20
    out, _, err = c.run(dfv, cache=cache)
    assert err == dfv.KVERR_LEN and torch.equal(out[nodes:], was[nodes:]) and not bool(out[:nodes].any())


@pytest.mark.parametrize("nodes", [2, 16, 33])
def test_the_same_bits_every_time_and_in_a_graph(dfv, nodes):
    c = Case([3000, 20], [nodes, 1], 8, 1, 128, 16, seed=13)
    cache, tree = c.cache(dfv), c.tree(dfv)
    ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, 8))
    q = c.q.cuda()
    was = dfv.tree_attention(cache, 0, tree, q, ws)
    out = torch.zeros_like(was)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dfv.tree_attention(cache, 0, tree, q, ws, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, was)
    cache.lens.copy_(i32([1000, 12]))
    g.replay()
    assert torch.equal(out, dfv.tree_attention(cache, 0, tree, q, ws))


@pytest.mark.parametrize("nodes", [2, 30])
def test_as_a_bf16_cache_of_the_same_values(dfv, nodes):
    """The values of codes fit bf16: both caches give the same attention but for the roundings of p."""
    c = Case([500, 77], [nodes, 1], 8, 2, 128, 16, seed=14)
    cache = c.cache(dfv)
    k, v = (valued(x.view(E4M3), e).to(BF).cuda() for x, e in zip(c.raw, c.exp))
    other = dfv.KVCache(k, v, c.table.cuda(), i32(c.lens))
    a, _, _ = c.run(dfv, cache=cache)
    b, _, _ = c.run(dfv, cache=other)
    o, _, to, _ = c.want()
    assert bool(((a.double() - b.double()).abs().cpu() <= 2 * to + 2.0 ** -8 * o.abs().amax()).all())
