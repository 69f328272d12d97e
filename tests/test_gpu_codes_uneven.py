"""Tree attention over codes where some tokens that every row sees are much larger than the others and have next to no weight:
what they do not weigh they must not cost either."""
from __future__ import annotations

import math

import pytest
import torch

from tests._prompt_util import E4M3, coded, valued
from tests.test_gpu_tree_attention_codes import Case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


def want(c, s):
    """(o, lse, tolerance of o, of lse) of sequence s's rows by the definition, chains of nodes.  Key j's weight is off by e_j:
    D + 2 roundings of the dot product at its own size, q as fp16 (2^-25 of the row's largest element), four roundings of
    x + b - M, 2^-21 for exp2.  The weights are rounded at 2^-11 of themselves, and at 2^-25 where they are subnormal: the
    largest is 2^(6 - 8) at least, M being at most 8 above the largest x + b.  The sums add a rounding a key, and the output its own 2^-8."""
    T, n, G = c.lens[s] + c.nodes[s], c.nodes[s], c.H // c.K
    at = torch.arange(T)
    pg, tok = c.table[s, at // c.page].long(), at % c.page
    (k, _), (v, vb) = ((x[0, pg, :, tok].view(E4M3), e[0, pg, :, tok]) for x, e in zip(c.raw, c.exp))
    code, b = v.double(), vb.double() - 127
    k, v = valued(k, _), valued(v, vb)
    scale = c.D ** -0.5
    hidden = torch.arange(T)[None, :] > c.lens[s] + torch.arange(n)[:, None]  # [node, key]
    o, lse, to, tl = [], [], [], []
    for h in range(c.K):
        q = c.q[c.off[s]:c.off[s + 1], h * G:(h + 1) * G].double()  # [node, head, dim]
        x = scale * q @ k[:, h].T
        x.masked_fill_(hidden[:, None], -math.inf)
        p = torch.softmax(x, -1)
        w = x / math.log(2) + b[:, h]
        top = w.amax(-1, keepdim=True)
        big = scale * q.abs() @ k[:, h].abs().T
        e = (c.D + 4) * U * big + scale * 2.0 ** -25 * q.abs().amax(-1, keepdim=True) * k[:, h].abs().sum(-1) + 2.0 ** -21 \
            + 4 * U * (2 * big + b[:, h].abs() + top.abs()) + (T + 16) * U
        y = p @ v[:, h]
        pe = (p * e).sum(-1, keepdim=True)
        small = 2.0 ** -23 * code[:, h].abs().sum(0) / (torch.exp2(w - top) * torch.exp2(-b[:, h])).sum(-1, keepdim=True)
        o.append(y)
        lse.append(torch.logsumexp(x, -1))
        to.append(2.0 ** -8 * y.abs() + 1.1 * ((p * (2.0 ** -11 + e)) @ v[:, h].abs() + y.abs() * pe) + small + 1e-30)
        tl.append(1.1 * pe[..., 0] + 4 * U * lse[-1].abs() + 4 * U)
    return [torch.cat(z, 1) for z in (o, lse, to, tl)]


def put(c, side, s, at, x):
    """Token `at` of sequence s becomes x [kv heads, dim]."""
    _, code, e = coded(x.double())
    pg, tok = int(c.table[s, at // c.page]), at % c.page
    c.raw[side][0, pg, :, tok] = code.float().to(E4M3).view(torch.uint8)
    c.exp[side][0, pg, :, tok] = (e + 127).to(torch.uint8)


# every row's query points at +4 of the first element, so a key of -size there has a score of -4 size / sqrt(D)
@pytest.mark.parametrize("heads,kv,dim,nodes", [(16, 2, 128, 16), (16, 2, 128, 25), (8, 4, 64, 20), (8, 4, 64, 3), (16, 2, 128, 2)])
@pytest.mark.parametrize("what,up", [("value", 5), ("value", 8), ("value", 10), ("value", 18), ("value", 24), ("value", 40), ("value", 100), ("key", 12),
                                     ("key", 20), ("key", 30), ("key", 90), ("both", 20), ("both", 40)])
def test_large_tokens_of_no_weight(dfv, what, up, heads, kv, dim, nodes):
    lens = [1500 + 100 * s for s in range(20)]
    c = Case(lens, [nodes] * len(lens), heads, kv, dim, 16, seed=up, masks="chain", spread=0.3)
    c.q[:, :, 0] = 4.0
    g = torch.Generator().manual_seed(1)
    size = 30 * math.sqrt(dim)  # a score of -120
    for s, n in enumerate(lens):
        for at in range(s % 7 + 3, n, 300):  # a tile in two or three
            x = torch.randn(kv, dim, generator=g)
            k = 0.1 * x
            k[:, 0] = -size
            if what in ("key", "both"):
                k[:, 0] = -float(2 ** up) * math.sqrt(dim)
            put(c, 0, s, at, k)
            if what in ("value", "both"):
                put(c, 1, s, at, x * 2.0 ** up)
    out, lse, err = c.run(dfv)
    assert err == 0
    for s in (0, 7, 12, 19):
        o, L, to, tl = want(c, s)
        r = slice(c.off[s], c.off[s + 1])
        d = (out[r].double().cpu() - o).abs()
        assert bool((d <= to).all()), "output off by %g of its tolerance" % float((d / to).max())
        d = (lse[r].double().cpu() - L).abs()
        assert bool((d <= tl).all()), "lse off by %g of its tolerance" % float((d / tl).max())
        # the tolerance is that of ordinary values: 2^-8 of the output, and 2^-11 of sum p |v|, which over n <= 3425 keys with
        # values of any sign is sqrt(n) = 59 times the output or less: 0.004 + 1.1 * 59 / 2048 = 0.036
        assert float((to / (o.abs() + 0.01 * o.abs().mean())).median()) < 2.0 ** -4


@pytest.mark.parametrize("heads,kv,dim,nodes", [(16, 2, 128, 16), (16, 2, 128, 25), (8, 4, 64, 20)])
@pytest.mark.parametrize("side,apart", [(0, n) for n in (14, 15, 16)] + [(1, n) for n in (7, 8, 9)])
def test_where_constants_of_a_tile_end(dfv, side, apart, heads, kv, dim, nodes):
    """Powers of a tile just as far apart as constants of the tile may be, or one further: tokens of weight at both ends."""
    lens = [1500 + 100 * s for s in range(20)]
    c = Case(lens, [nodes] * len(lens), heads, kv, dim, 16, seed=apart, masks="chain", spread=0.0)
    g = torch.Generator().manual_seed(2)
    e = c.exp[side]
    e.fill_(127 - 8 - apart)
    e[torch.rand(e.shape, generator=g) < 0.2] = 127 - 8
    if side == 0:
        c.q *= 0.25  # large keys do not take all weight
    out, lse, err = c.run(dfv)
    assert err == 0
    for s in (0, 7, 12, 19):
        o, L, to, tl = want(c, s)
        r = slice(c.off[s], c.off[s + 1])
        d = (out[r].double().cpu() - o).abs()
        assert bool((d <= to).all()), "output off by %g of its tolerance" % float((d / to).max())
        d = (lse[r].double().cpu() - L).abs()
        assert bool((d <= tl).all()), "lse off by %g of its tolerance" % float((d / tl).max())


@pytest.mark.parametrize("heads,kv,dim,nodes", [(16, 2, 128, 16), (16, 2, 128, 25), (8, 4, 64, 3), (16, 2, 128, 2)])
@pytest.mark.parametrize("low,high", [(-100, -8), (-100, 10), (-60, 50), (-5, 105)])
def test_values_far_apart_that_all_weigh(dfv, low, high, heads, kv, dim, nodes):
    """Values of two sizes 2^92 to 2^110 apart (zeros have the lowest power) with weights alike: the sum of the weights has them all."""
    lens = [1500 + 100 * s for s in range(20)]
    c = Case(lens, [nodes] * len(lens), heads, kv, dim, 16, seed=nodes, masks="chain", spread=0.0)
    g = torch.Generator().manual_seed(3)
    e = c.exp[1]
    e.fill_(127 + low)
    if low == -100:
        c.raw[1].zero_()
    large = torch.rand(e.shape, generator=g) < 0.3
    e[large] = 127 + high
    c.raw[1][large] = torch.randint(0x40, 0x7e, (int(large.sum()), dim), generator=g).to(torch.uint8)
    out, lse, err = c.run(dfv)
    assert err == 0
    for s in (0, 7, 12, 19):
        o, L, to, tl = want(c, s)
        r = slice(c.off[s], c.off[s + 1])
        d = (out[r].double().cpu() - o).abs()
        assert bool((d <= to).all()), "output off by %g of its tolerance" % float((d / to).max())
        d = (lse[r].double().cpu() - L).abs()
        assert bool((d <= tl).all()), "lse off by %g of its tolerance" % float((d / tl).max())
