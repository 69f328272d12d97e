"""Tree attention over the paged cache against its definition in 64 bits: head layouts, lengths from none to long,
page sizes, cache strides, masks (also ones that leave a row empty), what masked places hold, bad tables."""
from __future__ import annotations

import math
import random

import pytest
import torch

from tests._tree_util import Case, signed

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


def run(dfv, c: Case, cache=None, tree=None, q=None, **kw):
    if cache is None:
        cache, tree = c.gpu(dfv)
    ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, c.H))
    q = c.q.cuda() if q is None else q
    lse = torch.full((c.rows, c.H), 7.0, device="cuda")
    out = torch.full((c.rows, c.H, c.D), 7.0, dtype=c.dtype, device="cuda")
    dfv.tree_attention(cache, kw.pop("layer", 0), tree, q, ws, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert dfv.read_device_error(ws) == 0
    return out.double().cpu(), lse.double().cpu(), cache


def check(c: Case, out, lse, **kw):
    o, l, a, big, keys = c.attention(**kw)
    to, tl = c.tolerances(o, l, a, big, keys)
    assert torch.equal(torch.isinf(lse), torch.isinf(l))
    assert bool(((out - o).abs() <= to).all()), ((out - o).abs() - to).max()
    f = torch.isfinite(l)
    assert bool(((lse - l).abs() <= tl)[f].all()), ((lse - l).abs() - tl)[f].max()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 1), (8, 4), (10, 2), (14, 2), (16, 2), (16, 1), (3, 3)])
def test_heads_and_types(dfv, dtype, dim, heads, kv):
    c = Case([37, 0, 130], [5, 3, 1], heads, kv, dim, 16, dtype, seed=heads + dim)
    out, lse, cache = run(dfv, c)
    check(c, out, lse)
    assert cache.errors() == 0


@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 511, 1000])
@pytest.mark.parametrize("nodes", [1, 2, 16, 33, 64])
def test_lengths(dfv, length, nodes):
    c = Case([length], [nodes], 4, 2, 64, 16, BF, seed=length * 67 + nodes)
    check(c, *run(dfv, c)[:2])


@pytest.mark.parametrize("heads,kv,nodes", [(8, 1, 1), (8, 1, 2), (8, 1, 3), (8, 1, 4), (8, 1, 9), (8, 1, 16), (8, 1, 17),
                                            (8, 1, 64), (16, 1, 64), (5, 1, 13), (7, 1, 64), (2, 2, 64)])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_per_kv_head(dfv, heads, kv, nodes, dim):
    """Every split of nodes x heads over the row tiles."""
    c = Case([200, 63], [nodes, max(1, nodes // 2)], heads, kv, dim, 32, BF, seed=nodes + heads)
    check(c, *run(dfv, c)[:2])


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["head", "token", "mixed"])
@pytest.mark.parametrize("nodes", [1, 20])
def test_pages_and_strides(dfv, page, layout, nodes):
    c = Case([300, 5, 129], [nodes, 7, 1], 8, 2, 128, page, BF, seed=page, layers=2, layout=layout)
    out, lse, _ = run(dfv, c, layer=1)
    check(c, out, lse, layer=1)


@pytest.mark.parametrize("masks", ["tree", "chain", "any"])
@pytest.mark.parametrize("heads", [4, 32])
def test_masks(dfv, masks, heads):
    c = Case([0, 3, 64, 120, 0], [16, 64, 9, 31, 64], heads, 4, 64, 16, FP, seed=9, masks=masks)
    check(c, *run(dfv, c)[:2])


def test_rows_without_keys_are_zero(dfv):
    for heads in (4, 32):
        c = Case([0, 40], [64, 4], heads, 4, 128, 16, BF, seed=2, masks="any")
        c.masks[:64] = [0] * 64
        out, lse, _ = run(dfv, c)
        assert bool((out[:64] == 0).all()) and bool((lse[:64] == -math.inf).all())
        check(c, out, lse)


@pytest.mark.parametrize("nodes", [1, 4, 40])
def test_ragged_batches_and_sequences_without_rows(dfv, nodes):
    rng = random.Random(nodes)
    lens = [rng.randint(0, 400) for _ in range(23)]
    c = Case(lens, [rng.randint(0, nodes) if i else nodes for i in range(23)], 8, 2, 64, 16, BF, seed=5)
    check(c, *run(dfv, c)[:2])


def test_sequences_by_index(dfv):
    """The call's sequences are cache rows 2, 0: lengths and tables follow the index."""
    c = Case([50, 9, 77], [3, 1, 6], 4, 2, 64, 16, BF, seed=4)
    cache, _ = c.gpu(dfv)
    d = Case([77, 50], [6, 3], 4, 2, 64, 16, BF, seed=40)
    d.table, d.k, d.v = c.table[[2, 0]], c.k, c.v
    tree = d.tree(dfv, seq=torch.tensor([2, 0], dtype=torch.int32).cuda())
    check(d, *run(dfv, d, cache, tree)[:2])


@pytest.mark.parametrize("nodes", [1, 16, 64])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_long_cache(dfv, nodes, dtype):
    c = Case([20011], [nodes], 8, 1, 128, 64, dtype, seed=nodes)
    check(c, *run(dfv, c)[:2])


def test_large_scores(dfv):
    """Scores up to hundreds, growing along the cache: the running maximum moves in every tile."""
    for nodes in (1, 20):
        c = Case([700], [nodes], 8, 1, 128, 16, BF, seed=3)
        c.buf.mul_(4)
        ramp = torch.linspace(0.2, 2, c.table.shape[1])
        for j in range(c.table.shape[1]):
            if c.table[0, j] >= 0:
                c.k[0, c.table[0, j]] *= ramp[j]
        c.k, c.v = c._views(c.buf)
        check(c, *run(dfv, c)[:2])


def test_lowest_finite_and_infinite_scores(dfv):
    """A key of the type's lowest values and one of -inf against a positive query: p is 0, the others are unchanged."""
    for nodes in (1, 20):
        c = Case([90], [nodes], 4, 1, 64, 16, BF, seed=6, masks="chain")
        c.q.abs_()
        c.k[0, c.table[0, 1], 0, 3] = torch.finfo(BF).min
        c.k[0, c.table[0, 2], 0, 5] = -math.inf
        out, lse, _ = run(dfv, c)
        d = Case([90], [nodes], 4, 1, 64, 16, BF, seed=6, masks="chain")
        d.q.abs_()
        d.k[0, d.table[0, 1], 0, 3] = -100.0  # far below every other score as well
        d.k[0, d.table[0, 2], 0, 5] = -100.0
        check(d, out, lse)


@pytest.mark.parametrize("heads", [1, 8, 32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_masked_places_may_hold_anything(dfv, heads, bad):
    """Nodes that a row does not see, and everything past the last node, are poisoned in k and v."""
    kv = 1 if heads < 32 else 4
    c = Case([45, 130], [12, 40], heads, kv, 128, 32, BF, seed=8, masks="tree")
    n0 = 12
    hidden = {0: [3, 7, 8], 1: [0, 17, 39]}  # nodes nobody sees
    for s, js in hidden.items():
        for j in js:
            for i in range(c.nodes[s]):
                r = c.off[s] + i
                c.masks[r] &= ~(1 << j)
    want = c.attention()
    to, tl = c.tolerances(*want)
    for s, js in hidden.items():
        for pos in [c.lens[s] + j for j in js] + list(range(c.lens[s] + c.nodes[s], -(-(c.lens[s] + c.nodes[s]) // 32) * 32)):
            pg = c.table[s, pos // 32]
            c.k[0, pg, :, pos % 32] = bad
            c.v[0, pg, :, pos % 32] = bad
    free = sorted(set(range(c.k.shape[1])) - set(c.table.flatten().tolist()))
    c.k[0, free], c.v[0, free] = bad, bad
    out, lse, _ = run(dfv, c)
    assert n0 == c.nodes[0]
    f = torch.isfinite(want[1])
    assert bool(((out - want[0]).abs() <= to).all())
    assert bool(((lse - want[1]).abs() <= tl)[f].all()) and torch.equal(f, torch.isfinite(lse))


@pytest.mark.parametrize("heads", [2, 32])
def test_poison_reaches_only_the_rows_that_see_it(dfv, heads):
    """NaN and infinities in the values of one branch: rows of other branches keep their results."""
    kv = 2 if heads < 32 else 4
    c = Case([70], [24], heads, kv, 128, 16, BF, seed=12, masks="tree")
    c.masks = [1 | 1 << i if i else 1 for i in range(24)]  # a star: every node sees the root and itself
    want = c.attention()
    to, _ = c.tolerances(*want)
    for j, x in ((5, math.nan), (6, math.inf), (11, -math.inf)):
        pos = 70 + j
        c.v[0, c.table[0, pos // 16], :, pos % 16, 7] = x
    out, lse, _ = run(dfv, c)
    clean = [i for i in range(24) if i not in (5, 6, 11)]
    assert bool(((out - want[0]).abs() <= to)[clean].all())
    assert bool(torch.isnan(out[5, :, 7]).all())
    assert bool((out[6, :, 7] == math.inf).all()) and bool((out[11, :, 7] == -math.inf).all())
    others = [d for d in range(128) if d != 7]
    assert bool(((out - want[0]).abs() <= to)[:, :, others].all())


def test_nan_queries_stay_in_their_rows(dfv):
    for heads in (2, 32):
        c = Case([70], [20], heads, 2 if heads < 32 else 4, 64, 16, BF, seed=13)
        want = c.attention()
        to, _ = c.tolerances(*want)
        q = c.q.clone()
        q[4, 1, 3] = math.nan
        out, lse, _ = run(dfv, c, q=q.cuda())
        keep = torch.ones(20, heads, dtype=torch.bool)
        keep[4, 1] = False
        assert bool(((out - want[0]).abs() <= to)[keep].all())
        assert bool(torch.isnan(out[4, 1]).all()) and bool(torch.isnan(lse[4, 1]))


def test_strided_queries_and_outputs(dfv):
    for nodes in (2, 20):
        c = Case([99], [nodes], 8, 2, 64, 16, BF, seed=14)
        cache, tree = c.gpu(dfv)
        big = torch.zeros(nodes, 13, 72, dtype=BF, device="cuda")
        big[:, 3:11, :64] = c.q.cuda()
        ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, 8))
        wide = torch.full((8, nodes, 80), 5.0, dtype=BF, device="cuda")
        out = wide.permute(1, 0, 2)[:, :, 8:72]
        lse = torch.empty(nodes, 8, device="cuda")
        dfv.tree_attention(cache, 0, tree, big[:, 3:11, :64], ws, out=out, lse=lse)
        torch.cuda.synchronize()
        check(c, out.double().cpu(), lse.double().cpu())
        assert bool((wide[:, :, :8] == 5).all()) and bool((wide[:, :, 72:] == 5).all())


def test_other_scale_and_no_lse(dfv):
    for nodes in (1, 20):
        c = Case([150], [nodes], 8, 2, 128, 16, FP, seed=15)
        cache, tree = c.gpu(dfv)
        ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, 8))
        out = dfv.tree_attention(cache, 0, tree, c.q.cuda(), ws, scale=0.3)
        torch.cuda.synchronize()
        want = c.attention(scale=0.3)
        assert bool(((out.double().cpu() - want[0]).abs() <= c.tolerances(*want)[0]).all())


@pytest.mark.parametrize("nodes", [1, 24])
def test_offsets_past_32_bits(dfv, nodes):
    """Pages 2^27 elements apart: the last ones lie past 2^32 elements."""
    c = Case([500], [nodes], 4, 1, 64, 16, BF, seed=16)
    pages = c.k.shape[1]
    step = 1 << 27
    assert pages * step > 1 << 32
    buf = torch.zeros(pages * step + 4096, dtype=BF, device="cuda")
    view = lambda at: torch.as_strided(buf, (1, pages, 1, 16, 64), (0, step, 1024, 64, 1), at)  # noqa: E731
    k, v = view(0), view(2048)
    k.copy_(c.k.cuda())
    v.copy_(c.v.cuda())
    cache = dfv.KVCache(k, v, c.table.cuda(), torch.tensor([500], dtype=torch.int32).cuda())
    check(c, *run(dfv, c, cache, c.tree(dfv))[:2])
    del buf, k, v, cache
    torch.cuda.empty_cache()


def test_same_bits_again_and_graph_replay_with_new_lengths(dfv):
    for nodes, heads in ((1, 8), (16, 8), (40, 32)):
        c = Case([333, 90], [nodes, nodes], heads, 4, 128, 16, BF, seed=17)
        cache, tree = c.gpu(dfv)
        ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, heads))
        q = c.q.cuda()
        first = dfv.tree_attention(cache, 0, tree, q, ws)
        assert torch.equal(first, dfv.tree_attention(cache, 0, tree, q, ws))
        out = torch.empty_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dfv.tree_attention(cache, 0, tree, q, ws, out=out)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        cache.lens.copy_(torch.tensor([17, 91 - 1], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        d = Case([333, 90], [nodes, nodes], heads, 4, 128, 16, BF, seed=17)
        d.lens = [17, 90]
        want = d.attention()
        assert bool(((out.double().cpu() - want[0]).abs() <= d.tolerances(*want)[0]).all())


def test_another_stream_and_one_workspace_for_many_shapes(dfv):
    st = torch.cuda.Stream()
    shapes = [(1, 8), (16, 8), (3, 16), (64, 8), (1, 8)]
    cases = [Case([140 + 3 * i], [n], h, 2, 64, 16, BF, seed=20 + i) for i, (n, h) in enumerate(shapes)]
    made = [c.gpu(dfv) for c in cases]
    ws = dfv.alloc_workspace(max(dfv.tree_attention_workspace_size(k, t, c.H) for c, (k, t) in zip(cases, made)))
    outs = []
    torch.cuda.synchronize()
    for c, (k, t) in zip(cases, made):
        q = c.q.cuda()
        torch.cuda.synchronize()
        outs.append(dfv.tree_attention(k, 0, t, q, ws, stream=st, out=torch.empty_like(q)))
        st.synchronize()
    for c, o in zip(cases, outs):
        want = c.attention()
        assert bool(((o.double().cpu() - want[0]).abs() <= c.tolerances(*want)[0]).all())


@pytest.mark.parametrize("nodes,heads", [(1, 8), (20, 32)])
def test_bad_device_data_is_flagged(dfv, nodes, heads):
    """Lengths, sequence indexes, page ids and row offsets out of range: an error bit, and the other sequences' outputs
    unharmed."""
    c = Case([70, 60, 50, 40], [nodes] * 4, heads, 4, 64, 16, BF, seed=18)
    want = c.attention()
    to, _ = c.tolerances(*want)
    keep = list(range(c.off[1], c.off[2]))

    def attempt(change, bit, empty):
        cache, tree = c.gpu(dfv)
        change(cache, tree)
        out, lse, _ = run(dfv, c, cache, tree)
        assert cache.errors() == bit
        assert bool(((out - want[0]).abs() <= to)[keep].all())
        if empty:
            assert bool((out[:c.off[1]] == 0).all()) and bool((lse[:c.off[1]] == -math.inf).all())

    attempt(lambda k, t: k.lens[0].fill_(-5), dfv.KVERR_LEN, True)
    attempt(lambda k, t: k.lens[0].fill_(1 << 30), dfv.KVERR_LEN, True)
    attempt(lambda k, t: k.lens[0].fill_(2 ** 31 - 1), dfv.KVERR_LEN, True)
    attempt(lambda k, t: k.page_table[0, 1].fill_(-1), dfv.KVERR_PAGE, False)
    attempt(lambda k, t: k.page_table[0, 1].fill_(1 << 30), dfv.KVERR_PAGE, False)
    attempt(lambda k, t: t.row_off[0].fill_(-3), dfv.KVERR_LEN, False)
    attempt(lambda k, t: t.row_off[4].fill_(1 << 20), dfv.KVERR_LEN, False)

    cache, _ = c.gpu(dfv)
    tree = c.tree(dfv, seq=torch.tensor([4, 1, -1, 3], dtype=torch.int32).cuda())
    out, lse, _ = run(dfv, c, cache, tree)
    assert cache.errors() == dfv.KVERR_SEQ
    assert bool(((out - want[0]).abs() <= to)[keep].all()) and bool((out[:c.off[1]] == 0).all())


def test_mask_bits_past_the_tree_are_ignored(dfv):
    for nodes, heads in ((3, 4), (20, 32)):
        c = Case([61], [nodes], heads, 4, 64, 16, BF, seed=19)
        want = c.attention()
        c.masks = [m | (((1 << 64) - 1) ^ ((1 << nodes) - 1)) for m in c.masks]
        assert all(signed(m) < 0 for m in c.masks)
        out, _, _ = run(dfv, c)
        assert bool(((out - want[0]).abs() <= c.tolerances(*want)[0]).all())


@pytest.mark.parametrize("dim,heads,kv", [(64, 4, 1), (64, 16, 2), (128, 8, 1), (64, 16, 1), (128, 12, 1)])
def test_many_tiles_per_range(dfv, dim, heads, kv):
    """Long enough that every range goes round its ring of tiles several times."""
    c = Case([90001, 70003], [2, 1], heads, kv, dim, 64, FP, seed=dim + heads)
    check(c, *run(dfv, c)[:2])
