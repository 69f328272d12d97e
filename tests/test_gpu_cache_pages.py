"""The greedy walk of drafted trees and the cache's pages against plain Python: walks, commits, copies, reservations,
forks and releases."""
from __future__ import annotations

import random

import pytest
import torch

from tests._tree_util import Case, chain_mask, signed, tree_masks

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


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


# ---------------------------------------------------------------- greedy walk
def walk(masks, tokens, target):
    n = len(tokens)
    if n == 0:
        return []
    up = [((m & ((1 << i) - 1)).bit_length() - 1) for i, m in enumerate(masks)]
    path = [0]
    while True:
        nxt = [c for c in range(n) if up[c] == path[-1] and c != path[-1] and tokens[c] == target[path[-1]]]
        if not nxt:
            return path
        path.append(nxt[0])


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("kind", ["tree", "chain", "any"])
def test_walk(dfv, seed, kind):
    rng = random.Random(seed)
    nodes = [rng.randint(0, 64) for _ in range(30)] + [64, 1, 33, 32]
    off, masks, tokens, target = [0], [], [], []
    for n in nodes:
        off.append(off[-1] + n)
        masks += (tree_masks(n, rng, 4) if kind == "tree" else [chain_mask(i) for i in range(n)] if kind == "chain"
                  else [rng.getrandbits(64) for _ in range(n)])
        few = rng.choice([2, 3, 50])  # few tokens: long paths, siblings with the same token
        tokens += [rng.randrange(few) for _ in range(n)]
        target += [rng.randrange(few) for _ in range(n)]
    m = None if kind == "chain" else torch.tensor([signed(x) for x in masks], dtype=torch.int64).cuda()
    tree = dfv.TreeBatch(i32(off), off[-1], 64, mask=m)
    path, tau = dfv.accept_tree(tree, i32(tokens), i32(target))
    torch.cuda.synchronize()
    for s, n in enumerate(nodes):
        a, b = off[s], off[s + 1]
        want = walk(masks[a:b], tokens[a:b], target[a:b])
        assert int(tau[s]) == len(want)
        assert path[s].tolist() == want + [-1] * (64 - len(want))


def test_a_fully_accepted_chain_of_64(dfv):
    tree = dfv.TreeBatch(i32([0, 64]), 64, 64)
    tok = torch.arange(64, dtype=torch.int32).cuda()
    path, tau = dfv.accept_tree(tree, tok, tok + 1)
    assert int(tau) == 64 and path[0].tolist() == list(range(64))


# ---------------------------------------------------------------- commit
def paths_of(nodes, rng):
    out = []
    for n in nodes:
        t = rng.randint(0, n)
        out.append(sorted(rng.sample(range(n), t)))
    return out


def commit(dfv, c: Case, paths, width=None, new=None):
    cache, tree = c.gpu(dfv)
    width = width or tree.max_nodes
    path = i32([p + [-1] * (width - len(p)) for p in paths])
    ws = dfv.alloc_workspace(dfv.cache_workspace_size(cache))
    lens = dfv.cache_commit(cache, tree, path, i32([len(p) for p in paths]), ws, new_lens=new)
    torch.cuda.synchronize()
    assert not bool(ws[512:512 + 4096].any())  # tickets back at zero
    return cache, lens


def moved(c: Case, paths):
    """The cache after every path moved, row by row from the old one."""
    k, v = c.k.clone(), c.v.clone()
    for s, p in enumerate(paths):
        for j, x in enumerate(p):
            a, b = c.lens[s] + x, c.lens[s] + j
            pa, pb = c.table[s, a // c.page], c.table[s, b // c.page]
            k[:, pb, :, b % c.page] = c.k[:, pa, :, a % c.page]
            v[:, pb, :, b % c.page] = c.v[:, pa, :, a % c.page]
    return k, v


@pytest.mark.parametrize("layout", ["head", "token", "mixed"])
@pytest.mark.parametrize("page,dim,kv", [(8, 64, 1), (16, 128, 4), (64, 16, 3), (256, 256, 2)])
def test_commit(dfv, layout, page, dim, kv):
    rng = random.Random(page)
    nodes = [64, 1, 17, 0, 40, 8, 63]
    c = Case([0, 5, page, 3, page - 1, 2 * page - 1, 100], nodes, kv, kv, dim, page, BF, seed=page, layers=3, layout=layout)
    for _ in range(3):
        paths = paths_of(nodes, rng)
        cache, lens = commit(dfv, c, paths)
        k, v = moved(c, paths)
        assert torch.equal(cache.k.cpu(), k) and torch.equal(cache.v.cpu(), v)
        assert lens.data_ptr() == cache.lens.data_ptr()
        assert lens.tolist() == [a + len(p) for a, p in zip(c.lens, paths)]
        assert cache.errors() == 0


def test_commit_of_long_paths(dfv):
    nodes = [64, 64, 64]
    c = Case([7, 16, 0], nodes, 2, 2, 64, 16, FP, seed=1, layers=2)
    paths = [list(range(64)), list(range(1, 64)), [0] + list(range(2, 64))]
    cache, lens = commit(dfv, c, paths)
    k, v = moved(c, paths)
    assert torch.equal(cache.k.cpu(), k) and torch.equal(cache.v.cpu(), v)
    assert lens.tolist() == [71, 79, 63]


def test_commit_into_other_lengths_leaves_the_old_ones(dfv):
    c = Case([7, 16], [5, 6], 2, 2, 64, 16, BF, seed=2)
    new = i32([-9, -9])
    cache, lens = commit(dfv, c, [[0, 3], [0, 1, 5]], new=new)
    assert lens.tolist() == [9, 19] and cache.lens.tolist() == [7, 16]


def test_bad_paths_keep_the_sequence(dfv):
    c = Case([7, 16, 9], [5, 6, 4], 2, 2, 64, 16, BF, seed=3, layers=2)
    for bad in ([0, 0], [2, 1], [0, 5], [-1, 2], [0, 1 << 20]):
        cache, lens = commit(dfv, c, [bad, [0, 4], [1, 3]], width=9)
        k, v = moved(c, [[], [0, 4], [1, 3]])
        assert torch.equal(cache.k.cpu(), k) and torch.equal(cache.v.cpu(), v)
        assert lens.tolist() == [7, 18, 11]
        assert cache.errors() == dfv.KVERR_PATH
    cache, tree = c.gpu(dfv)
    ws = dfv.alloc_workspace(dfv.cache_workspace_size(cache))
    path = i32([[0] * 6] * 3)
    lens = dfv.cache_commit(cache, tree, path, i32([-1, 7, 1]), ws)
    assert lens.tolist() == [7, 16, 10] and cache.errors() == dfv.KVERR_PATH
    cache, tree = c.gpu(dfv)
    cache.page_table[0, 0] = 1 << 28
    lens = dfv.cache_commit(cache, tree, i32([[0, 3, -1, -1, -1, -1]] * 3), i32([2, 2, 2]), ws)
    assert lens.tolist() == [7, 18, 11] and cache.errors() & dfv.KVERR_PAGE


# ---------------------------------------------------------------- pages
class Pool:
    """The page calls in plain Python."""

    def __init__(self, c: Case, refs):
        self.page, self.refs = c.page, list(refs)
        self.table = c.table.tolist()
        self.lens = list(c.lens)
        self.k, self.v = c.k.clone(), c.v.clone()

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def free(self, seqs):
        for s in seqs:
            for j, p in enumerate(self.table[s]):
                if p >= 0:
                    self.refs[p] -= 1
                    self.table[s][j] = -1
            self.lens[s] = 0

    def reserve(self, seqs, new):
        """Whether the pool ran short."""
        short = False
        for s, n in zip(seqs, new):
            want = range(-(-(self.lens[s] + n) // self.page))
            miss = [j for j in want if self.table[s][j] < 0]
            got = self.free_pages()[:len(miss)]
            short |= len(got) < len(miss)
            if short:  # this one and all after it get nothing
                continue
            for j, p in zip(miss, got):
                self.table[s][j], self.refs[p] = p, 1
        return short

    def fork(self, src, dst):
        lens = [self.lens[s] for s in src]
        rows = [list(self.table[s]) for s in src]
        out = False
        for a, b, n in zip(rows, dst, lens):
            full, rest = divmod(n, self.page)
            if rest:
                got = self.free_pages()
                if out or not got:
                    out = True
                    continue
                p, old = got[0], a[full]
                self.refs[p] = 1
                self.k[:, p, :, :rest], self.v[:, p, :, :rest] = self.k[:, old, :, :rest], self.v[:, old, :, :rest]
                self.table[b][full] = p
            for j in range(full):
                self.table[b][j] = a[j]
                self.refs[a[j]] += 1
            self.lens[b] = n
        return out

    def same(self, cache):
        torch.cuda.synchronize()
        assert cache.page_table.tolist() == self.table
        assert cache.lens.tolist() == self.lens
        assert cache.refs.tolist() == self.refs
        assert torch.equal(cache.k.cpu(), self.k) and torch.equal(cache.v.cpu(), self.v)


def pool(dfv, lens, page=16, empty=4, spare_pages=6, seed=0, layout="head", dim=64, wide=3):
    c = Case(list(lens) + [0] * empty, [0] * (len(lens) + empty), 2, 2, dim, page, BF, seed=seed, layers=2, layout=layout,
             extra=spare_pages, spare=wide)
    refs = torch.zeros(c.k.shape[1], dtype=torch.int32)
    refs[c.table[c.table >= 0].long()] = 1
    c.nodes = [0] * len(c.lens)
    k, v = c._views(c.buf.cuda())
    cache = dfv.KVCache(k, v, c.table.cuda(), i32(c.lens), refs=refs.cuda())
    return cache, Pool(c, refs.tolist()), dfv.alloc_workspace(dfv.cache_workspace_size(cache))


@pytest.mark.parametrize("layout", ["head", "token", "mixed"])
@pytest.mark.parametrize("page", [8, 16, 128])
def test_fork_and_free(dfv, layout, page):
    cache, plain, ws = pool(dfv, [0, 1, page, page + 3, 3 * page - 1], page, empty=8, spare_pages=9, layout=layout)
    src, dst = [4, 3, 3, 2, 1, 4, 0], [5, 6, 7, 8, 9, 10, 11]
    dfv.pages_fork(cache, i32(src), i32(dst), ws)
    assert not plain.fork(src, dst)
    plain.same(cache)
    dfv.pages_free(cache, i32([4, 7, 0, 2]))
    plain.free([4, 7, 0, 2])
    plain.same(cache)
    dfv.pages_fork(cache, i32([5, 6]), i32([4, 2]), ws)  # into the freed places, onto the freed pages
    plain.fork([5, 6], [4, 2])
    plain.same(cache)
    assert cache.errors() == 0


def test_a_sequence_dropped_twice_and_an_empty_one(dfv):
    cache, plain, ws = pool(dfv, [40, 33])
    dfv.pages_fork(cache, i32([0]), i32([2]), ws)
    plain.fork([0], [2])
    dfv.pages_free(cache, i32([0, 0, 3, 0]))
    plain.free([0])
    plain.same(cache)
    assert cache.errors() == 0


def test_forks_without_pages_stay_empty(dfv):
    cache, plain, ws = pool(dfv, [20, 33], empty=4, spare_pages=2)
    dfv.pages_fork(cache, i32([0, 1, 1, 0]), i32([2, 3, 4, 5]), ws)
    assert plain.fork([0, 1, 1, 0], [2, 3, 4, 5])
    plain.same(cache)
    assert cache.errors() == dfv.KVERR_NO_PAGE
    assert cache.lens.tolist() == [20, 33, 20, 33, 0, 0]


def test_refused_forks(dfv):
    cache, plain, ws = pool(dfv, [20, 33], empty=3)
    # a destination in use, out of range, given twice; a source out of range; itself
    dfv.pages_fork(cache, i32([0, 0, 0, 0, 9, 3]), i32([1, 99, 2, 2, 4, 3]), ws)
    plain.fork([0], [2])
    plain.same(cache)
    assert cache.errors() == dfv.KVERR_SEQ


def test_reserve(dfv):
    rng = random.Random(3)
    cache, plain, ws = pool(dfv, [0, 1, 16, 19, 47, 5], empty=6, spare_pages=50, wide=12)
    for _ in range(4):
        seqs = rng.sample(range(12), rng.randint(1, 12))
        new = [rng.randint(0, 64) for _ in seqs]
        dfv.pages_reserve(cache, i32(seqs), i32(new), ws)
        assert not plain.reserve(seqs, new)
        plain.same(cache)
        drop = rng.sample(range(12), 2)
        dfv.pages_free(cache, i32(drop))
        plain.free(drop)
        plain.same(cache)
    assert cache.errors() == 0


def test_reserve_runs_short(dfv):
    cache, plain, ws = pool(dfv, [16, 16, 16], empty=0, spare_pages=3, wide=8)
    dfv.pages_reserve(cache, i32([1, 0, 2]), i32([16, 64, 1]), ws)
    assert plain.reserve([1, 0, 2], [16, 64, 1])
    plain.same(cache)
    assert cache.errors() == dfv.KVERR_NO_PAGE


def test_refused_reservations(dfv):
    cache, plain, ws = pool(dfv, [16, 20], empty=2, spare_pages=20, wide=4)
    wide = cache.page_table.shape[1]
    dfv.pages_reserve(cache, i32([0, -1, 99, 1, 0]), i32([16, 1, 1, 20, 32]), ws)
    plain.reserve([0, 1], [16, 20])
    plain.same(cache)
    assert cache.errors() == dfv.KVERR_SEQ
    cache.err.zero_()
    dfv.pages_reserve(cache, i32([2, 3]), i32([wide * 16 + 1, -4]), ws)
    plain.same(cache)
    assert cache.errors() == dfv.KVERR_LEN


def test_a_large_pool_hands_out_the_lowest_pages(dfv):
    n = 100003
    cache = dfv.KVCache.empty(1, n, 8, 1, 16, 4, 7000)
    free = sorted(random.Random(5).sample(range(n), 6001))
    cache.refs.fill_(1)
    cache.refs[torch.tensor(free).cuda()] = 0
    ws = dfv.alloc_workspace(dfv.cache_workspace_size(cache))
    dfv.pages_reserve(cache, i32([2, 0]), i32([8 * 6000, 8]), ws)
    assert cache.page_table[2, :6000].tolist() == free[:6000]
    assert cache.page_table[0, :2].tolist() == [free[6000], -1]
    assert int((cache.refs == 0).sum()) == 0 and cache.errors() == 0


@pytest.mark.parametrize("layout", ["head", "token", "mixed"])
def test_copy_pages(dfv, layout):
    c = Case([100], [0], 2, 2, 64, 16, FP, seed=6, layers=3, layout=layout)
    cache, _ = c.gpu(dfv)
    dfv.cache_copy_pages(cache, i32([0, 3, 0, 5]), i32([1, 2, 4, 5]))
    k, v = c.k.clone(), c.v.clone()
    for a, b in ((0, 1), (3, 2), (0, 4)):
        k[:, b], v[:, b] = c.k[:, a], c.v[:, a]
    assert torch.equal(cache.k.cpu(), k) and torch.equal(cache.v.cpu(), v) and cache.errors() == 0
    dfv.cache_copy_pages(cache, i32([0, -1, 1 << 30]), i32([1 << 20, 1, 2]))
    assert torch.equal(cache.k.cpu(), k) and cache.errors() == dfv.KVERR_PAGE


def test_offsets_past_32_bits(dfv):
    step = 1 << 27
    buf = torch.zeros(40 * step + 4096, dtype=BF, device="cuda")
    view = lambda at: torch.as_strided(buf, (1, 40, 1, 16, 64), (0, step, 1024, 64, 1), at)  # noqa: E731
    k, v = view(0), view(2048)
    table = torch.full((3, 4), -1, dtype=torch.int32)
    table[0, 0], table[0, 1] = 39, 38
    refs = torch.ones(40, dtype=torch.int32)
    refs[37] = 0
    cache = dfv.KVCache(k, v, table.cuda(), i32([20, 0, 0]), refs=refs.cuda())
    rows = torch.randn(16, 64).to(BF).cuda()
    k[0, 38, 0], v[0, 38, 0] = rows, -rows
    ws = dfv.alloc_workspace(dfv.cache_workspace_size(cache))
    dfv.pages_fork(cache, i32([0]), i32([1]), ws)
    assert cache.page_table[1].tolist() == [39, 37, -1, -1]
    assert torch.equal(k[0, 37, 0, :4], rows[:4]) and torch.equal(v[0, 37, 0, :4], -rows[:4])
    assert not bool(k[0, 37, 0, 4:].any())
    tree = dfv.TreeBatch(i32([0, 6]), 6, 6)
    dfv.cache_commit(cache, tree, i32([[0, 3, 5, -1, -1, -1]]), i32([3]), ws)
    assert torch.equal(k[0, 38, 0, 4:7], rows[[4, 7, 9]])
    del buf, k, v, cache
    torch.cuda.empty_cache()


def test_a_whole_step_in_a_graph(dfv):
    """reserve, rotary append, attention, rules, walk, commit, drop and fork captured once and replayed: the same state,
    step by step, as the calls made eagerly."""
    def make():
        g = torch.Generator().manual_seed(11)
        cache = dfv.KVCache.empty(2, 60, 16, 2, 64, 5, 10)
        cache.k.copy_(torch.randn(cache.k.shape, generator=g).to(BF))
        cache.v.copy_(torch.randn(cache.v.shape, generator=g).to(BF))
        cache.page_table[:3, 0] = i32([7, 3, 9])
        cache.refs[[7, 3, 9]] = 1
        cache.lens[:3] = i32([5, 0, 13])
        rng = random.Random(2)
        nodes = [6, 1, 17]
        masks = [m for n in nodes for m in tree_masks(n, rng)]
        tree = dfv.TreeBatch(i32([0, 6, 7, 24]), 24, 17, mask=torch.tensor([signed(m) for m in masks], dtype=torch.int64).cuda())
        s = dict(cache=cache, tree=tree, rope=dfv.Rope(64), ws=dfv.alloc_workspace(dfv.cache_workspace_size(cache)),
                 aws=dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, 8)),
                 lws=dfv.alloc_workspace(dfv.logits_workspace_size(24)), all=i32([0, 1, 2]), n=i32([6, 1, 17]),
                 qkv=torch.randn(24, 12, 64, generator=g).to(BF).cuda(), x=torch.randn(24, 40, generator=g).cuda(),
                 tokens=torch.randint(0, 40, (24,), generator=g, dtype=torch.int32).cuda(),
                 rules=dfv.LogitRules(repetition=torch.tensor([1.1, 1.2, 1.3]).cuda()), src=i32([2, 0]), dst=i32([3, 4]))
        return s

    def step(s):
        c, t = s["cache"], s["tree"]
        dfv.pages_reserve(c, s["all"], s["n"], s["ws"])
        pos = torch.arange(24, dtype=torch.int32, device="cuda") + c.lens[0]
        out = []
        for layer in range(2):
            q = dfv.rope_append(c, layer, t, s["rope"], s["qkv"][:, :8], s["qkv"][:, 8:10], s["qkv"][:, 10:], pos)
            out.append(dfv.tree_attention(c, layer, t, q, s["aws"]))
        x, best = dfv.logits_process(s["x"], t, s["tokens"], s["rules"], s["lws"])
        path, tau = dfv.accept_tree(t, s["tokens"], best)
        dfv.cache_commit(c, t, path, tau, s["ws"])
        dfv.pages_free(c, s["dst"])
        dfv.pages_fork(c, s["src"], s["dst"], s["ws"])
        return out + [x, best, path, tau]

    def state(s, out):
        c = s["cache"]
        return [x.clone() for x in out + [c.k, c.v, c.page_table, c.lens, c.refs, c.err]]

    a, b = make(), make()
    warm = make()
    step(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(b)
    for _ in range(3):
        want = state(a, step(a))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, state(b, out)):
            assert torch.equal(x, y)
    assert a["cache"].errors() == 0
