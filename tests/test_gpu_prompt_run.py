"""A prompt in two chunks, drafted nodes and a commit, one call after the other as a serving loop makes them, over caches in
16 bits and in codes: each attention against the definition over what the cache holds, the whole once more as a captured
graph, and calls on two streams at once."""
from __future__ import annotations

import pytest
import torch

from tests._prompt_util import E4M3, attention, check, offsets
from tests._tree_util import Case as Tree
from tests.test_gpu_tree_attention_codes import Case as CodesTree

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
FIRST, NEXT, NODES = [20, 0, 33], [5, 17, 140], [4, 1, 7]


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


def batch(dfv, counts):
    return dfv.RowBatch(i32(offsets(counts)), sum(counts), max(counts))


class Run:
    """The operators' case of `kind` with the test's lengths, and its device state."""

    def __init__(self, dfv, kind, heads, kv, dim, page):
        self.dfv, self.kind, self.dt, self.H, self.K, self.D = dfv, kind, BF if kind == E4M3 else kind, heads, kv, dim
        total = [a + b for a, b in zip(FIRST, NEXT)]
        if kind == E4M3:
            self.tree = CodesTree(total, NODES, heads, kv, dim, page, seed=3, layers=2)
        else:
            self.tree = Tree(total, NODES, heads, kv, dim, page, kind, seed=3, layers=2)
        c = self.tree
        self.cache = c.cache(dfv) if kind == E4M3 else c.gpu(dfv)[0]
        self.cache.lens.zero_()
        g = torch.Generator(device="cuda").manual_seed(4)
        rand = lambda n: torch.randn(n, heads + 2 * kv, dim, device="cuda", generator=g).to(self.dt)  # noqa: E731
        self.qkv = [rand(sum(n)) for n in (FIRST, NEXT, NODES)]
        self.gains = [(1 + 0.3 * torch.randn(dim, device="cuda", generator=g)).to(self.dt) for _ in range(2)]
        self.rope = dfv.Rope(dim)
        self.rows = [batch(dfv, n) for n in (FIRST, NEXT, NODES)]
        self.keys = batch(dfv, total)
        self.nodes = c.tree(dfv)
        start = [0] * 3
        self.pos = []
        for n in (FIRST, NEXT, NODES):
            self.pos.append(i32([start[s] + i for s, m in enumerate(n) for i in range(m)]))
            start = [a + b for a, b in zip(start, n)]
        self.path = torch.full((3, max(NODES)), -1, dtype=torch.int32, device="cuda")
        self.path[:, 0] = 0
        self.path[0, 1], self.path[2, 1], self.path[2, 2] = 2, 3, 5
        self.tau = i32([2, 1, 3])
        size = max([dfv.prompt_attention_workspace_size(r, heads, kv, dim) for r in self.rows[:2]]
                   + [dfv.tree_attention_workspace_size(self.cache, self.nodes, heads), dfv.cache_workspace_size(self.cache)])
        self.ws = dfv.alloc_workspace(size)  # one for every call

    def append(self, i, layer=1, **kw):
        q, k, v = self.qkv[i][:, :self.H], self.qkv[i][:, self.H:self.H + self.K], self.qkv[i][:, self.H + self.K:]
        q = self.dfv.norm_rope_append(self.cache, layer, self.rows[i], self.rope, q, k, v, self.pos[i], q_gain=self.gains[0],
                                      k_gain=self.gains[1], **kw)
        return q, v

    def first(self):
        k = torch.empty(sum(FIRST), self.K, self.D, dtype=self.dt, device="cuda")
        q, v = self.append(0, k_out=k)
        o = self.dfv.prompt_attention(self.rows[0], q, k, v, self.ws)
        self.cache.lens.add_(self.rows[0].row_off[1:] - self.rows[0].row_off[:-1])
        return q, k, v, o

    def rest(self):
        q, _ = self.append(1)
        k, v = self.dfv.cache_read(self.cache, 1, self.keys)
        o = self.dfv.prompt_attention(self.rows[1], q, k, v, self.ws, keys=self.keys)
        self.cache.lens.add_(self.rows[1].row_off[1:] - self.rows[1].row_off[:-1])
        qn, _ = self.append(2)
        on = self.dfv.tree_attention(self.cache, 1, self.nodes, qn, self.ws)
        return q, k, v, o, qn, on

    def commit(self):
        return self.dfv.cache_commit(self.cache, self.nodes, self.path, self.tau, self.ws)

    def state(self):
        return [x for x in (self.cache.k, self.cache.v, self.cache.k_exp, self.cache.v_exp, self.cache.lens) if x is not None]


SHAPES = [(8, 2, 128, 16), (7, 1, 64, 8), (32, 2, 128, 32)]  # the last: more than 16 rows per kv head


@pytest.mark.parametrize("kind", [BF, HF, E4M3])
@pytest.mark.parametrize("heads,kv,dim,page", SHAPES)
def test_two_chunks_nodes_and_a_commit(dfv, kind, heads, kv, dim, page):
    r = Run(dfv, kind, heads, kv, dim, page)
    scale = dim ** -0.5
    bits = lambda x: x.view(torch.uint8) if x.dtype == E4M3 else x  # noqa: E731
    q, k, v, o = r.first()
    off = offsets(FIRST)
    check(o, None, r.dt, dim, max(FIRST), *attention(*(x.cpu() for x in (q, k, v)), off, off, scale))
    if kind != E4M3:  # what later chunks read are the rows that this one attended to
        kr, vr = dfv.cache_read(r.cache, 1, r.rows[0])
        assert torch.equal(kr, k) and torch.equal(vr, v)
    was = [x.clone() for x in r.state()]
    q, k, v, o, qn, on = r.rest()
    assert r.cache.lens.tolist() == [25, 17, 173]
    total = offsets([25, 17, 173])
    check(o, None, r.dt, dim, 173, *attention(*(x.cpu() for x in (q, k, v)), offsets(NEXT), total, scale))
    c = r.tree
    c.q = qn.cpu()
    if kind == E4M3:
        for to, fr in ((c.raw, (r.cache.k, r.cache.v)), (c.exp, (r.cache.k_exp, r.cache.v_exp))):
            for i, x in enumerate(fr):
                to[i] = bits(x).cpu()
        want, _, tol, _ = c.want(layer=1)
    else:
        c.k, c.v = r.cache.k.cpu(), r.cache.v.cpu()
        w = c.attention(layer=1)
        want, tol = w[0], c.tolerances(*w)[0]
    d = (on.double().cpu() - want).abs()
    assert bool((d <= tol).all()), "nodes off by %g of the tolerance" % float((d / tol).max())
    nodes = dfv.cache_read(r.cache, 1, batch(dfv, [29, 18, 180]))  # with the nodes' rows behind the tokens
    assert r.commit().tolist() == [27, 18, 176]
    kept = dfv.cache_read(r.cache, 1, batch(dfv, [27, 18, 176]))
    for a, b in zip(kept, nodes):
        assert torch.equal(a[:26], b[:26]) and torch.equal(a[26], b[27])  # sequence 0: nodes 0 and 2
        assert torch.equal(a[27:45], b[29:47])
        assert torch.equal(a[45:219], b[47:221]) and torch.equal(a[219:221], b[[223, 225]])  # sequence 2: 0, 3 and 5
    assert r.cache.errors() == 0 and dfv.read_device_error(r.ws) == 0
    # the same from the first chunk's state, captured and replayed twice
    ended = [x.clone() for x in r.state()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = r.rest()
        r.commit()
    for _ in range(2):
        for x, y in zip(r.state(), was):
            bits(x).copy_(bits(y))
        g.replay()
        for x, y in zip(again, (q, k, v, o, qn, on)):
            assert torch.equal(x, y)
        for x, y in zip(r.state(), ended):
            assert torch.equal(bits(x), bits(y))
    assert r.cache.errors() == 0 and dfv.read_device_error(r.ws) == 0


@pytest.mark.parametrize("kind", [BF, E4M3])
def test_two_streams_at_once(dfv, kind):
    """Two caches, each on its own stream with its own workspace, interleaved call by call: as one after the other."""
    want = []
    for heads in (8, 32):
        r = Run(dfv, kind, heads, 2, 128, 16)
        want.append((r.first()[3], *r.rest()[3::2]))
    torch.cuda.synchronize()
    pair = [Run(dfv, kind, heads, 2, 128, 16) for heads in (8, 32)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pair]
    got = [[], []]
    for step in ("first", "rest"):
        for r, s, to in zip(pair, streams, got):
            with torch.cuda.stream(s):
                out = getattr(r, step)()
                to += out[3::2]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("kind", [BF, E4M3])
def test_pages_behind_4_gb(dfv, kind):
    """The same calls over pages whose bytes are more than 2^32 behind the cache's start give the same bits; what nobody wrote is
    left as it is found there."""
    total, H, K, D, page, some = [25, 17, 173], 32, 8, 128, 256, 8
    far = (1 << 32) // (K * page * D * (1 if kind == E4M3 else 2)) + 5
    qkv = torch.randn(sum(total), H + 2 * K, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)).to(BF)
    pos = i32([i for n in total for i in range(n)])
    rows, tree = batch(dfv, total), dfv.TreeBatch(i32([0, 1, 2, 6]), 6, 4)
    got = []
    for first in (0, far):
        k, v = (torch.empty(1, first + some, K, page, D, dtype=kind, device="cuda") for _ in range(2))
        exp = [torch.full((1, first + some, K, page), 127, dtype=torch.uint8, device="cuda") if kind == E4M3 else None for _ in range(2)]
        table = i32([[first + 3, -1], [first + 6, -1], [first + 1, -1]])
        cache = dfv.KVCache(k, v, table, i32([0, 0, 0]), k_exp=exp[0], v_exp=exp[1])
        q = dfv.norm_rope_append(cache, 0, rows, dfv.Rope(D), qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:], pos)
        back = dfv.cache_read(cache, 0, rows)
        out = [q, *back]
        for nodes in (tree, dfv.TreeBatch(i32([0, 8, 9, 17]), 17, 8)):  # few and many rows per kv head
            cache.lens.copy_(i32([n - 8 for n in total]))
            ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, nodes, H))
            out.append(dfv.tree_attention(cache, 0, nodes, q[:nodes.n_rows], ws))
        assert cache.errors() == 0
        got.append(out)
        del k, v, cache
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_rows_behind_4_gb(dfv):
    """Rows whose stride takes them past 2^32 bytes, as compact ones."""
    n, H, K, D, pitch = 160, 8, 2, 128, 1 << 24
    rows, keys = batch(dfv, [60, 100]), batch(dfv, [60, 100])
    flat = torch.randn(n, H + 2 * K, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(10)).to(BF)
    wide = torch.empty(n, pitch, dtype=BF, device="cuda")
    part = lambda at, m: wide[:, at * D:(at + m) * D].unflatten(1, (m, D))  # noqa: E731
    q, k, v, o = part(0, H), part(H, K), part(H + K, K), part(H + 2 * K, H)
    for x, y in ((q, flat[:, :H]), (k, flat[:, H:H + K]), (v, flat[:, H + K:])):
        x.copy_(y)
    ws = dfv.alloc_workspace(dfv.prompt_attention_workspace_size(rows, H, K, D))
    want = dfv.prompt_attention(rows, flat[:, :H], flat[:, H:H + K], flat[:, H + K:], ws)
    dfv.prompt_attention(rows, q, k, v, ws, keys=keys, out=o)
    assert torch.equal(o, want)
    # and through the append and the read, in place
    cache = dfv.KVCache.empty(1, 24, 16, K, D, 2, 12)
    cache.page_table.copy_(torch.arange(24, dtype=torch.int32).view(2, 12))
    pos = i32([*range(60), *range(100)])
    want = dfv.norm_rope_append(cache, 0, rows, dfv.Rope(D), flat[:, :H], flat[:, H:H + K], flat[:, H + K:], pos)
    kept = dfv.cache_read(cache, 0, rows)
    dfv.norm_rope_append(cache, 0, rows, dfv.Rope(D), q, k, v, pos, out=q, k_out=k)
    assert torch.equal(q, want) and torch.equal(k, kept[0])
    dfv.cache_read(cache, 0, rows, k=o[:, :K], v=o[:, K:2 * K])
    assert torch.equal(o[:, :K], kept[0]) and torch.equal(o[:, K:2 * K], kept[1])


@pytest.mark.parametrize("kind", [BF, E4M3])
def test_a_given_stream(dfv, kind):
    """Calls on a stream that is not the current one, their results of that stream's memory: as on the current one."""
    r = Run(dfv, kind, 8, 2, 128, 16)
    want = [x.clone() for x in r.first()]
    r.cache.lens.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x = r.qkv[0]
    k = torch.empty_like(want[1])
    s.wait_stream(torch.cuda.current_stream())
    q = dfv.norm_rope_append(r.cache, 1, r.rows[0], r.rope, x[:, :8], x[:, 8:10], x[:, 10:], r.pos[0], q_gain=r.gains[0],
                             k_gain=r.gains[1], k_out=k, stream=s)
    back = dfv.cache_read(r.cache, 1, r.rows[0], stream=s)
    o = dfv.prompt_attention(r.rows[0], q, k, x[:, 10:], r.ws, stream=s)
    s.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(o, want[3])
    for a, b in zip(back, dfv.cache_read(r.cache, 1, r.rows[0])):
        assert torch.equal(a, b)


def test_the_same_sequence_twice(dfv):
    """Two parts of a call that read one sequence; for storing, a sequence may be in a call once."""
    r = Run(dfv, BF, 8, 2, 128, 16)
    r.first()
    rows = dfv.RowBatch(i32([0, 33, 53, 63]), 63, 33, seq=i32([2, 0, 2]))
    k, v = dfv.cache_read(r.cache, 1, rows)
    k1, v1 = dfv.cache_read(r.cache, 1, r.rows[0])
    for a, b in ((k, k1), (v, v1)):
        assert torch.equal(a[:33], b[20:]) and torch.equal(a[33:53], b[:20]) and torch.equal(a[53:], b[20:30])
    assert r.cache.errors() == 0
