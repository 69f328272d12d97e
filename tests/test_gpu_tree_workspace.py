"""One zero-filled workspace for all tree-verify calls of a stream: whatever a call leaves in it, the next one of another
kind gives what it gives with a workspace of its own."""
from __future__ import annotations

import random

import pytest
import torch

from tests._tree_util import signed, tree_masks

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


class Step:
    """State of a serving step, made from the seed alone, and the calls on it."""

    def __init__(self, dfv, seqs, nodes, group, seed):
        self.dfv, self.S = dfv, seqs
        rng = random.Random(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = [nodes - s % 3 if nodes > 3 else nodes for s in range(seqs)]
        off = [0]
        for x in n:
            off.append(off[-1] + x)
        self.rows, self.H = off[-1], 2 * group
        masks = [signed(m) for x in n for m in tree_masks(x, rng)]
        i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
        self.tree = dfv.TreeBatch(i32(off), self.rows, max(n), mask=torch.tensor(masks, device="cuda"))
        c = dfv.KVCache.empty(2, 40 * seqs, 16, 2, 64, 2 * seqs, 24)
        c.k.normal_(generator=g)
        c.v.normal_(generator=g)
        self.cache, self.all = c, i32(list(range(seqs)))
        self.grow = [i32([30 + 5 * (s % 4) for s in range(seqs)]), i32([nodes] * seqs)]
        self.forks = i32([s + seqs for s in range(seqs)])
        self.q = torch.randn(self.rows, self.H, 64, generator=g, device="cuda").bfloat16()
        V = 9001
        self.x = torch.randn(self.rows, V, generator=g, device="cuda")
        self.tokens = torch.randint(0, V, (self.rows,), generator=g, device="cuda", dtype=I32)
        self.rules = dfv.LogitRules(repetition=torch.full((seqs,), 1.3, device="cuda"))
        self.path = torch.full((seqs, max(n)), -1, dtype=I32, device="cuda")
        self.path[:, 0], self.path[:, 1:2] = 0, 2 if min(n) > 2 else -1
        self.tau = i32([2 if min(n) > 2 else 1] * seqs)

    def size(self):
        d = self.dfv
        return max(d.tree_attention_workspace_size(self.cache, self.tree, self.H), d.logits_workspace_size(self.rows),
                   d.cache_workspace_size(self.cache))

    def reserve(self, ws, i=0):
        self.dfv.pages_reserve(self.cache, self.all, self.grow[i], ws)

    def attention(self, ws):
        return self.dfv.tree_attention(self.cache, 1, self.tree, self.q, ws)

    def logits(self, ws):
        return self.dfv.logits_process(self.x, self.tree, self.tokens, self.rules, ws)

    def commit(self, ws):
        return self.dfv.cache_commit(self.cache, self.tree, self.path, self.tau, ws).clone()

    def fork(self, ws):
        self.dfv.pages_fork(self.cache, self.all, self.forks, ws)
        got = self.cache.page_table.clone(), self.cache.lens.clone(), self.cache.refs.clone()
        self.dfv.pages_free(self.cache, self.forks)
        return got


def results(dfv, shape, order, seed, shared):
    s = Step(dfv, *shape, seed)
    one = dfv.alloc_workspace(s.size()) if shared else None
    ws = lambda: one if shared else dfv.alloc_workspace(s.size())  # noqa: E731
    s.reserve(ws())
    s.cache.lens[:s.S] = s.grow[0]  # as if that many tokens had been committed
    out = []
    for name in order:
        s.reserve(ws(), 1)
        got = getattr(s, name)(ws())
        out += list(got) if isinstance(got, tuple) else [got]
    torch.cuda.synchronize()
    assert s.cache.errors() == 0
    return [x.cpu() for x in out] + [s.cache.k.cpu(), s.cache.lens.cpu(), s.cache.page_table.cpu()]


@pytest.mark.parametrize("shape", [(3, 8, 4), (20, 64, 4), (20, 64, 8), (2, 1, 1)])
@pytest.mark.parametrize("order", [["attention", "logits", "commit"], ["fork", "logits", "commit", "attention"],
                                   ["logits", "attention", "fork", "commit", "logits", "fork", "attention", "logits"]])
def test_one_workspace_for_every_kind_of_call(dfv, shape, order):
    for i, (a, b) in enumerate(zip(results(dfv, shape, order, 5, True), results(dfv, shape, order, 5, False))):
        assert torch.equal(a, b), i
