"""Tree attention over many short sequences, several of which a CTA takes one after the other: what one of them holds
that is not finite reaches its own rows, every time, and no other sequence's."""
from __future__ import annotations

import math

import pytest
import torch

from tests._tree_util import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


@pytest.mark.parametrize("heads,kv,nodes,S", [(4, 2, 2, 600), (4, 1, 4, 500), (8, 1, 4, 300), (16, 1, 16, 120)])
def test_values_that_are_not_finite_stay_with_their_sequence(dfv, heads, kv, nodes, S):
    c = Case([(37 * s) % 90 for s in range(S)], [1 + s % nodes for s in range(S)], heads, kv, 64, 16, torch.bfloat16, seed=31)
    want = c.attention()
    tol, _ = c.tolerances(*want)
    bad = torch.zeros(c.rows, dtype=torch.bool)
    for s in range(0, S, 3):  # the root, which every node of its tree sees
        pos = c.lens[s]
        c.v[0, c.table[s, pos // 16], :, pos % 16, 5] = math.inf
        bad[c.off[s]:c.off[s + 1]] = True
    cache, tree = c.gpu(dfv)
    ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, heads))
    q = c.q.cuda()
    first = dfv.tree_attention(cache, 0, tree, q, ws)
    for _ in range(10):
        assert torch.equal(dfv.tree_attention(cache, 0, tree, q, ws), first)
    out = first.double().cpu()
    assert dfv.read_device_error(ws) == 0 and cache.errors() == 0
    assert bool((out[bad][:, :, 5] == math.inf).all())
    rest = [d for d in range(64) if d != 5]
    assert bool(((out - want[0]).abs() <= tol)[:, :, rest].all())
    assert bool(((out - want[0]).abs() <= tol)[~bad].all())


def test_three_row_tiles_and_a_workspace_of_the_largest_tree(dfv):
    """513 to 768 rows per kv head; one workspace, sized for the largest tree, for all smaller ones."""
    ws = None
    for heads, kv, nodes, dim in ((12, 1, 64, 128), (12, 1, 43, 128), (12, 1, 42, 128), (12, 1, 5, 128), (12, 1, 64, 64), (9, 1, 64, 128)):
        c = Case([700, 130], [nodes, max(1, nodes // 3)], heads, kv, dim, 16, torch.bfloat16, seed=nodes + dim)
        want = c.attention()
        tol, tol_lse = c.tolerances(*want)
        cache, tree = c.gpu(dfv)
        if ws is None:
            ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, heads))
        lse = torch.empty(c.rows, heads, device="cuda")
        out = dfv.tree_attention(cache, 0, tree, c.q.cuda(), ws, lse=lse)
        torch.cuda.synchronize()
        assert dfv.read_device_error(ws) == 0
        assert bool(((out.double().cpu() - want[0]).abs() <= tol).all())
        assert bool(((lse.double().cpu() - want[1]).abs() <= tol_lse).all())
