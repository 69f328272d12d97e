"""A key that a row does not attend to leaves the row's bits as they are, however large the key and its value are and
however much the rows that do attend to it change."""
from __future__ import annotations

import pytest
import torch

from tests import _tree_util, test_gpu_prompt_attention as prompts, test_gpu_tree_attention_codes as codes

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


def trees(counts, own=True):
    """(masks, rows that do not see the hidden nodes): in each tree, the middle node is seen by no other, and by itself if
    `own`; the others see themselves and those before them."""
    masks, keep = [], []
    for n in counts:
        for i in range(n):
            hidden = 1 << (n // 2)
            masks.append(((2 << i) - 1) & ~hidden | (hidden if own and i == n // 2 else 0))
            keep.append(not (own and i == n // 2))
    return masks, torch.tensor(keep)


def same(a, b, keep):
    return torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1][keep], b[1][keep])


# trees at the end of a tile, across two, and with nothing before them; so many pairs that a CTA takes several tiles of each
FEW, MANY = [200, 0, 125], [500 + 17 * s for s in range(24)]
# 1 to 512 rows per kv head
CODES = [(heads, dim, nodes, own) for heads, dim in ((8, 128), (2, 64), (16, 64)) for nodes in (2, 3, 7, 16, 17, 40, 64) for own in (True, False)
         if heads * nodes <= 512] + [(8, 64, 1, False), (8, 128, 1, False)]


@pytest.mark.parametrize("lens,kv,heads,dim,nodes,own", [(FEW, 1) + c for c in CODES] + [(MANY, 8, 64, 128, n, True) for n in (2, 16, 25)]
                         + [(MANY, 8, 16, 64, 40, True), (MANY, 8, 64, 64, 2, False)])
def test_codes(dfv, lens, kv, heads, dim, nodes, own):
    counts = [nodes] * len(lens)
    c = codes.Case(lens, counts, heads, kv, dim, 16, seed=nodes + heads)
    c.masks, keep = trees(counts, own)
    keep = keep.cuda()
    was, exps = c.run(dfv), c.exp
    for sides in ((0,), (1,), (0, 1)):
        for up in (8, 20, 30, 100, -90) if lens is FEW else (30,):
            c.exp = [x.clone() for x in exps]
            for s, n in enumerate(counts):
                at = lens[s] + n // 2
                for side in sides:
                    e = c.exp[side][0, int(c.table[s, at // 16]), :, at % 16]
                    e.copy_((e.int() + up).clamp(127 - 100, 127 + 120).to(torch.uint8))
            got = c.run(dfv)
            assert got[2] == 0 and same(got, was, keep), "sides %s, 2^%d" % (sides, up)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,kv,heads,dim,nodes", [(FEW, 1) + c for c in ((8, 128, 2), (2, 64, 8), (8, 128, 16), (8, 64, 40), (8, 128, 64))]
                         + [(MANY, 8, 16, 64, 8), (MANY, 8, 64, 128, 2), (MANY, 8, 64, 128, 16), (MANY, 8, 16, 64, 40), (MANY, 8, 64, 64, 25)])
def test_16_bits(dfv, lens, kv, heads, dim, nodes, dtype):
    counts = [nodes] * len(lens)
    c = _tree_util.Case(lens, counts, heads, kv, dim, 16, dtype, seed=nodes + heads)
    c.masks, keep = trees(counts)

    def run(side=None, factor=1.0):
        cache, tree = c.gpu(dfv)
        if side is not None:
            for s, n in enumerate(counts):
                at = lens[s] + n // 2
                (cache.k, cache.v)[side][0, int(c.table[s, at // 16]), :, at % 16] *= factor
        ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, heads))
        lse = torch.zeros(c.rows, heads, device="cuda")
        out = dfv.tree_attention(cache, 0, tree, c.q.cuda(), ws, lse=lse)
        assert dfv.read_device_error(ws) == 0 and cache.errors() == 0
        return out, lse

    was, keep = run(), keep.cuda()
    for side in (0, 1):
        for factor in (30.0, -30.0, 1e4, 1e30 if dtype == BF else 1e3) if lens is FEW else (30.0, -30.0):
            assert same(run(side, factor), was, keep), "%s times %g" % ("kv"[side], factor)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,dim,rows,keys", [(8, 128, [40], [40]), (1, 64, [200], [200]), (4, 64, [130, 7], [130, 300]), (8, 128, [300], [1700]),
                                                 (16, 64, [70, 33], [70, 33])])
def test_prompts(dfv, heads, dim, rows, keys, dtype):
    """Positions before a key."""
    c = prompts.Case(rows, keys, heads, 1, dim, dtype, seed=3)
    was = c.run(dfv)[:2]
    for i in (1, rows[0] // 2, rows[0] - 1):  # positions of the first prompt
        at = keys[0] - rows[0] + i
        keep = torch.ones(c.n, dtype=torch.bool, device="cuda")
        keep[i:rows[0]] = False
        for side in (0, 1):
            for factor in (30.0, -30.0, 1e4, 1e30 if dtype == BF else 1e3):
                x = [c.k.clone(), c.v.clone()]
                x[side][at] *= factor
                assert same(c.run(dfv, k=x[0].cuda(), v=x[1].cuda())[:2], was, keep), "%s of position %d times %g" % ("kv"[side], i, factor)
