"""Scores so large that fp32 holds them in steps of several units of log2: weights stay finite, outputs within their values."""
from __future__ import annotations

import itertools
import math

import pytest
import torch

from tests import _tree_util, test_gpu_prompt_attention as prompts, test_gpu_tree_attention_codes as codes
from tests._prompt_util import E4M3, coded, valued

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


def rising(n, dim, size, step, q0, k0):
    """(q, k, scale): scores of about `size`, in units of log2, that rise by `step` over the n keys (but for the types' rounding)."""
    k = torch.zeros(n, dim)
    k[:, 0] = k0
    k[:, 1] = torch.linspace(0, 1, n) * 32.0
    q = torch.zeros(dim)
    q[0], q[1] = q0, q0 * k0 * step / size / 32.0
    return q, k, size / (q0 * k0) * math.log(2)


# dot products of one bit and of more: their product with the scale is exact, or rounds
FIRST = ((32.0, 1024.0), (33.0, 1000.0))
CODED = ((64.0, 512.0), (79.0, 416.0))  # that e4m3 holds
SIZES = [2.0 ** e for e in (24, 24.7, 25, 25.6, 26, 26.5, 27, 28, 28.6, 29.3, 30, 30.5, 31)]
STEPS = (0.0, 4.0, 7.9, 8.0, 16.0, 40.0)


def inside(out, v):
    assert bool(torch.isfinite(out).all())
    # a mean of values, rounded: no further out than the largest
    assert float(out.float().abs().max()) <= float(v.float().abs().max()) * (1 + 2.0 ** -7)


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("dim,nodes", [(64, 1), (128, 2), (64, 20), (128, 16), (128, 33)])
def test_trees(dfv, dim, nodes, dtype):
    lens = [1500, 900]
    c = _tree_util.Case(lens, [nodes] * 2, 8, 1, dim, 16, dtype, seed=1)
    c.masks = None
    for size, step, (q0, k0) in itertools.product(SIZES, STEPS, FIRST):
        cache, tree = c.gpu(dfv)
        q, k, scale = rising(lens[0] + nodes, dim, size, step, q0, k0)
        for s, n in enumerate(lens):
            at = torch.arange(n + nodes)
            cache.k[0, c.table[s, at // 16].long().cuda(), 0, (at % 16).cuda()] = k[:n + nodes].to(dtype).cuda()
        ws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, 8))
        out = dfv.tree_attention(cache, 0, tree, q.to(dtype).cuda().expand(c.rows, 8, dim).contiguous(), ws, scale=scale)
        assert dfv.read_device_error(ws) == 0
        inside(out, c.v)


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("dim,rows,keys", [(64, 40, 1500), (128, 300, 1700), (128, 137, 137)])
def test_prompts(dfv, dim, rows, keys, dtype):
    c = prompts.Case([rows], [keys], 8, 1, dim, dtype, seed=2)
    for size, step, (q0, k0) in itertools.product(SIZES, STEPS, FIRST):
        q, k, scale = rising(keys, dim, size, step, q0, k0)
        c.q, c.k = q.to(dtype).expand(rows, 8, dim).contiguous(), k.to(dtype)[:, None].contiguous()
        out, _, err = c.run(dfv, scale=scale)
        assert err == 0
        inside(out, c.v)


@pytest.mark.parametrize("dim,nodes", [(64, 1), (128, 2), (64, 20), (128, 16), (128, 33)])
def test_codes(dfv, dim, nodes):
    lens = [1500, 900]
    c = codes.Case(lens, [nodes] * 2, 8, 1, dim, 16, seed=3, masks="chain", spread=0.1)
    v = valued(c.raw[1].view(E4M3), c.exp[1])
    for size, step, (q0, k0) in itertools.product(SIZES, STEPS, CODED):
        q, k, scale = rising(lens[0] + nodes, dim, size, step, q0, k0)
        _, code, e = coded(k.double())
        for s, n in enumerate(lens):
            at = torch.arange(n + nodes)
            pg = c.table[s, at // 16].long()
            c.raw[0][0, pg, 0, at % 16] = code[:n + nodes].float().to(E4M3).view(torch.uint8)
            c.exp[0][0, pg, 0, at % 16] = (e[:n + nodes] + 127).to(torch.uint8)
        c.q = q.to(BF).expand(c.rows, 8, dim).contiguous()
        out, _, err = c.run(dfv, scale=scale)
        assert err == 0
        inside(out, v)
