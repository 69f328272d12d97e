"""lse of tree attention over codes where one key is seen and its product is exact: what the powers' handling adds shows alone."""
from __future__ import annotations

import math

import pytest
import torch

from tests._prompt_util import E4M3, coded
from tests.test_gpu_tree_attention_codes import Case

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nodes", [1, 2, 16, 40])
@pytest.mark.parametrize("value", [300.0, 1.0, 2.0 ** -30])
def test_one_key(dfv, dim, nodes, value):
    c = Case([1] * 9, [nodes] * 9, 8, 1, dim, 16, seed=nodes, masks="chain")
    c.masks = [0] * c.rows  # the committed token only
    for side, x in ((0, 1.0), (1, value)):
        v = torch.zeros(1, dim, dtype=torch.float64)
        v[0, 0] = x
        _, code, e = coded(v)
        for s in range(9):
            c.raw[side][0, int(c.table[s, 0]), :, 0] = code.float().to(E4M3).view(torch.uint8)
            c.exp[side][0, int(c.table[s, 0]), :, 0] = (e + 127).to(torch.uint8)
    b = float(e[0])
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = (torch.rand(c.q.shape[:2], generator=torch.Generator().manual_seed(1)) * 0.9 + 0.1).to(torch.bfloat16)
    out, lse, err = c.run(dfv, scale=1.0)
    assert err == 0
    x = c.q[..., 0].double()
    # in units of log2: the scale's two roundings and the score's, x + b rounded, M - 6 and x - z rounded at up to
    # |b| + 8, the power 2^-22 of itself, log2 of a sum of up to 2^(6 - b) by an ulp; then the sum and the product with ln 2
    t = math.log(2) * (3 * U * 1.5 * x + U * (x * 1.5 + abs(b)) + 2 * U * (abs(b) + 8) + 2.0 ** -22 / math.log(2) + 2 * U * (6 + abs(b))) + 2 * U * x
    d = (lse.double().cpu() - x).abs()
    assert bool((d <= t).all()), "lse off by %g of its tolerance" % float((d / t).max())
    assert torch.equal(out[..., 0].float().cpu(), torch.full(x.shape, float(code[0, 0] * 2.0 ** b)))
