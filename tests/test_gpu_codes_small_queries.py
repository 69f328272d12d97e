"""Tree attention over codes with queries so small, and keys so large, that only their products are of ordinary size."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_tree_attention_codes import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nodes", [2, 16, 40])
@pytest.mark.parametrize("down", [60, 90, 105, 118])
def test_products_of_ordinary_size(dfv, dim, nodes, down):
    """q 2^-down and K 2^down times as large: powers of two change no rounding, so the definition's tolerance stays."""
    c = Case([700, 90], [nodes, nodes], 8, 1, dim, 16, seed=down)
    c.q = (c.q.float() * 2.0 ** -down).to(torch.bfloat16)
    c.exp[0] = (c.exp[0].int() + down).clamp(27, 247).to(torch.uint8)
    c.check(dfv)
