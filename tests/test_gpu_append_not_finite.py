"""What is not finite in queries and keys: rows that leave norm_rope_append are those of a 16-bit cache, whatever the cache holds."""
from __future__ import annotations

import pytest
import torch

from tests import test_gpu_norm_rope_append as append
from tests._prompt_util import E4M3

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("heads,kv,dim,rot", [(4, 2, 64, 32), (3, 1, 128, 128), (8, 4, 128, 64), (2, 2, 256, 16), (5, 1, 16, 16)])
def test_rows_out_of_a_cache_in_codes(dfv, heads, kv, dim, rot, norm, inter):
    c = append.Case([5, 0], [9, 3], heads, kv, dim, 16, E4M3, seed=dim, norm=norm)
    g = torch.Generator().manual_seed(2)
    for value in (float("inf"), -float("inf"), float("nan")):  # one in about every other head, in and behind what is turned
        for h in range(heads + 2 * kv):
            r = torch.randint(0, c.n, (3,), generator=g)
            c.qkv[r, h, torch.randint(0, dim, (3,), generator=g)] = value
            c.qkv[r[0], h, dim - 1] = value
    got = {}
    for kind in (E4M3, BF):
        cache = dfv.KVCache.empty(1, 4, 16, kv, dim, 2, 2, dtype=kind)
        cache.page_table.copy_(torch.arange(4, dtype=torch.int32).view(2, 2))
        cache.lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        rows = dfv.RowBatch(append.i32(c.off), c.n, max(c.rows))
        q, k, v = c.split(c.qkv.cuda())
        k_out = torch.zeros(c.n, kv, dim, dtype=BF, device="cuda")
        gains = [x if x is None else x.cuda() for x in c.gains]
        q_out = dfv.norm_rope_append(cache, 0, rows, dfv.Rope(dim, rot_dim=rot, interleaved=inter), q, k, v, c.positions.cuda(),
                                     q_gain=gains[0], k_gain=gains[1], k_out=k_out)
        assert cache.errors() == 0
        got[kind] = q_out.cpu(), k_out.cpu()
    for a, b in zip(got[E4M3], got[BF]):
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(7.0, 8.0, 9.0), b.nan_to_num(7.0, 8.0, 9.0))
    if rot < dim and not norm:  # what is only passed through
        assert bool((torch.isinf(got[BF][0]) == torch.isinf(c.qkv[:, :heads]))[..., rot:].all())
