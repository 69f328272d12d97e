"""Results of calls on a given stream: they come from that stream's memory, as under torch.cuda.stream(stream).  A block
of the current stream's may still be read by what was queued there before, which the given stream does not wait for."""
from __future__ import annotations

import pytest
import torch

from speculative_decoding_moe_gb300 import inputs

pytestmark = pytest.mark.gpu
I32, BF = torch.int32, torch.bfloat16


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


@pytest.fixture(scope="module")
def calls(dfv):
    """Calls that make their results, by name: stream -> results."""
    rows, H, V = 5, 4, 100
    cache = dfv.KVCache.empty(1, 4, 16, 2, 64, 2, 2)
    cache.page_table.copy_(torch.tensor([[0, 1], [2, 3]], dtype=I32))
    tree = dfv.TreeBatch(torch.tensor([0, 3, 5], dtype=I32).cuda(), rows, 3)
    q, n = torch.randn(rows, H, 64, device="cuda").to(BF), torch.zeros(rows, dtype=I32, device="cuda")
    rope = dfv.Rope(64)
    aws = dfv.alloc_workspace(dfv.tree_attention_workspace_size(cache, tree, H))
    lws = dfv.alloc_workspace(dfv.logits_workspace_size(rows))
    x = torch.randn(rows, V, device="cuda")
    shape = inputs.LayerShape(d=512, n_experts=16, top_k=4, d_ff=128)
    layer = dfv.Layer(inputs.make_layer(shape, 1, device="cuda"))
    h = torch.randn(4, 512, device="cuda").to(BF)
    mws, bws = dfv.alloc_workspace(dfv.workspace_size(layer, 4)), dfv.alloc_workspace(dfv.batch_workspace_size(layer, 4))
    gws = dfv.alloc_workspace(dfv.accept_workspace_size(4, V))
    torch.cuda.synchronize()
    return {
        "rope_append": lambda s: [dfv.rope_append(cache, 0, tree, rope, q, q[:, :2], q[:, 2:], n, stream=s)],
        "tree_attention": lambda s: [dfv.tree_attention(cache, 0, tree, q, aws, stream=s)],
        "logits_process": lambda s: dfv.logits_process(x, tree, None, dfv.LogitRules(), lws, stream=s),
        "accept_tree": lambda s: dfv.accept_tree(tree, n, n, stream=s),
        "route_topk": lambda s: dfv.route_topk(layer, h, mws, stream=s).values(),
        "moe_block_forward": lambda s: [dfv.moe_block_forward(layer, h, mws, stream=s)],
        "moe_batch_forward": lambda s: [dfv.moe_batch_forward(layer, h, 1, bws, stream=s)],
        "accept_greedy": lambda s: dfv.accept_greedy(x, n[:4], gws, stream=s),
        "accept_greedy_noalloc": lambda s: dfv.accept_greedy_noalloc(x, n[:4], stream=s),
    }


def pool_of(t):
    """Handle of the stream whose memory the tensor is in."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


NAMES = ["rope_append", "tree_attention", "logits_process", "accept_tree", "route_topk", "moe_block_forward",
         "moe_batch_forward", "accept_greedy", "accept_greedy_noalloc"]


@pytest.mark.parametrize("name", NAMES)
def test_results_are_in_the_streams_memory(calls, name):
    here = torch.cuda.current_stream()
    plain = list(calls[name](None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = list(calls[name](side))
    torch.cuda.synchronize()
    assert torch.cuda.current_stream() == here
    assert all(pool_of(t) == here.cuda_stream for t in plain)
    assert all(pool_of(t) == side.cuda_stream for t in other)
    given = list(calls[name](here))
    torch.cuda.synchronize()
    assert all(pool_of(t) == here.cuda_stream for t in given)
    with torch.cuda.stream(side):
        back = list(calls[name](here))  # the default stream's handle is 0
    torch.cuda.synchronize()
    assert all(pool_of(t) == here.cuda_stream for t in back)
    for a, b in zip(plain, other):
        assert torch.equal(a, b) or name == "route_topk"  # what route_topk leaves past the woken experts is not written
