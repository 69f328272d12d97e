"""What the tree-verify binding refuses by itself, before the library is asked (CPU)."""
import pytest
import torch

BF, I = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def dfv():
    from speculative_decoding_moe_gb300 import build, dfv as m
    build.build()
    return m


@pytest.fixture
def setup(dfv):
    k = torch.zeros(1, 4, 2, 16, 64, dtype=BF)
    cache = dfv.KVCache(k, k.clone(), torch.zeros(3, 4, dtype=I), torch.zeros(3, dtype=I), refs=torch.zeros(4, dtype=I))
    tree = dfv.TreeBatch(torch.tensor([0, 3, 5], dtype=I), 5, 3)
    return cache, tree, torch.zeros(4096, dtype=torch.uint8)


def calls(dfv, cache, tree, ws):
    q, n = torch.zeros(5, 4, 64, dtype=BF), torch.zeros(5, dtype=I)
    return [lambda: dfv.rope_append(cache, 0, tree, dfv.Rope(64, device="cpu"), q, q[:, :2], q[:, :2], n),
            lambda: dfv.tree_attention(cache, 0, tree, q, ws),
            lambda: dfv.logits_process(torch.zeros(5, 100), tree, None, dfv.LogitRules(), ws),
            lambda: dfv.accept_tree(tree, n, n),
            lambda: dfv.cache_commit(cache, tree, torch.zeros(2, 3, dtype=I), torch.zeros(2, dtype=I), ws),
            lambda: dfv.cache_copy_pages(cache, n[:1], n[:1]),
            lambda: dfv.pages_reserve(cache, n[:1], n[:1], ws),
            lambda: dfv.pages_fork(cache, n[:1], n[:1], ws),
            lambda: dfv.pages_free(cache, n[:1])]


@pytest.mark.parametrize("which", range(9))
def test_host_tensors(dfv, setup, which):
    with pytest.raises(ValueError, match="CUDA tensors"):
        calls(dfv, *setup)[which]()


@pytest.mark.parametrize("which", (1, 2, 4, 6, 7))
def test_workspaces(dfv, setup, which):
    cache, tree, ws = setup
    for bad, error in ((None, ValueError), (7, TypeError), (ws[::2], ValueError)):
        with pytest.raises(error, match="ws"):
            calls(dfv, cache, tree, bad)[which]()


def test_kinds_of_arguments(dfv, setup):
    cache, tree, ws = setup
    q, n = torch.zeros(5, 4, 64, dtype=BF), torch.zeros(5, dtype=I)
    with pytest.raises(TypeError, match="q must be a tensor"):
        dfv.tree_attention(cache, 0, tree, [1.0], ws)
    with pytest.raises(ValueError, match="q is missing"):
        dfv.tree_attention(cache, 0, tree, None, ws)
    with pytest.raises(TypeError):
        dfv.tree_attention(cache, "0", tree, q, ws)
    with pytest.raises(ValueError, match="32 bits"):
        dfv.tree_attention(cache, 1 << 40, tree, q, ws)
    with pytest.raises(TypeError):
        dfv.tree_attention(cache, 0, tree, q, ws, scale="1")
    with pytest.raises(TypeError, match="bf16 or fp32"):
        dfv.logits_process(torch.zeros(5, 100, dtype=torch.float16), tree, None, dfv.LogitRules(), ws)
    with pytest.raises(ValueError, match="no out"):
        dfv.logits_process(torch.zeros(5, 100), tree, None, dfv.LogitRules(), ws, out=torch.zeros(5, 100), store=False)
    with pytest.raises(ValueError, match="like logits"):
        dfv.logits_process(torch.zeros(5, 100), tree, None, dfv.LogitRules(), ws, out=torch.zeros(5, 100, dtype=BF))
    with pytest.raises(ValueError, match="path must have shape"):
        dfv.cache_commit(cache, tree, n, n[:2], ws)
    with pytest.raises(ValueError, match="tau must have shape"):
        dfv.accept_tree(tree, n, n, tau=n)


def test_descriptors_follow(dfv, setup):
    """The descriptors that the C calls and the extension get are the same memory."""
    import ctypes
    cache, tree, _ = setup
    for x in (cache, tree, dfv.LogitRules()):
        assert ctypes.addressof(x.c) == x.addr


class Queue:
    def __init__(self, index, handle):
        self.device_index, self.cuda_stream = index, handle


def test_calls_are_refused_on_another_device_than_the_tensors(dfv, monkeypatch):
    """The library launches on the current device: tensors, stream and current device have to be the same one's."""
    monkeypatch.setattr(dfv, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(dfv, "_current_device", lambda: 1, raising=False)
    assert dfv._on(None, 1) == 101 and dfv._on(Queue(1, 7), 1) == 7
    for stream, index in ((None, 0), (Queue(0, 7), 0), (Queue(1, 7), 0), (Queue(0, 7), 1)):
        with pytest.raises(ValueError, match="device"):
            dfv._on(stream, index)
    assert dfv._on(None, -1) == 0  # host tensors: refused by the call itself
