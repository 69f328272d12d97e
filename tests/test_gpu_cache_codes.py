"""A cache in codes through the calls that move its rows: commits, copies and forks take the exponents along."""
from __future__ import annotations

import random

import pytest
import torch

from tests._prompt_util import E4M3

pytestmark = pytest.mark.gpu


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


def filled(dfv, lens, room, kv, dim, page, layers, layout, seqs=None, seed=0):
    """Sequences of lens[s] tokens with room for `room` more, every byte of the cache random."""
    rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
    seqs = seqs or len(lens)
    need = [-(-(a + room) // page) for a in lens]
    pages = sum(need) + seqs + 2
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.full((seqs, max(need) + 1), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    for s, m in enumerate(need):
        mine = [order.pop() for _ in range(m)]
        table[s, :m] = torch.tensor(mine, dtype=torch.int32)
        refs[mine] = 1
    shape = (2, layers, pages, kv, page, dim) if layout == "head" else (2, layers, pages, page, kv, dim)
    raw = torch.randint(0, 256, shape, generator=g).to(torch.uint8).cuda()
    exp = torch.randint(0, 256, (2, layers, pages, kv, page), generator=g).to(torch.uint8).cuda()
    kv_ = raw.view(E4M3)
    k, v = (kv_[0], kv_[1]) if layout == "head" else (kv_[0].transpose(2, 3), kv_[1].transpose(2, 3))
    return dfv.KVCache(k, v, table.cuda(), i32(lens + [0] * (seqs - len(lens))), refs=refs.cuda(), k_exp=exp[0], v_exp=exp[1])


def everything(cache):
    return [x.cpu().clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_exp, cache.v_exp)]


@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("page,dim,kv", [(8, 64, 1), (16, 128, 4), (64, 16, 3), (256, 256, 70)])
def test_commit(dfv, layout, page, dim, kv):
    rng = random.Random(page)
    lens, nodes = [0, 5, page, page - 1, 2 * page - 1], [64, 1, 17, 0, 63]
    layers = 1 if kv > 8 else 3
    cache = filled(dfv, lens, 64, kv, dim, page, layers, layout, seed=page)
    off = [0]
    for n in nodes:
        off.append(off[-1] + n)
    tree = dfv.TreeBatch(i32(off), off[-1], 64)
    ws = dfv.alloc_workspace(dfv.cache_workspace_size(cache))
    paths = [sorted(rng.sample(range(n), rng.randint(0, n))) for n in nodes]
    was = everything(cache)
    dfv.cache_commit(cache, tree, i32([p + [-1] * (64 - len(p)) for p in paths]), i32([len(p) for p in paths]), ws)
    want = [x.clone() for x in was]
    for s, p in enumerate(paths):
        for j, x in enumerate(p):
            a, b = lens[s] + x, lens[s] + j
            pa, pb = int(cache.page_table[s, a // page]), int(cache.page_table[s, b // page])
            for w, o in zip(want, was):
                w[:, pb, :, b % page] = o[:, pa, :, a % page]
    assert all(torch.equal(a, b) for a, b in zip(everything(cache), want))
    assert cache.lens.tolist() == [a + len(p) for a, p in zip(lens, paths)] and cache.errors() == 0


@pytest.mark.parametrize("layout", ["head", "token"])
def test_copies_and_forks(dfv, layout):
    page, lens = 16, [37, 16, 5]
    cache = filled(dfv, lens, 0, 3, 64, page, 2, layout, seqs=6, seed=3)
    was = everything(cache)
    dfv.cache_copy_pages(cache, i32([1, 4]), i32([2, 0]))
    for x in was:
        x[:, 2], x[:, 0] = x[:, 1].clone(), x[:, 4].clone()
    assert all(torch.equal(a, b) for a, b in zip(everything(cache), was))
    ws = dfv.alloc_workspace(dfv.cache_workspace_size(cache))
    dfv.pages_fork(cache, i32([0, 1, 2]), i32([3, 4, 5]), ws)
    now = everything(cache)
    table = cache.page_table.cpu()
    for s, n in enumerate(lens):
        for i in range(n):
            a, b = int(table[s, i // page]), int(table[s + 3, i // page])
            assert a == b or i // page == n // page
            for x, o in zip(now, was):
                assert torch.equal(x[:, b, :, i % page], o[:, a, :, i % page])
    copies = [int(table[s + 3, n // page]) for s, n in enumerate(lens) if n % page]
    for x, o in zip(now, was):  # nothing but the used rows of the copied pages changed
        for s, n in enumerate(lens):
            if n % page:
                x[:, int(table[s + 3, n // page]), :, :n % page] = o[:, int(table[s + 3, n // page]), :, :n % page]
        assert torch.equal(x, o)
    assert len(set(copies)) == 2 and cache.errors() == 0
