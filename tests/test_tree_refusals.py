"""What the tree-verify entry points refuse, without a GPU: the C ABI with made-up addresses, the binding with CPU
tensors.  Nothing here is launched."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def dfv():
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


CACHE = dict(n_layers=4, n_pages=100, page_size=16, n_kv_heads=4, head_dim=128, dtype=1, max_seqs=8, max_pages=64,
             k=0x10000, v=0x20000, stride_layer=100 * 8192, stride_page=8192, stride_head=2048, stride_token=128,
             page_table=0x30000, lens=0x40000, refs=0x50000, err=0x60000)
TREE = dict(n_seqs=2, n_rows=20, max_nodes=16, seq=None, row_off=0x70000, mask=0x80000)


def cache(dfv, **kw):
    return ctypes.byref(dfv.CCache(**{**CACHE, **kw}))


def tree(dfv, **kw):
    return ctypes.byref(dfv.CTree(**{**TREE, **kw}))


BAD_CACHE = [(dict(n_layers=0), INVALID), (dict(n_pages=0), INVALID), (dict(n_kv_heads=-1), INVALID), (dict(dtype=0), UNSUPPORTED),
             (dict(dtype=2), UNSUPPORTED), (dict(page_size=4), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
             (dict(page_size=512), UNSUPPORTED), (dict(head_dim=72), UNSUPPORTED), (dict(head_dim=272), UNSUPPORTED),
             (dict(k=0), INVALID), (dict(v=0x20008), INVALID), (dict(stride_page=-8), INVALID), (dict(stride_head=4), INVALID),
             (dict(stride_token=64), INVALID), (dict(page_table=0), INVALID), (dict(lens=0), INVALID),
             (dict(page_table=0x30002), INVALID), (dict(lens=0x40001), INVALID), (dict(refs=0x50002), INVALID), (dict(err=0x60001), INVALID),
             (dict(max_seqs=0), INVALID), (dict(max_pages=1 << 28), UNSUPPORTED), (dict(n_kv_heads=2000), UNSUPPORTED)]
BAD_TREE = [(dict(n_seqs=0), INVALID), (dict(n_seqs=1025), INVALID), (dict(n_rows=0), INVALID), (dict(max_nodes=0), INVALID),
            (dict(max_nodes=65), INVALID), (dict(row_off=0), INVALID), (dict(row_off=0x70002), INVALID), (dict(seq=0x70003), INVALID), (dict(mask=0x80004), INVALID), (dict(n_rows=1 << 20), INVALID)]


def rope(dfv, c=None, t=None, **kw):
    a = dict(layer=0, heads=32, rot=128, inter=0, scale=1.0, turns=0x1000, q=0x2000, qr=4096, qh=128, k=0x3000, kr=512, kh=128,
             v=0x4000, vr=512, vh=128, pos=0x5000, o=0x6000, orow=4096, oh=128)
    a.update(kw)
    return dfv.lib().dfv_rope_append(c or cache(dfv), a["layer"], t or tree(dfv), a["heads"], a["rot"], a["inter"], a["scale"],
                                     a["turns"], a["q"], a["qr"], a["qh"], a["k"], a["kr"], a["kh"], a["v"], a["vr"], a["vh"],
                                     a["pos"], a["o"], a["orow"], a["oh"], None)


def attn(dfv, c=None, t=None, **kw):
    a = dict(layer=0, heads=32, scale=0.1, q=0x2000, qr=4096, qh=128, o=0x6000, orow=4096, oh=128, lse=None, ws=0x9000, n=1 << 32)
    a.update(kw)
    return dfv.lib().dfv_tree_attention(c or cache(dfv), a["layer"], t or tree(dfv), a["heads"], a["scale"], a["q"], a["qr"],
                                        a["qh"], a["o"], a["orow"], a["oh"], a["lse"], a["ws"], a["n"], None)


def logits(dfv, t=None, rules=None, **kw):
    a = dict(x=0x2000, row=1000, dtype=1, V=1000, tokens=0x3000, out=0x4000, out_row=1000, best=0x5000, ws=0x9000, n=1 << 20)
    a.update(kw)
    r = dict(hist=0x1000, hist_len=0x1100, hist_row=50, repetition=0x1200)
    r.update(rules or {})
    return dfv.lib().dfv_logits_process(a["x"], a["row"], a["dtype"], a["V"], t or tree(dfv), a["tokens"],
                                        ctypes.byref(dfv.CRules(**r)), a["out"], a["out_row"], a["best"], a["ws"], a["n"], None)


def commit(dfv, c=None, t=None, **kw):
    a = dict(path=0x1000, row=16, tau=0x2000, new=0x3000, ws=0x9000, n=1 << 20)
    a.update(kw)
    return dfv.lib().dfv_cache_commit(c or cache(dfv), t or tree(dfv), a["path"], a["row"], a["tau"], a["new"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_caches(dfv, kw, status):
    L = dfv.lib()
    c = cache(dfv, **kw)
    assert rope(dfv, c) == status and attn(dfv, c) == status and commit(dfv, c) == status
    assert L.dfv_last_error_detail()
    assert L.dfv_cache_copy_pages(c, 0x1000, 0x2000, 3, None) == status
    assert L.dfv_pages_reserve(c, 0x1000, 0x2000, 3, 0x9000, 1 << 20, None) == status
    assert L.dfv_pages_fork(c, 0x1000, 0x2000, 3, 0x9000, 1 << 20, None) == status
    assert L.dfv_pages_free(c, 0x1000, 3, None) == status
    assert L.dfv_cache_workspace_size(c) == 0
    assert L.dfv_tree_attention_workspace_size(c, tree(dfv), 32) == 0


@pytest.mark.parametrize("kw,status", BAD_TREE)
def test_trees(dfv, kw, status):
    t = tree(dfv, **kw)
    assert rope(dfv, t=t) == status and attn(dfv, t=t) == status and commit(dfv, t=t) == status and logits(dfv, t=t) == status
    assert dfv.lib().dfv_accept_tree(t, 0x1000, 0x2000, 0x3000, 64, 0x4000, None) == status
    assert dfv.lib().dfv_tree_attention_workspace_size(cache(dfv), t, 32) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(layer=-1), INVALID), (dict(layer=4), INVALID), (dict(heads=0), INVALID), (dict(rot=0), UNSUPPORTED),
    (dict(rot=24), UNSUPPORTED), (dict(rot=144), UNSUPPORTED), (dict(inter=2), INVALID), (dict(scale=math.inf), INVALID),
    (dict(scale=math.nan), INVALID), (dict(turns=0), INVALID), (dict(turns=0x1004), INVALID), (dict(pos=0), INVALID), (dict(pos=0x5002), INVALID),
    (dict(q=0), INVALID), (dict(k=0x3002), INVALID), (dict(v=0), INVALID), (dict(o=0), INVALID), (dict(qr=-8), INVALID),
    (dict(kh=12), INVALID), (dict(vr=4), INVALID), (dict(orow=1), INVALID), (dict(o=0x2000, orow=8192), INVALID)])
def test_rope(dfv, kw, status):
    assert rope(dfv, **kw) == status
    assert dfv.lib().dfv_last_error_detail()


@pytest.mark.parametrize("args,status", [
    ((24, 1e4, 0, 1, 1, 0, 1), UNSUPPORTED), ((0, 1e4, 0, 1, 1, 0, 1), UNSUPPORTED), ((272, 1e4, 0, 1, 1, 0, 1), UNSUPPORTED),
    ((64, 1.0, 0, 1, 1, 0, 1), INVALID), ((64, math.nan, 0, 1, 1, 0, 1), INVALID), ((64, math.inf, 0, 1, 1, 0, 1), INVALID),
    ((64, 1e4, 4, 1, 1, 0, 1), UNSUPPORTED), ((64, 1e4, -1, 1, 1, 0, 1), UNSUPPORTED), ((64, 1e4, 1, 0.5, 1, 0, 1), INVALID),
    ((64, 1e4, 2, math.nan, 1, 0, 1), INVALID), ((64, 1e4, 3, 2, 0, 1, 32), INVALID), ((64, 1e4, 3, 2, 4096, 32, 1), INVALID),
    ((64, 1e4, 3, 2, 4096, -1, 1), INVALID)])
def test_rope_tables(dfv, args, status):
    assert dfv.lib().dfv_rope_table(*args, (ctypes.c_uint64 * 128)()) == status


def test_rope_table_values(dfv):
    """The turn per position as a 64-bit fraction: within 2^-51 of the formula relatively, and half a unit."""
    for kind, (name, factor) in enumerate([("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("bands", 16.0)]):
        t = (ctypes.c_uint64 * 64)()
        assert dfv.lib().dfv_rope_table(128, 5e5, kind, factor, 8192.0, 1.0, 4.0, t) == 0
        theta = 5e5 * (8.0 ** (128 / 126) if name == "ntk" else 1)
        for i in range(64):
            f = theta ** (-2 * i / 128)
            if name == "linear":
                f /= 4
            if name == "bands":
                g = min(1.0, max(0.0, (8192 * f / (2 * math.pi) - 1) / 3))
                f = (1 - g) * f / 16 + g * f
            want = f / (2 * math.pi) * 2.0 ** 64
            assert abs(t[i] - want) <= want * 2.0 ** -49 + 0.5
    assert dfv.lib().dfv_rope_table(64, 1e4, 0, 1.0, 1.0, 0.0, 1.0, None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(layer=4), INVALID), (dict(heads=30), INVALID), (dict(heads=0), INVALID), (dict(heads=68), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID), (dict(q=0), INVALID),
    (dict(q=0x2004), INVALID), (dict(o=0), INVALID), (dict(o=0x2000), INVALID), (dict(qr=3), INVALID), (dict(oh=-8), INVALID), (dict(lse=0x7002), INVALID),
    (dict(ws=0), WORKSPACE), (dict(ws=0x9010), WORKSPACE), (dict(n=255), WORKSPACE)])
def test_attention(dfv, kw, status):
    assert attn(dfv, **kw) == status
    assert dfv.lib().dfv_last_error_detail()


@pytest.mark.parametrize("dim", [16, 96, 256])
def test_attention_head_sizes(dfv, dim):
    c = cache(dfv, head_dim=dim, stride_token=256, stride_head=4096, stride_page=16384)
    assert attn(dfv, c) == UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=4), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(V=0), INVALID), (dict(V=1 << 29), INVALID),
    (dict(best=0x5002), INVALID), (dict(tokens=0x3001), INVALID), (dict(rules=dict(bias=0x102)), INVALID),
    (dict(rules=dict(allowed=0x101)), INVALID), (dict(rules=dict(hist=0x1002)), INVALID),
    (dict(x=0), INVALID), (dict(x=0x2001), INVALID), (dict(out=0x4001), INVALID), (dict(dtype=0, x=0x2002), INVALID),
    (dict(out=None, best=None), INVALID), (dict(row=999), INVALID), (dict(out_row=10), INVALID),
    (dict(out=0x2000, out_row=1200), INVALID), (dict(tokens=None), INVALID), (dict(rules=dict(hist_len=None)), INVALID),
    (dict(rules=dict(hist_row=-1)), INVALID), (dict(rules=dict(hist_row=1 << 24)), UNSUPPORTED), (dict(rules=dict(bias=0x100, bias_row=999)), INVALID),
    (dict(rules=dict(allowed=0x100, allowed_row=31)), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=0x9080), WORKSPACE),
    (dict(n=600), WORKSPACE)])
def test_logits(dfv, kw, status):
    assert logits(dfv, **kw) == status
    assert dfv.lib().dfv_last_error_detail()


def test_logits_without_rules(dfv):
    assert dfv.lib().dfv_logits_process(0x2000, 1000, 1, 1000, tree(dfv), None, None, 0x4000, 1000, None, 0x9000, 1 << 20, None) == INVALID
    assert dfv.lib().dfv_logits_workspace_size(0) == 0
    assert dfv.lib().dfv_logits_workspace_size((64 << 10) + 1) == 0


@pytest.mark.parametrize("kw,status", [(dict(path=0), INVALID), (dict(tau=0), INVALID), (dict(new=0), INVALID), (dict(new=0x3002), INVALID), (dict(row=15), INVALID),
                                       (dict(ws=0), WORKSPACE), (dict(ws=0x9001), WORKSPACE), (dict(n=4096), WORKSPACE)])
def test_commit(dfv, kw, status):
    assert commit(dfv, **kw) == status


def test_page_lists(dfv):
    L, c = dfv.lib(), cache(dfv)
    bare = cache(dfv, refs=None)
    for n in (0, -1, 1025):
        assert L.dfv_pages_reserve(c, 0x1000, 0x2000, n, 0x9000, 1 << 20, None) == INVALID
        assert L.dfv_pages_fork(c, 0x1000, 0x2000, n, 0x9000, 1 << 20, None) == INVALID
        assert L.dfv_pages_free(c, 0x1000, n, None) == INVALID
    assert L.dfv_cache_copy_pages(c, 0x1000, 0x2000, 0, None) == INVALID
    assert L.dfv_cache_copy_pages(c, None, 0x2000, 1, None) == INVALID
    assert L.dfv_pages_reserve(c, None, 0x2000, 1, 0x9000, 1 << 20, None) == INVALID
    assert L.dfv_pages_fork(c, 0x1000, None, 1, 0x9000, 1 << 20, None) == INVALID
    assert L.dfv_pages_free(c, None, 1, None) == INVALID
    assert L.dfv_pages_free(c, 0x1002, 1, None) == INVALID
    assert L.dfv_cache_copy_pages(c, 0x1000, 0x2001, 1, None) == INVALID
    assert L.dfv_pages_reserve(bare, 0x1000, 0x2000, 1, 0x9000, 1 << 20, None) == INVALID
    assert L.dfv_pages_fork(bare, 0x1000, 0x2000, 1, 0x9000, 1 << 20, None) == INVALID
    assert L.dfv_pages_free(bare, 0x1000, 1, None) == INVALID
    assert L.dfv_pages_reserve(c, 0x1000, 0x2000, 1, 0x9000, 100, None) == WORKSPACE
    assert L.dfv_pages_fork(c, 0x1000, 0x2000, 1, None, 1 << 20, None) == WORKSPACE
    for a in ((0, 0x2000, 0x3000, 0x4000), (0x1000, 0, 0x3000, 0x4000), (0x1000, 0x2000, 0, 0x4000), (0x1000, 0x2000, 0x3000, 0)):
        assert L.dfv_accept_tree(tree(dfv), a[0], a[1], a[2], 64, a[3], None) == INVALID
    assert L.dfv_accept_tree(tree(dfv), 0x1000, 0x2000, 0x3000, 15, 0x4000, None) == INVALID


# ---------------------------------------------------------------- the binding
def kv(dtype=torch.bfloat16, **kw):
    return torch.zeros(2, 5, 2, 16, 64, dtype=dtype), torch.zeros(2, 5, 2, 16, 64, dtype=dtype)


def test_binding_caches(dfv):
    k, v = kv()
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    c = dfv.KVCache(k, v, t, n)
    assert c.errors() == 0 and (c.c.stride_layer, c.c.stride_page, c.c.stride_head, c.c.stride_token) == k.stride()[:4]
    assert dfv.cache_workspace_size(c) > 0
    with pytest.raises(TypeError):
        dfv.KVCache(k.float(), v.float(), t, n)
    for args in ((k[0], v[0], t, n), (k, v[:1], t, n), (k, v.half(), t, n), (k, v, t[0], n), (k, v, t, n[:2]), (k, v, t.T, n),
                 (k.transpose(3, 4), v.transpose(3, 4), t, n), (k, v.permute(0, 1, 3, 2, 4).contiguous().permute(0, 1, 3, 2, 4), t, n)):
        with pytest.raises(ValueError):
            dfv.KVCache(*args)
    with pytest.raises(TypeError):
        dfv.KVCache(k, v, t.long(), n)
    with pytest.raises(ValueError):
        dfv.KVCache(k, v, t, n, refs=torch.zeros(4, dtype=torch.int32))


def test_binding_trees_and_rules(dfv):
    off = torch.tensor([0, 3, 5], dtype=torch.int32)
    dfv.TreeBatch(off, 5, 3, mask=torch.zeros(5, dtype=torch.int64))
    for bad in (dict(mask=torch.zeros(4, dtype=torch.int64)), dict(seq=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            dfv.TreeBatch(off, 5, 3, **bad)
    with pytest.raises(TypeError):
        dfv.TreeBatch(off, 5, 3, mask=torch.zeros(5, dtype=torch.int32))
    with pytest.raises(TypeError):
        dfv.TreeBatch(off.long(), 5, 3)
    with pytest.raises(ValueError):
        dfv.TreeBatch(off[:1], 5, 3)
    h = torch.zeros(2, 7, dtype=torch.int32)
    with pytest.raises(ValueError):
        dfv.LogitRules(hist=h)
    with pytest.raises(ValueError):
        dfv.LogitRules(hist=h, hist_len=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        dfv.LogitRules(repetition=torch.ones(2), presence=torch.ones(3))
    with pytest.raises(TypeError):
        dfv.LogitRules(bias=torch.zeros(1, 10, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        dfv.Rope(128, scaling="cubic", device="cpu")
    with pytest.raises(dfv.DfvError):
        dfv.Rope(128, rot_dim=24, device="cpu")
    assert dfv.Rope(128, scaling="bands", factor=math.e, device="cpu").scale == pytest.approx(1.1)


def test_binding_arguments(dfv):
    k, v = kv()
    c = dfv.KVCache(k, v, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    t = dfv.TreeBatch(torch.tensor([0, 3, 5], dtype=torch.int32), 5, 3)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    ws = torch.zeros(4096, dtype=torch.uint8)
    pos = torch.zeros(5, dtype=torch.int32)
    r = dfv.Rope(64, device="cpu")
    for bad in (q[:4], q[..., :32], q.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            dfv.tree_attention(c, 0, t, bad, ws)
        with pytest.raises(ValueError):
            dfv.rope_append(c, 0, t, r, bad, q[:, :2], q[:, :2], pos)
    with pytest.raises(TypeError):
        dfv.tree_attention(c, 0, t, q.half(), ws)
    with pytest.raises(TypeError):
        dfv.tree_attention(c, 0, t, q, ws, lse=torch.zeros(5, 4, dtype=torch.float64))
    with pytest.raises(ValueError):
        dfv.rope_append(c, 0, t, dfv.Rope(128, device="cpu"), q, q[:, :2], q[:, :2], pos)
    with pytest.raises(TypeError):
        dfv.rope_append(c, 0, t, r, q, q[:, :2], q[:, :2], pos.long())
    x = torch.zeros(5, 100, dtype=torch.bfloat16)
    rules = dfv.LogitRules(bias=torch.zeros(1, 99))
    with pytest.raises(ValueError):
        dfv.logits_process(x, t, None, rules, ws)
    with pytest.raises(ValueError):
        dfv.logits_process(x[:4], t, None, dfv.LogitRules(), ws)
    with pytest.raises(ValueError):
        dfv.logits_process(x, t, None, dfv.LogitRules(repetition=torch.ones(3)), ws)
    with pytest.raises(ValueError):
        dfv.logits_process(x, t, None, dfv.LogitRules(allowed=torch.zeros(2, 4, dtype=torch.int32)), ws)
    with pytest.raises(TypeError):
        dfv.accept_tree(t, pos.long(), pos)
    with pytest.raises(ValueError):
        dfv.cache_commit(c, t, torch.zeros(3, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), ws)
    with pytest.raises(ValueError):
        dfv.pages_fork(c, pos[:2], pos[:3], ws)
