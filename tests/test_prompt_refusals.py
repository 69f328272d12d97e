"""What the prompt calls and caches in codes refuse, without a GPU: the C ABI with made-up addresses, the binding with CPU
tensors.  Nothing here is launched."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dfv():
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


CACHE = dict(n_layers=4, n_pages=100, page_size=16, n_kv_heads=4, head_dim=128, dtype=5, max_seqs=8, max_pages=64,
             k=0x10000, v=0x20000, stride_layer=100 * 8192, stride_page=8192, stride_head=2048, stride_token=128,
             page_table=0x30000, lens=0x40000, refs=0x50000, err=0x60000, k_exp=0x70000, v_exp=0x80000)
ROWS = dict(n_seqs=2, n_rows=2000, max_rows=1600, seq=None, row_off=0x70000)


def cache(dfv, **kw):
    return ctypes.byref(dfv.CCache(**{**CACHE, **kw}))


def rows(dfv, **kw):
    return ctypes.byref(dfv.CRows(**{**ROWS, **kw}))


def append(dfv, c=None, r=None, **kw):
    a = dict(layer=0, heads=32, qg=0x500, kg=0x600, eps=1e-6, rot=128, inter=0, scale=1.0, turns=0x1000, q=0x2000, qr=4096, qh=128,
             k=0x3000, kr=512, kh=128, v=0x4000, vr=512, vh=128, pos=0x5000, o=0x6000, orow=4096, oh=128, ko=None, kor=512, koh=128)
    a.update(kw)
    return dfv.lib().dfv_norm_rope_append(c or cache(dfv), a["layer"], r or rows(dfv), a["heads"], a["qg"], a["kg"], a["eps"], a["rot"],
                                          a["inter"], a["scale"], a["turns"], a["q"], a["qr"], a["qh"], a["k"], a["kr"], a["kh"],
                                          a["v"], a["vr"], a["vh"], a["pos"], a["o"], a["orow"], a["oh"], a["ko"], a["kor"], a["koh"], None)


def read(dfv, c=None, r=None, **kw):
    a = dict(layer=0, k=0x3000, kr=512, kh=128, v=0x4000, vr=512, vh=128)
    a.update(kw)
    return dfv.lib().dfv_cache_read(c or cache(dfv), a["layer"], r or rows(dfv), a["k"], a["kr"], a["kh"], a["v"], a["vr"], a["vh"], None)


def prompt(dfv, r=None, keys=None, **kw):
    a = dict(dtype=1, heads=32, kv=4, dim=128, scale=0.1, q=0x2000, qr=4096, qh=128, k=0x3000, kr=512, kh=128, v=0x4000, vr=512, vh=128,
             o=0x6000, orow=4096, oh=128, lse=None, err=None, ws=0x9000, n=1 << 32)
    a.update(kw)
    return dfv.lib().dfv_prompt_attention(a["dtype"], r or rows(dfv), keys, a["heads"], a["kv"], a["dim"], a["scale"], a["q"], a["qr"],
                                          a["qh"], a["k"], a["kr"], a["kh"], a["v"], a["vr"], a["vh"], a["o"], a["orow"], a["oh"],
                                          a["lse"], a["err"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), UNSUPPORTED), (dict(dtype=6), UNSUPPORTED), (dict(k_exp=0), INVALID), (dict(v_exp=0), INVALID), (dict(k_exp=0x70002), INVALID),
    (dict(v_exp=0x80001), INVALID), (dict(stride_page=8192 + 8), INVALID), (dict(stride_head=2056), INVALID), (dict(stride_token=136), INVALID),
    (dict(stride_layer=8), INVALID), (dict(page_size=24), UNSUPPORTED), (dict(k=0x10008), INVALID), (dict(lens=0), INVALID), (dict(n_pages=0), INVALID)])
def test_caches(dfv, kw, status):
    c, L = cache(dfv, **kw), dfv.lib()
    assert append(dfv, c) == status and read(dfv, c) == status
    assert L.dfv_last_error_detail()
    assert L.dfv_cache_copy_pages(c, 0x1000, 0x2000, 3, None) == status
    assert L.dfv_pages_fork(c, 0x1000, 0x2000, 3, 0x9000, 1 << 20, None) == status
    assert L.dfv_cache_workspace_size(c) == 0


def test_caches_in_16_bits_need_no_exponents(dfv):
    """The two fields behind `err` are read for codes only: a caller's shorter struct stays good."""
    assert dfv.lib().dfv_cache_workspace_size(cache(dfv, dtype=1, k_exp=1, v_exp=3)) > 0
    assert read(dfv, cache(dfv, dtype=1, k_exp=1, v_exp=3), k=0, v=0) == INVALID  # its own refusal
    assert dfv.CCache.k_exp.offset == dfv.CCache.err.offset + 8 and dfv.CCache.v_exp.offset == dfv.CCache.err.offset + 16


@pytest.mark.parametrize("kw,status", [
    (dict(n_seqs=0), INVALID), (dict(n_seqs=1025), INVALID), (dict(n_rows=0), INVALID), (dict(n_rows=(1 << 24) + 1), INVALID),
    (dict(max_rows=0), INVALID), (dict(max_rows=(1 << 24) + 1), INVALID), (dict(row_off=0), INVALID), (dict(row_off=0x70002), INVALID),
    (dict(seq=0x1001), INVALID)])
def test_rows(dfv, kw, status):
    r = rows(dfv, **kw)
    assert append(dfv, r=r) == status and read(dfv, r=r) == status and prompt(dfv, r) == status and prompt(dfv, keys=r) == status
    assert dfv.lib().dfv_prompt_attention_workspace_size(r, 32, 4, 128) == 0
    assert append(dfv, r=None, c=None, layer=9) == INVALID
    assert dfv.lib().dfv_cache_read(cache(dfv), 0, None, 0x3000, 512, 128, 0x4000, 512, 128, None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(layer=-1), INVALID), (dict(layer=4), INVALID), (dict(heads=0), INVALID), (dict(rot=0), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
    (dict(rot=144), UNSUPPORTED), (dict(inter=2), INVALID), (dict(scale=math.inf), INVALID), (dict(turns=0), INVALID), (dict(turns=0x1004), INVALID),
    (dict(pos=0), INVALID), (dict(pos=0x5002), INVALID), (dict(q=0), INVALID), (dict(k=0x3002), INVALID), (dict(v=0), INVALID), (dict(o=0), INVALID),
    (dict(qr=-8), INVALID), (dict(kh=12), INVALID), (dict(vr=4), INVALID), (dict(orow=1), INVALID), (dict(o=0x2000, orow=8192), INVALID),
    (dict(qg=0x508), INVALID), (dict(kg=0x602), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID), (dict(ko=0x7004), INVALID),
    (dict(ko=0x7000, kor=4), INVALID), (dict(ko=0x7000, koh=-8), INVALID), (dict(ko=0x3000, kor=1024), INVALID), (dict(ko=0x2000), INVALID),
    (dict(ko=0x4000), INVALID), (dict(ko=0x6000), INVALID)])
def test_append(dfv, kw, status):
    assert append(dfv, **kw) == status
    assert dfv.lib().dfv_last_error_detail()


@pytest.mark.parametrize("kw,status", [
    (dict(layer=-1), INVALID), (dict(layer=4), INVALID), (dict(k=0, v=0), INVALID), (dict(k=0x3008), INVALID), (dict(v=0x4004), INVALID),
    (dict(kr=4), INVALID), (dict(kh=-8), INVALID), (dict(vr=1), INVALID), (dict(vh=9), INVALID)])
def test_read(dfv, kw, status):
    assert read(dfv, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED), (dict(heads=30), INVALID), (dict(heads=0), INVALID), (dict(kv=0), INVALID),
    (dict(kv=2000, heads=2000), INVALID), (dict(heads=68), UNSUPPORTED), (dict(dim=96), UNSUPPORTED), (dict(dim=256), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID), (dict(q=0), INVALID), (dict(q=0x2004), INVALID),
    (dict(k=0), INVALID), (dict(v=0x4008), INVALID), (dict(o=0), INVALID), (dict(o=0x2000), INVALID), (dict(o=0x3000), INVALID), (dict(o=0x4000), INVALID),
    (dict(qr=3), INVALID), (dict(oh=-8), INVALID), (dict(kr=1 << 36), INVALID), (dict(kr=0), UNSUPPORTED), (dict(vh=0), UNSUPPORTED), (dict(qr=0), UNSUPPORTED), (dict(qh=0), UNSUPPORTED),
    (dict(lse=0x7002), INVALID), (dict(err=0x7001), INVALID), (dict(ws=0), WORKSPACE), (dict(ws=0x9010), WORKSPACE), (dict(n=255), WORKSPACE)])
def test_prompt(dfv, kw, status):
    assert prompt(dfv, **kw) == status
    assert dfv.lib().dfv_last_error_detail()


def test_prompt_batches(dfv):
    assert dfv.lib().dfv_prompt_attention(1, None, None, 32, 4, 128, 0.1, 0x2000, 4096, 128, 0x3000, 512, 128, 0x4000, 512, 128, 0x6000, 4096, 128,
                                          None, None, 0x9000, 1 << 32, None) == INVALID
    assert prompt(dfv, keys=rows(dfv, n_seqs=3)) == INVALID
    size = dfv.lib().dfv_prompt_attention_workspace_size
    assert size(rows(dfv), 32, 4, 128) > size(rows(dfv), 32, 4, 64) > 0
    # one workspace serves every batch of a head size
    assert size(rows(dfv, n_seqs=1000, n_rows=1 << 24, max_rows=1 << 24), 32, 4, 128) == size(rows(dfv, n_seqs=1, n_rows=1, max_rows=1), 8, 8, 128)
    assert size(None, 32, 4, 128) == 0 and size(rows(dfv), 32, 5, 128) == 0 and size(rows(dfv), 32, 4, 80) == 0


# ---------------------------------------------------------------- the binding
def test_binding_caches(dfv):
    k, v = (torch.zeros(2, 5, 2, 16, 64).to(E4M3) for _ in range(2))
    e = torch.zeros(2, 5, 2, 16, dtype=torch.uint8)
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    c = dfv.KVCache(k, v, t, n, k_exp=e, v_exp=e)
    assert c.c.dtype == 5 and c.c.k_exp == e.data_ptr()
    for bad in (dict(), dict(k_exp=e), dict(k_exp=e, v_exp=e[..., :8]), dict(k_exp=e, v_exp=e.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            dfv.KVCache(k, v, t, n, **bad)
    with pytest.raises(TypeError):
        dfv.KVCache(k, v, t, n, k_exp=e, v_exp=e.int())
    with pytest.raises(TypeError):
        dfv.KVCache(k.float().to(torch.float8_e5m2), v.float().to(torch.float8_e5m2), t, n, k_exp=e, v_exp=e)
    b = torch.zeros(2, 5, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dfv.KVCache(b, b.clone(), t, n, k_exp=e, v_exp=e)
    c = dfv.KVCache.empty(2, 5, 16, 2, 64, 3, 4, dtype=E4M3, device="cpu")
    assert c.k.dtype == E4M3 and c.k_exp.shape == (2, 5, 2, 16) and not bool(c.k.float().any())


def test_binding_arguments(dfv):
    c = dfv.KVCache.empty(2, 5, 16, 2, 64, 3, 4, dtype=E4M3, device="cpu")
    off = torch.tensor([0, 3, 5], dtype=torch.int32)
    r = dfv.RowBatch(off, 5, 3)
    for bad in (off[:1], off.view(1, 3)):
        with pytest.raises(ValueError):
            dfv.RowBatch(bad, 5, 3)
    with pytest.raises(TypeError):
        dfv.RowBatch(off.long(), 5, 3)
    with pytest.raises(ValueError):
        dfv.RowBatch(off, 5, 3, seq=off)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    kv, pos, rope = q[:, :2], torch.zeros(5, dtype=torch.int32), dfv.Rope(64, device="cpu")
    gain, ws = torch.ones(64, dtype=torch.bfloat16), torch.zeros(4096, dtype=torch.uint8)
    for kw in (dict(q_gain=gain[:32]), dict(k_gain=torch.ones(128, dtype=torch.bfloat16)[::2])):
        with pytest.raises(ValueError):
            dfv.norm_rope_append(c, 0, r, rope, q, kv, kv, pos, **kw)
    with pytest.raises(ValueError):
        dfv.norm_rope_append(c, 0, r, rope, q, kv, kv, pos, k_out=q)
    for kw in (dict(q_gain=gain.float()), dict(out=q.half()), dict(k_out=kv.half())):
        with pytest.raises(TypeError):
            dfv.norm_rope_append(c, 0, r, rope, q, kv, kv, pos, **kw)
    tree = dfv.TreeBatch(off, 5, 3)  # another descriptor
    for call in (lambda: dfv.norm_rope_append(c, 0, tree, rope, q, kv, kv, pos), lambda: dfv.cache_read(c, 0, tree),
                 lambda: dfv.prompt_attention(tree, q, kv, kv, ws), lambda: dfv.prompt_attention(r, q, kv, kv, ws, keys=tree),
                 lambda: dfv.tree_attention(c, 0, r, q, ws), lambda: dfv.rope_append(c, 0, r, rope, q, kv, kv, pos),
                 lambda: dfv.cache_commit(c, r, pos.view(1, 5), pos[:2], ws)):
        with pytest.raises(AttributeError):
            call()
    with pytest.raises(TypeError):  # rows of a cache in codes are bf16
        dfv.norm_rope_append(c, 0, r, rope, q.half(), kv.half(), kv.half(), pos)
    with pytest.raises(ValueError):
        dfv.norm_rope_append(c, 0, r, rope, q[:4], kv, kv, pos)
    with pytest.raises(ValueError):
        dfv.norm_rope_append(c, 0, r, dfv.Rope(128, device="cpu"), q, kv, kv, pos)
    with pytest.raises(TypeError):
        dfv.cache_read(c, 0, r, k=kv.half(), v=kv)
    with pytest.raises(ValueError):
        dfv.cache_read(c, 0, r, k=kv[:4], v=kv)
    with pytest.raises(ValueError):  # host tensors
        dfv.cache_read(c, 0, r)
    with pytest.raises(ValueError):
        dfv.prompt_attention(r, q, kv, kv, ws)
    with pytest.raises(TypeError):
        dfv.prompt_attention(r, q.float(), kv, kv, ws)
    with pytest.raises(TypeError):
        dfv.prompt_attention(r, q, kv.half(), kv, ws)
    with pytest.raises(ValueError):
        dfv.prompt_attention(r, q, kv, kv[:, :1], ws)
    with pytest.raises(ValueError):
        dfv.prompt_attention(r, q, kv, kv, ws, keys=dfv.RowBatch(off, 6, 3))
    with pytest.raises(TypeError):
        dfv.prompt_attention(r, q, kv, kv, ws, err=torch.zeros(1))
