"""Checks of the tree-verify entry points on the host, one by one (CPU; nothing here is launched)."""
from __future__ import annotations

import ctypes

import pytest

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def dfv():
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


def tree(dfv, **kw):
    a = dict(n_seqs=2, n_rows=20, max_nodes=16, seq=None, row_off=0x70000, mask=0x80000)
    return ctypes.byref(dfv.CTree(**{**a, **kw}))


def logits(dfv, rules, V=1000, tokens=0x3000):
    return dfv.lib().dfv_logits_process(0x2000, V, 1, V, tree(dfv), tokens, ctypes.byref(dfv.CRules(**rules)), 0x4000, V, 0x5000,
                                        0x9000, 1 << 30, None)


@pytest.mark.parametrize("rules", [dict(hist=0x1000, hist_row=50), dict(hist=0x1000, hist_row=50, bias=0x1200),
                                   dict(hist=0x1000, hist_row=50, prompt_len=0x1300), dict(hist=0x1000, hist_len=0x1100, hist_row=-1)])
def test_a_history_needs_its_lengths_with_penalties_and_without(dfv, rules):
    assert logits(dfv, rules) == INVALID
    assert b"hist" in dfv.lib().dfv_last_error_detail()


def cache(dfv, **kw):
    a = dict(n_layers=4, n_pages=100, page_size=16, n_kv_heads=4, head_dim=128, dtype=1, max_seqs=8, max_pages=64, k=0x10000,
             v=0x20000, stride_layer=100 * 8192, stride_page=8192, stride_head=2048, stride_token=128, page_table=0x30000,
             lens=0x40000, refs=0x50000, err=0x60000)
    return ctypes.byref(dfv.CCache(**{**a, **kw}))


@pytest.mark.parametrize("group", range(1, 17))
@pytest.mark.parametrize("kv,dim,seqs", [(1, 128, 1), (4, 64, 33)])
def test_an_attention_workspace_serves_smaller_trees(dfv, group, kv, dim, seqs):
    """The size for trees of up to max_nodes nodes is enough for any smaller tree, also of fewer sequences."""
    c = cache(dfv, n_kv_heads=kv, head_dim=dim)
    size = lambda n, s: dfv.lib().dfv_tree_attention_workspace_size(c, tree(dfv, n_seqs=s, max_nodes=n), kv * group)  # noqa: E731
    sizes = [size(n, seqs) for n in range(1, 65)]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    assert all(size(n, max(1, seqs // 2)) <= sizes[n - 1] for n in range(1, 65))


def test_what_calls_leave_in_a_workspace_lies_behind_the_counters_of_all(dfv):
    """Counters that have to be zero come first, at the same places for every call: the other calls' workspaces hold
    those of the largest logits call in front."""
    L = dfv.lib()
    counters = L.dfv_logits_workspace_size(64 * 1024)
    assert L.dfv_logits_workspace_size(1) < counters
    assert L.dfv_cache_workspace_size(cache(dfv, n_pages=1)) > counters
    assert L.dfv_tree_attention_workspace_size(cache(dfv, n_kv_heads=1, head_dim=64), tree(dfv, n_seqs=1, max_nodes=1), 1) > counters


@pytest.mark.parametrize("V", [65535 * 4096 + 1, 1 << 28])
def test_vocabularies_beyond_the_slices_of_a_launch(dfv, V):
    assert logits(dfv, {}, V=V) == INVALID
    assert b"V=" in dfv.lib().dfv_last_error_detail()


def test_reservations_whose_missing_entries_cannot_be_counted(dfv):
    """The kernel sums the missing table entries of all sequences in 32 bits; n_new is device data and may ask for all."""
    L = dfv.lib()
    c = cache(dfv, page_size=8, stride_page=4096, stride_head=1024, max_pages=1 << 27)
    assert L.dfv_pages_reserve(c, 0x1000, 0x2000, 16, 0x9000, 1 << 30, None) == UNSUPPORTED
    assert b"table" in L.dfv_last_error_detail()


def test_a_rotary_plan_of_no_elements_is_refused(dfv):
    """rot_dim 0 is not "the whole head": that is None."""
    assert dfv.Rope(128, device="cpu").rot_dim == 128 and dfv.Rope(128, rot_dim=64, device="cpu").rot_dim == 64
    with pytest.raises(dfv.DfvError, match="rot_dim 0"):
        dfv.Rope(128, rot_dim=0, device="cpu")


def test_a_rotary_plan_from_frequencies(dfv):
    """Frequencies of the caller's own, as a whole turn's 64-bit fractions: within half a unit and the roundings of the
    quotient by 2 pi (2^-52 relatively)."""
    import math
    from fractions import Fraction
    f = [1.0, 0.37, 1e-3, 2.5e-7, 0.0, 3.0, -0.5, 7.0]
    r = dfv.Rope(64, rot_dim=16, freqs=f, scale=1.1, device="cpu")
    assert r.rot_dim == 16 and r.scale == 1.1
    for got, x in zip(r.turns.tolist(), f):
        d = (Fraction(got, 1 << 64) - Fraction(x) / Fraction(2 * math.pi)) % 1
        assert min(d, 1 - d) <= Fraction(1, 1 << 65) + abs(Fraction(x)) / (1 << 52)
    plain = dfv.Rope(64, theta=1e4, device="cpu").turns
    own = dfv.Rope(64, freqs=[1e4 ** (-2 * i / 64) for i in range(32)], device="cpu")
    assert own.scale == 1.0 and all(abs(a - b) <= 1 + abs(b) * 2.0 ** -50 for a, b in zip(own.turns.tolist(), plain.tolist()))
    for bad in (dict(freqs=f), dict(freqs=f[:7], rot_dim=16), dict(freqs=f[:7] + [math.inf], rot_dim=16),
                dict(freqs=f, rot_dim=16, scaling="linear", factor=2.0)):
        with pytest.raises(ValueError):
            dfv.Rope(64, device="cpu", **bad)
    with pytest.raises(dfv.DfvError):
        dfv.Rope(64, freqs=[1.0] * 12, rot_dim=24, device="cpu")
