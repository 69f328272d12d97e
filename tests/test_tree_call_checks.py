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
