"""Rotary positions and the append to the paged cache against the formula in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

from tests._tree_util import HALF_STEP, Case

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dfv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_moe_gb300 import build as b
    b.build()
    from speculative_decoding_moe_gb300 import dfv as m
    return m


def frequencies(rot, theta, scaling="none", factor=1.0, original=4096.0, low=1.0, high=32.0):
    out = []
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "bands":
            g = min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low)))
            f = (1 - g) * f / factor + g * f
        out.append(f)
    return out


def turned(x, positions, freqs, inter, scale):
    """(rotated rows, tolerance): half a step for the rounding; the angle is off by 2 pi (2^-32 + 2^-25) for the turn's
    32 bits and their conversion and by position * 2^-50 for the table, sine and cosine by 2 units, products and sum by
    three roundings."""
    r = 2 * len(freqs)
    y, mag = x.double().clone(), x.double().abs().clone()
    for m, f in enumerate(freqs):
        a, b = (2 * m, 2 * m + 1) if inter else (m, m + r // 2)
        ang = positions.double() * f
        c, s = torch.cos(ang)[:, None] * scale, torch.sin(ang)[:, None] * scale
        u, w = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = u * c - w * s, w * c + u * s
        mag[..., a] = mag[..., b] = (u.abs() + w.abs()) * abs(scale)
    far = positions.double().abs()[:, None, None] * 2.0 ** -50
    tol = HALF_STEP[x.dtype] * y.abs() * (1 + 1e-6) + mag * (2 * math.pi * (2.0 ** -32 + 2.0 ** -25) + far + 8 * 2.0 ** -24)
    tol[..., r:] = 0
    if x.dtype == FP:
        tol[..., :r] += 2.0 ** -25
    return y, tol


def step(dfv, c: Case, rot, inter, positions, theta=1e4, scaling="none", factor=1.0, in_place=False, layer=0, scale=None,
         cache=None, tree=None):
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(c.rows, c.H + 2 * c.K, c.D, generator=g).to(c.dtype)
    if cache is None:
        cache, tree = c.gpu(dfv)
    before = (cache.k.clone(), cache.v.clone())
    rope = dfv.Rope(c.D, rot_dim=rot, theta=theta, interleaved=inter, scaling=scaling, factor=factor, scale=scale)
    dev = qkv.cuda()
    q, k, v = dev[:, :c.H], dev[:, c.H:c.H + c.K], dev[:, c.H + c.K:]
    out = dfv.rope_append(cache, layer, tree, rope, q, k, v, positions.cuda(), out=q if in_place else None)
    torch.cuda.synchronize()
    f = frequencies(rot, theta, scaling, factor)
    want, tol = turned(qkv, positions, f, inter, rope.scale)
    return cache, before, out.double().cpu(), qkv, want, tol


def check(c: Case, cache, before, out, qkv, want, tol, layer=0, stored=None):
    assert bool(((out - want[:, :c.H]).abs() <= tol[:, :c.H]).all())
    k, v = (x.double().cpu() for x in before)
    kt = torch.zeros_like(k)
    for s, n in enumerate(c.nodes):
        for i in range(n):
            if stored is not None and not stored(s, i):
                continue
            r, at = c.off[s] + i, c.lens[s] + i
            pg = c.table[s, at // c.page]
            k[layer, pg, :, at % c.page] = want[r, c.H:c.H + c.K]
            kt[layer, pg, :, at % c.page] = tol[r, c.H:c.H + c.K]
            v[layer, pg, :, at % c.page] = qkv[r, c.H + c.K:].double()
    assert bool(((cache.k.double().cpu() - k).abs() <= kt).all())
    assert torch.equal(cache.v.double().cpu(), v)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 96), (256, 256), (16, 16), (80, 48)])
@pytest.mark.parametrize("inter", [False, True])
def test_layouts_and_partial_heads(dfv, dtype, dim, rot, inter):
    c = Case([30, 0, 16], [5, 1, 3], 6, 2, dim, 16, dtype, seed=dim + rot)
    pos = torch.arange(c.rows, dtype=torch.int32) * 37
    check(c, *step(dfv, c, rot, inter, pos))


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("bands", 16.0)])
@pytest.mark.parametrize("theta", [1e4, 1e6])
def test_scaling(dfv, scaling, factor, theta):
    c = Case([100], [9], 4, 1, 128, 16, BF, seed=3)
    pos = torch.tensor([0, 1, 2, 31, 4095, 4096, 32767, 100000, 131071], dtype=torch.int32)
    check(c, *step(dfv, c, 128, False, pos, theta=theta, scaling=scaling, factor=factor))


def test_far_and_negative_positions(dfv):
    c = Case([10], [6], 2, 2, 64, 16, FP, seed=4)
    pos = torch.tensor([-1, -5000, 1 << 20, (1 << 24) + 1, (1 << 27) + 3, -(1 << 20)], dtype=torch.int32)
    check(c, *step(dfv, c, 64, False, pos))
    check(c, *step(dfv, c, 64, True, pos, theta=5e5))


@pytest.mark.parametrize("layout", ["head", "token", "mixed"])
@pytest.mark.parametrize("page", [8, 64, 256])
def test_cache_strides_and_page_borders(dfv, layout, page):
    c = Case([page - 1, page, 2 * page - 3, 0], [4, 2, 64, 1], 3, 3, 64, page, BF, seed=5, layers=2, layout=layout)
    pos = torch.arange(c.rows, dtype=torch.int32)
    check(c, *step(dfv, c, 64, False, pos, layer=1), layer=1)


def test_in_place(dfv):
    c = Case([7, 70], [16, 5], 8, 2, 128, 16, BF, seed=6)
    pos = torch.arange(c.rows, dtype=torch.int32) + 50
    check(c, *step(dfv, c, 64, True, pos, in_place=True))


def test_a_factor_on_cos_and_sin_and_a_plain_copy_of_the_tail(dfv):
    c = Case([7], [3], 8, 2, 128, 16, BF, seed=7)
    pos = torch.tensor([5, 6, 7], dtype=torch.int32)
    check(c, *step(dfv, c, 64, False, pos, scale=1.25))


def test_rows_of_a_sequence_without_a_page_are_not_stored(dfv):
    c = Case([14, 30], [4, 3], 2, 1, 64, 16, BF, seed=8)
    pos = torch.arange(c.rows, dtype=torch.int32)
    cache, tree = c.gpu(dfv)
    cache.page_table[0, 1] = -1  # tokens 16, 17 of the first sequence
    got = step(dfv, c, 64, False, pos, cache=cache, tree=tree)
    check(c, *got, stored=lambda s, i: s == 1 or i < 2)
    assert cache.errors() == dfv.KVERR_PAGE
    cache.err.zero_()
    cache.page_table[0, 1] = cache.n_pages
    step(dfv, c, 64, False, pos, cache=cache, tree=tree)
    assert cache.errors() == dfv.KVERR_PAGE


def test_bad_lengths_and_indexes_are_flagged_and_store_nothing(dfv):
    c = Case([14, 30], [4, 3], 2, 1, 64, 16, BF, seed=9)
    pos = torch.arange(c.rows, dtype=torch.int32)
    for bad in (-1, 1 << 20, 2 ** 31 - 1):
        cache, tree = c.gpu(dfv)
        cache.lens[0] = bad
        got = step(dfv, c, 64, False, pos, cache=cache, tree=tree)
        check(c, *got, stored=lambda s, i: s == 1)
        assert cache.errors() == dfv.KVERR_LEN
    cache, _ = c.gpu(dfv)
    tree = c.tree(dfv, seq=torch.tensor([2, 1], dtype=torch.int32).cuda())
    check(c, *step(dfv, c, 64, False, pos, cache=cache, tree=tree), stored=lambda s, i: s == 1)
    assert cache.errors() == dfv.KVERR_SEQ


def test_many_rows(dfv):
    c = Case([k * 3 for k in range(40)], [1 + 13 * k % 64 for k in range(40)], 5, 1, 64, 32, FP, seed=10)
    pos = torch.arange(c.rows, dtype=torch.int32) * 11
    check(c, *step(dfv, c, 32, False, pos))
