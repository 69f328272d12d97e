"""Rotary append with the caller's own frequencies: a ramp that is linear in the pair's index between two of them, which
the "bands" scaling (linear in the turns over the original context) does not give."""
from __future__ import annotations

import math

import pytest
import torch

from tests._tree_util import Case
from tests.test_gpu_rope_append import BF, check, dfv, frequencies, turned  # noqa: F401

pytestmark = pytest.mark.gpu


def by_index(rot, theta, factor, original, low=1.0, high=32.0):
    at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
    out = []
    for i in range(rot // 2):
        f, g = theta ** (-2 * i / rot), min(1.0, max(0.0, (i - first) / (last - first)))
        out.append((1 - g) * f + g * f / factor)
    return out


@pytest.mark.parametrize("inter", [False, True])
def test_a_ramp_over_the_pairs(dfv, inter):  # noqa: F811
    c = Case([100, 3], [9, 2], 4, 1, 128, 16, BF, seed=3)
    pos = torch.tensor([0, 1, 2, 31, 4095, 4096, 32767, 100000, 131071, 7, 8], dtype=torch.int32)
    f = by_index(128, 1e6, 4.0, 32768)
    rope = dfv.Rope(128, interleaved=inter, freqs=f, scale=0.1 * math.log(4.0) + 1)
    qkv = torch.randn(c.rows, c.H + 2 * c.K, c.D, generator=torch.Generator().manual_seed(2)).to(BF)
    cache, tree = c.gpu(dfv)
    before = (cache.k.clone(), cache.v.clone())
    dev = qkv.cuda()
    out = dfv.rope_append(cache, 0, tree, rope, dev[:, :4], dev[:, 4:5], dev[:, 5:], pos.cuda())
    torch.cuda.synchronize()
    want, tol = turned(qkv, pos, f, inter, rope.scale)
    check(c, cache, before, out.double().cpu(), qkv, want, tol)
    bands = frequencies(128, 1e6, "bands", 4.0, original=32768.0)  # differs where both ramps run
    assert max(abs(a / b - 1) for a, b in zip(bands, f)) > 0.02
