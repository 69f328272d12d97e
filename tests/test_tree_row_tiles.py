"""The range model of the attention kernels with three CTAs per range: 152 is no multiple of three, and rows of 513 to
768 (nodes x query heads of a kv head) need that many."""
from __future__ import annotations

import random

import pytest

from tests import test_tree_ranges as model


@pytest.mark.parametrize("seed", range(100, 116))
def test_every_tile_in_one_range_and_every_state_read_once(monkeypatch, seed):
    drawn = []

    class Rng(random.Random):
        def choice(self, seq):
            drawn.append(seq)
            return 3 if seq == [1, 1, 2, 4] else super().choice(seq)

    monkeypatch.setattr(model.random, "Random", Rng)
    model.test_every_tile_in_one_range_and_every_state_read_once(seed)
    assert [1, 1, 2, 4] in drawn
