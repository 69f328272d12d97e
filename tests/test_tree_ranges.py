"""CPU models of the tree-attention kernels' host-visible arithmetic: the cut of the work line into ranges, where partial
states are stored and which of them the join reads, the division by the query heads of a kv head, the phases of the
tile rings, and the rotary table's integer angles."""
from __future__ import annotations

import math
import random
from fractions import Fraction

import pytest

CTAS = 152


def ranges_of(U, n):
    return n if U >= n else U if U > 0 else 1


def start(g, U, G):
    return g * U // G


def group_of(u, U, G):
    return ((u + 1) * G - 1) // U


def units(lens, nodes, heads, tile, over):
    return [heads * (over + max(1, -(-(a + n) // tile))) if n else 0 for a, n in zip(lens, nodes)]


@pytest.mark.parametrize("seed", range(24))
def test_every_tile_in_one_range_and_every_state_read_once(seed):
    rng = random.Random(seed)
    S, heads, tile, over = rng.choice([1, 2, 7, 40, 300]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([3, 5, 6])
    lens = [rng.choice([0, 1, rng.randint(0, 300), rng.randint(0, 40000)]) for _ in range(S)]
    nodes = [rng.randint(0, 3) for _ in range(S)]
    n_rt = rng.choice([1, 1, 2, 4])
    n_groups = CTAS // n_rt
    per = units(lens, nodes, heads, tile, over)
    U = sum(per)
    if U == 0:
        return
    G = ranges_of(U, n_groups)
    owner, stored, told = {}, {}, {}
    base = [sum(per[:s]) for s in range(S)]
    for g in range(G):
        u, end = start(g, U, G), start(g + 1, U, G)
        assert u < end and g < n_groups
        b = max(s for s in range(S) if base[s] <= u and per[s] and u < base[s] + per[s])
        bb = base[b]
        while u < end:
            if per[b] == 0 or u >= bb + per[b]:
                bb += per[b]
                b += 1
                continue
            pair = per[b] // heads
            h, p0 = divmod(u - bb, pair)
            p1 = min(pair, p0 + (end - u))
            last = u - p0 + pair - 1
            u += p1 - p0
            t0, t1, T = max(0, p0 - over), max(0, p1 - over), pair - over
            if t0 >= t1:
                continue
            for t in range(t0, t1):
                assert (b, h, t) not in owner
                owner[b, h, t] = g
            if not (t0 == 0 and t1 == T):  # a partial state
                for rt in range(n_rt):
                    slot = 2 * (g * n_rt + rt) + (t0 == 0)
                    assert slot not in stored and slot < 2 * n_groups * n_rt
                    stored[slot] = (b, h, g, rt)
            if t0 == 0:
                assert (b, h) not in told
                told[b, h] = (g, 1 if t1 == T else group_of(last, U, G) - g + 1)
    assert len(owner) == U - over * heads * sum(n > 0 for n in nodes)
    read = set()
    for s in range(S):
        for h in range(heads if nodes[s] else 0):
            g0, n = told[s, h]
            if n < 2:
                continue
            for rt in range(n_rt):
                for k in range(n):
                    slot = 2 * ((g0 + k) * n_rt + rt) + (k == 0)
                    assert stored[slot] == (s, h, g0 + k, rt)
                    read.add(slot)
    assert read == set(stored)


def test_32_bit_arithmetic_is_exact_where_it_is_used():
    assert (CTAS * (1 << 24)) < 1 << 32  # g U and (u + 1) G
    for G in range(1, 17):
        inv = (65536 + G - 1) // G
        assert all((r * inv) >> 16 == r // G for r in range(1024 + 256))
        assert (1024 + 256) * inv < 1 << 32


@pytest.mark.parametrize("dual", [False, True])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 17])
def test_ring_order_of_keys_and_values(dual, n):
    """The producers' order is the MMAs' order, and a value tile's place in it is what the clean-up of the last tile
    computes; a slot's earlier occupant is long consumed when a warpgroup waits for a value tile of it."""
    ahead = 1 if dual else 2
    slots = 5 if dual else 6
    loads = [("k", k) for k in range(min(ahead, n))]
    for j in range(n):
        loads.append(("v", j))
        if j + ahead < n:
            loads.append(("k", j + ahead))
    uses = []
    if dual:
        uses.append(("k", 0))
        for j in range(n):
            uses.append(("v", j))
            if j + 1 < n:
                uses.append(("k", j + 1))
    else:
        uses += [("k", k) for k in range(min(2, n))]
        for j in range(n):
            uses.append(("v", j))
            if j + 2 < n:
                uses.append(("k", j + 2))
    assert loads == uses and len(loads) == 2 * n
    for j in range(n):
        at = j + min(n, j + ahead)
        assert loads[at] == ("v", j)
        before = at - slots
        if before >= 0:
            assert before < loads.index(("k", j))


def test_two_groups_of_consumers_never_share_a_stage():
    """Tiles of a range alternate between the groups anew in every segment; each group's stages are its own, so each of
    its warps sees every phase of their barriers."""
    rng = random.Random(1)
    per = 5
    turn = [0, 0]
    seen = {}
    for _ in range(200):
        for t in range(rng.randint(1, 30)):
            g = t & 1
            stage, phase = g * per + turn[g] % per, turn[g] // per
            turn[g] += 1
            assert seen.get(stage, -1) == phase - 1  # phases in order, none skipped by the group
            seen[stage] = phase
            assert stage // per == g


def test_rotary_angles_are_exact_fractions_of_a_turn():
    """position * turns mod 2^64, upper 32 bits as signed, against rational arithmetic: off by less than 2^-32 turns (the
    bits dropped) and |position| 2^-65 (the table's rounding)."""
    for f in (1.0, 0.73, 1e-3, 3.3e-6):
        x = Fraction(f / (2 * math.pi))
        F = round(x * 2 ** 64)
        for pos in (0, 1, 2, 4095, 131071, (1 << 31) - 1, -1, -131071):
            turn = (pos % (1 << 64)) * F % (1 << 64)
            hi = turn >> 32
            hi -= (1 << 32) if hi >> 31 else 0
            d = (Fraction(hi, 2 ** 32) - pos * x) % 1
            assert min(d, 1 - d) <= Fraction(1, 2 ** 32) + Fraction(abs(pos), 2 ** 65)
