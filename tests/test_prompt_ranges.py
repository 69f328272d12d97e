"""CPU model of the prompt attention's work line (prompt_attn.cu): the closed form for the blocks of the tiles before a
tile, the cut of the line into ranges, and the partial states that the join reads.  Constants come from the source."""
from __future__ import annotations

import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_moe_gb300", "csrc")
TEXT = open(os.path.join(CSRC, "prompt_attn.cu")).read()
KEYS, TILE, OVER, CTAS = 128, 256, int(re.search(r"kOver = (\d+);", TEXT).group(1)), 152


def limit(n, nk, i):
    return min(nk, max(0, nk - n + i + 1))


def blocks(n, nk, G, t):
    return max(1, -(-limit(n, nk, min(n - 1, (TILE * t + TILE - 1) // G)) // KEYS))


def tiles(n, G):
    return -(-n * G // TILE)


def blocks_before(n, nk, G, i):
    """The kernel's closed form, statement by statement (C's division: no operand is negative where it divides)."""
    B = (255 + G * (KEYS + nk - n)) >> 7
    i1 = 0 if B >= G else (G - B + 1) // 2
    if i <= i1:
        return i
    c, w = 2 * i1 + B, i - i1
    a, r = w // G, w % G
    f = [(2 * u + c) // G for u in range(G)]
    assert c >= 0
    return i1 + a * sum(f) + G * a * (a - 1) + sum(f[:r]) + 2 * a * r


@pytest.mark.parametrize("G", range(1, 17))
def test_the_closed_form(G):
    rng = random.Random(G)
    for _ in range(40):
        n = rng.choice([1, 2, 31, 32, 33, 128, 700, 2500])
        nk = rng.choice([0, 1, n // 2, n - 1, n, n + 1, n + 127, n + 128, n + 5000])
        m, run = tiles(n, G), 0
        for t in range(m):
            assert blocks_before(n, nk, G, t) == run
            run += blocks(n, nk, G, t)


def head_units(n, nk, G):
    m = tiles(n, G)
    return 0 if m == 0 else OVER * m + blocks_before(n, nk, G, m - 1) + blocks(n, nk, G, m - 1)


def walk(seqs, G, heads, whole):
    """Every range's segments (b, h, t, t0, t1, T, last unit), as PromptWalk goes."""
    U = sum(heads * head_units(n, nk, G) for n, nk in seqs)
    ranges = CTAS if U >= CTAS else max(U, 1)
    out = []
    for g in range(CTAS):
        u, end = (g * U // ranges, (g + 1) * U // ranges) if g < ranges else (0, 0)
        segs = []
        if u < end:
            base = b = 0
            while not base <= u < base + heads * head_units(*seqs[b], G):
                base += heads * head_units(*seqs[b], G)
                b += 1
            n, nk = seqs[b]
            m = tiles(n, G)
            h, w = divmod(u - base, head_units(n, nk, G))
            lo, hi = 0, m
            while hi - lo > 1:
                mid = (lo + hi) // 2
                if OVER * mid + blocks_before(n, nk, G, mid) <= w:
                    lo = mid
                else:
                    hi = mid
            t, p0 = lo, w - (OVER * lo + blocks_before(n, nk, G, lo))
            if whole and p0:
                u += OVER + blocks(n, nk, G, t) - p0
                p0 = 0
                t += 1
            first = True
            while True:
                t += not first
                first = False
                if u >= end:
                    break
                while t >= m:
                    t = 0
                    h += 1
                    if h >= heads or m == 0:
                        h = 0
                        b += 1
                        n, nk = seqs[b]
                        m = tiles(n, G)
                T = blocks(n, nk, G, t)
                p1 = OVER + T if whole else min(OVER + T, p0 + end - u)
                last = u - p0 + OVER + T - 1
                t0, t1 = max(0, p0 - OVER), max(0, p1 - OVER)
                u += p1 - p0
                p0 = 0
                if t0 < t1:
                    segs.append((b, h, t, t0, t1, T, last))
        out.append(segs)
    return U, ranges, out


CASES = [([(1, 1)], 8, 4), ([(137, 137)], 8, 4), ([(2039, 2039), (0, 0), (700, 700), (1, 5000)], 7, 2), ([(5, 0), (300, 20)], 3, 1),
         ([(0, 0), (0, 9), (64, 40000)], 1, 8), ([(16381, 16381)], 8, 4), ([(n, n + 3 * n % 77) for n in range(0, 400, 13)], 5, 3)]


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("seqs,G,heads", CASES)
def test_every_block_is_done_once(seqs, G, heads, whole):
    U, ranges, out = walk(seqs, G, heads, whole)
    done = {}
    for segs in out:
        for b, h, t, t0, t1, T, _ in segs:
            for j in range(t0, t1):
                assert done.setdefault((b, h, t, j), 0) == 0
                done[b, h, t, j] = 1
    assert len(done) == sum(heads * sum(blocks(n, nk, G, t) for t in range(tiles(n, G))) for n, nk in seqs)
    if whole:
        assert all(t0 == 0 and t1 == T for segs in out for _, _, _, t0, t1, T, _ in segs)


@pytest.mark.parametrize("seqs,G,heads", CASES)
def test_the_join_reads_what_was_left(seqs, G, heads):
    """A range tells of at most one tile; the ranges it names hold that tile's states, in the slots that the join reads,
    and no state is left unread or written twice."""
    U, ranges, out = walk(seqs, G, heads, False)
    slots = {}
    for g, segs in enumerate(out):
        for b, h, t, t0, t1, T, last in segs:
            if (t0, t1) != (0, T):
                at = 2 * g + (t0 == 0)
                assert at not in slots
                slots[at] = (b, h, t, t0, t1)
    for g, segs in enumerate(out):
        told = [s for s in segs if s[3] == 0 and s[4] < s[5]]
        assert len(told) <= 1
        for b, h, t, _, _, T, last in told:
            n = ((last + 1) * ranges - 1) // U - g + 1
            assert n >= 2
            at = 0
            for k in range(n):
                s = slots.pop(2 * (g + k) + (k == 0))
                assert s[:3] == (b, h, t) and s[3] == at
                at = s[4]
            assert at == T
    assert not slots


def test_the_quotient_by_the_group():
    """over_g: the product's error stays below one part in 2^16 / G for the numbers that occur (a tile's 256 rows and a
    remainder below G)."""
    for G in range(1, 17):
        inv = (65536 + G - 1) // G
        assert all(r * inv >> 16 == r // G for r in range(256 + G))
