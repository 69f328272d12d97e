"""CPU model of the prompt attention's work line (prompt_attn.cu): the closed form for the blocks of the tiles before a
tile, the cut of the line into ranges, and the partial states that the join reads.  Constants come from the source."""
from __future__ import annotations

import math
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_moe_gb300", "csrc")
TEXT = open(os.path.join(CSRC, "prompt_attn.cu")).read()
KEYS, TILE, OVER, CTAS = 128, 256, int(re.search(r"kOver = (\d+);", TEXT).group(1)), 152


def positions(G):
    return TILE // G & ~7


def limit(n, nk, i):
    return min(nk, max(0, nk - n + i + 1))


def blocks(n, nk, G, t):
    return max(1, -(-limit(n, nk, min(n, (t + 1) * positions(G)) - 1) // KEYS))


def tiles(n, G):
    return -(-n // positions(G))


def blocks_before(n, nk, G, i):
    """The kernel's closed form, statement by statement (C's division: no operand is negative where it divides)."""
    P = positions(G)
    C = P + KEYS - 1 + nk - n
    run, rise = KEYS // math.gcd(P, KEYS), P // math.gcd(P, KEYS)
    assert run <= 16
    i1 = 0 if C >= KEYS else (KEYS - C + P - 1) // P
    if i <= i1:
        return i
    c, w = P * i1 + C, i - i1
    a, r = w // run, w % run
    f = [(P * u + c) // KEYS for u in range(run)]
    assert c >= 0
    return i1 + a * sum(f) + rise * run * (a * (a - 1) // 2) + sum(f[:r]) + rise * a * r


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


def test_the_head_of_a_row():
    """head_of: the quotient of a tile's row by its positions."""
    for G in range(1, 17):
        P = positions(G)
        assert P % 8 == 0 and P * G <= TILE
        inv = (65536 + P - 1) // P
        assert all(r * inv >> 16 == r // P for r in range(TILE))


# ---------------------------------------------------------------- the ring and the barriers
@pytest.mark.parametrize("NB", [2, 3])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 9])
def test_the_order_of_the_ring(NB, n):
    """What the producers load, the products use and the cleaning warp looks for is in the same order, and a block's place
    is free after its second use."""
    LA = NB - 1
    order = [("k", j) for j in range(min(LA, n))]
    for t in range(n):
        order.append(("v", t))
        if t + LA < n:
            order.append(("k", t + LA))
    item_k = lambda j: j if j < LA else min(2 * j - LA + 1, n + j)  # noqa: E731
    item_v = lambda j: j + min(n, j + LA)  # noqa: E731
    assert len(order) == 2 * n
    for j in range(n):
        assert order[item_k(j)] == ("k", j) and order[item_v(j)] == ("v", j)
    used = []
    for i in range(-NB, 2 * n):
        if i >= 0:
            used.append(item_v(i >> 1))
        if 0 <= i + NB < 2 * n:
            used.append(item_k((i + NB) >> 1))
    first = [used.index(x) for x in range(2 * n)]
    assert first == sorted(first) and all(used.count(x) == 2 for x in range(2 * n))


@pytest.mark.parametrize("NB", [2, 3])
def test_no_wait_by_parity_meets_two_phases(NB):
    """Every order of the MMA warp and the two warpgroups that the barriers allow, over two tiles: whoever waits for block b on
    a barrier finds block b's phase there, not a later one, and nobody waits for ever."""
    n, tiles_ = 3, 2
    mma = []
    for _ in range(tiles_):
        for i in range(-NB, 2 * n):
            if i >= 0:
                mma += [("wait", "p", i & 1, i >> 1, hf) for hf in (0, 1)]
            if 0 <= i + NB < 2 * n:
                mma.append(("post", "s", (i + NB) & 1, (i + NB) >> 1, 0))
        mma.append(("tile",))
    # the MMA warp's events with blocks counted over both tiles
    at, m = 0, []
    for e in mma:
        if e[0] == "tile":
            at += n
        else:
            m.append((e[0], e[1], e[2], e[3] + at, e[4]))
    wg = [[e for b in range(n * tiles_) for e in (("wait", "s", w, b, 0), ("post", "p", w, b, 0), ("post", "p", w, b, 1))] for w in (0, 1)]
    progs = [m] + wg
    seen, todo = set(), [((0, 0, 0), ())]
    while todo:
        pcs, posted = todo.pop()
        if (pcs, posted) in seen:
            continue
        seen.add((pcs, posted))
        done = dict(posted)  # (kind, warpgroup, parity, half) -> phases done
        moved = False
        for k, pc in enumerate(pcs):
            if pc == len(progs[k]):
                continue
            what, kind, w, b, hf = progs[k][pc]
            key = (kind, w, b & 1, hf)
            if what == "wait":
                assert done.get(key, 0) <= (b >> 1) + 1, "a later phase is done"
                if done.get(key, 0) < (b >> 1) + 1:
                    continue
                new = posted
            else:
                assert done.get(key, 0) == b >> 1
                new = tuple(sorted({**done, key: (b >> 1) + 1}.items()))
            moved = True
            todo.append((pcs[:k] + (pc + 1,) + pcs[k + 1:], new))
        assert moved or all(pc == len(q) for pc, q in zip(pcs, progs)), "nobody can go on"


def test_a_tile_a_range():
    """Where ranges are tiles: the host's bound holds all of them, and CTA g's sequence, head and tile are the line's g-th."""
    rng = random.Random(7)
    assert "tiles = (long long)L.p.Hkv * (L.p.n_rows / L.pos + L.p.n_seqs)" in TEXT
    for _ in range(300):
        G, heads = rng.randint(1, 16), rng.randint(1, 8)
        rows = [rng.choice((0, 1, rng.randint(1, 40), rng.randint(1, 900))) for _ in range(rng.randint(1, 12))]
        line = [(b, h, t) for b, n in enumerate(rows) for h in range(heads) for t in range(tiles(n, G))]
        assert len(line) <= heads * (max(sum(rows), 1) // positions(G) + len(rows))
        for g, want in enumerate(line):
            base = 0
            for b, n in enumerate(rows):
                m = tiles(n, G)
                if g < base + heads * m:
                    w = g - base
                    assert (b, w // m, w - w // m * m) == want
                    break
                base += heads * m
