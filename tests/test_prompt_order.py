"""What the warps of the prompt kernel may overtake: its barriers as a graph of events, each after those that it waits for, for
segments of every length and any number of blocks at their end that are cleaned.  Numbers of slots are read from the source."""
from __future__ import annotations

import graphlib
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_moe_gb300", "csrc")
TEXT = open(os.path.join(CSRC, "prompt_attn.cu")).read()


def shape(dim):
    k64, v64, k128, v128 = (int(re.search(r"kK = D == 64 \? (\d+) : (\d+), kV = D == 64 \? (\d+) : (\d+);", TEXT).group(i)) for i in (1, 3, 2, 4))
    nb64, nb128 = map(int, re.search(r"kNB = D == 64 \? (\d+) : (\d+);", TEXT).groups())
    return (k64, v64, nb64) if dim == 64 else (k128, v128, nb128)


class Events:
    """done[x]: everything that has happened when x does.  A circle (a kernel that would wait for ever) does not sort."""

    def __init__(self, segments, dim):
        """segments: (blocks, of which the last so many are cleaned)"""
        kK, self.kV, NB = shape(dim)
        todo, add = {}, None
        todo, chains = {}, {}

        def add(who, x, pre=()):  # in program order of `who`
            todo[x] = [*pre, *([chains[who]] if who in chains else [])]
            chains[who] = x

        g = 0
        self.blocks, self.dirty = 0, []
        for s, (n, d) in enumerate(segments):
            for t in range(1 - NB, n):  # the producers: V t, K t + NB - 1
                if t >= 0:
                    add("copies", ("copy v", g + t), [("did pv", 1, g + t - self.kV)])
                if t + NB - 1 < n:
                    add("copies", ("copy k", g + t + NB - 1), [("did qk", 1, g + t + NB - 1 - kK)])
            last = g + n - 1
            add("clean", ("begin", s), [("did qk", 1, g - 1)] if s else [])  # Q's place is free; the flag is cleared
            for b in range(g + n - d, g + n):
                add("clean", ("asked", b), [("dirty", b)])
                add("clean", ("has v", b), [("copy v", b)])
                add("clean", ("clean", b))
                self.dirty.append(b)
            # ---- the MMA warp
            def qk(w, b):
                add("mma", ("qk", w, b), [("copy k", b), ("begin", s)])
                add("tensor", ("did qk", w, b), [("qk", w, b)])

            def pv(w, b):
                add("mma", ("pv", w, b), [("p", w, b), ("copy v", b)])
                add("tensor", ("did pv", w, b), [("pv", w, b)])

            qk(0, g)
            qk(1, g)
            if NB == 3 and n > 1:
                qk(0, g + 1)
            if d == n:
                add("mma", ("dirty", g))
            for j in range(n):
                b = g + j
                if j >= n - d:
                    add("mma", ("cleaned", b), [("clean", b)])
                if j + 1 < n and j + 1 >= n - d:
                    add("mma", ("dirty", b + 1))
                add("mma", ("full v", b), [("copy v", b)])
                pv(0, b)
                if j + 1 < n:
                    qk(0 if NB == 2 else 1, b + 1)
                pv(1, b)
                if j + NB - 1 < n:
                    qk(1 if NB == 2 else 0, b + NB - 1)
            for w in (0, 1):
                for b in range(g, g + n):
                    add("wg%d" % w, ("scores", w, b), [("did qk", w, b)])
                    add("wg%d" % w, ("p", w, b))
                add("wg%d" % w, ("read", w, s), [("did pv", w, last)])
            g += n
        self.blocks, self.segments = g, len(segments)
        self.todo = {x: [y for y in pre if y in todo] for x, pre in todo.items()}
        self.done = {}
        for x in graphlib.TopologicalSorter(self.todo).static_order():
            self.done[x] = frozenset().union(*(self.done[y] | {y} for y in self.todo[x]))

    def after(self, late, early):
        assert late not in self.todo or early not in self.todo or early in self.done[late], "%s does not wait for %s" % (late, early)


def cuts():
    rng = random.Random(6)
    yield [(1, 1)] * 12
    yield [(9, 1)] * 2
    yield [(5, 0), (1, 1), (1, 1), (2, 2), (3, 3), (1, 0), (1, 0), (4, 2)]
    for _ in range(10):
        yield [(n, rng.randint(0, min(n, 3))) for n in (rng.choice((1, 1, 2, 3, 6)) for _ in range(8))]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("segments", list(cuts()), ids=str)
def test_nothing_is_overtaken(dim, segments):
    e = Events(segments, dim)
    flags = int(re.search(r"s_bad\[(\d+)\];", TEXT).group(1))
    for b in e.dirty:  # the ring's phases, as the cleaning warp meets them
        e.after(("has v", b), ("full v", b - e.kV))
        e.after(("has v", b), ("copy v", b - e.kV))
        e.after(("copy v", b + e.kV), ("has v", b))
        e.after(("pv", 0, b), ("clean", b))
    for a, b in zip(e.dirty, e.dirty[1:]):  # one block in hand
        e.after(("dirty", b), ("asked", a))
        e.after(("clean", b), ("cleaned", a))
    for b in range(e.blocks):
        for w in (0, 1):
            e.after(("did qk", w, b + 2), ("scores", w, b))  # two barriers in turn
            e.after(("p", w, b + 2), ("pv", w, b))
    for s in range(e.segments):
        for w in (0, 1):
            e.after(("begin", s + flags), ("read", w, s))
