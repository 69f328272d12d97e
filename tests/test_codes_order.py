"""What the warps of the codes kernel on the tensor cores may overtake: its barriers as a graph of events, each after those that
it waits for, for tiles cut into segments of every kind.  Numbers of slots and flags are read from the source."""
from __future__ import annotations

import graphlib
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_moe_gb300", "csrc")
TEXT = open(os.path.join(CSRC, "tree_attn_codes_tc.cu")).read()


def constant(name):
    return int(re.search(r"constexpr int %s = (\d+)" % name, TEXT).group(1))


def slots(dim, dual):
    k64, k128, v64, v128 = map(int, re.search(r"kK = D == 64 \? (\d+) : (\d+), kV = D == 64 \? (\d+) : (\d+);", TEXT).groups())
    ck64, ckd, cks, cv64, cv128 = map(int, re.search(r"kCK = D == 64 \? (\d+) : DUAL \? (\d+) : (\d+), kCV = D == 64 \? (\d+) : (\d+);", TEXT).groups())
    return (k64, v64, ck64, cv64) if dim == 64 else (k128, v128, ckd if dual else cks, cv128)


class Events:
    """done[x]: everything that has happened when x does.  A circle (a kernel that would wait for ever) does not sort."""

    def __init__(self, segments, dim, dual):
        self.done, kK, kV, kCK, kCV = {}, *slots(dim, dual)
        self.n, self.seg = sum(segments), [s for s, m in enumerate(segments) for _ in range(m)]
        first = [sum(segments[:s]) for s in range(len(segments))]
        self.todo = {}
        add = self.todo.__setitem__
        warps = (0, 1)  # of each kind
        for k in range(self.n):
            s = self.seg[k]
            for w in warps:
                add(("copy k", k), [("copy k", k - 1), *(("widen k", v, k - kCK) for v in warps)])
                add(("copy v", k), [("copy v", k - 1), *(("widen v", v, k - kCV) for v in warps)])
                add(("tell", w, k), [("copy k", k), ("widen k", w, k - 1)])
                add(("widen k", w, k), [("tell", w, k), ("did qk", k - kK)])
                add(("clean", w, k), [("copy v", k), ("widen v", w, k - 1)])
                add(("below", w, k), [("clean", w, k), *(("tell", v, k) for v in warps)])  # waits for what was told, and reads it
                add(("widen v", w, k), [("below", w, k), ("did pv", k - kV)])
                before = ("p", w, k - 1) if k != first[s] else ("rows", w, s)
                add(("scores", w, k), [before, ("did qk", k)])  # waits for the scores
                add(("pv wait", w, k), [("scores", w, k)])
                add(("p", w, k), [("pv wait", w, k)])
        order = []  # the MMA warp's
        for s, m in enumerate(segments):
            f = first[s]
            ahead = 1 if dual else 2
            order += [("qk", f + i, s) for i in range(min(ahead, m))]
            for j in range(m):
                order.append(("pv", f + j, s))
                if j + ahead < m:
                    order.append(("qk", f + j + ahead, s))
        was = was_did = None
        for what, k, s in order:
            pre = [was] if was else []
            if what == "qk":
                pre += [("widen k", v, k) for v in warps] + [("rows", w, s) for w in warps]
                if dual and k != first[s]:  # a warpgroup's next scores: over its P
                    pre += [("pv", k - 1)]
            else:
                pre += [("widen v", v, k) for v in warps] + [("p", w, k) for w in warps]
            add((what, k), pre)
            add(("did " + what, k), [(what, k)] + ([was_did] if was_did else []))
            was, was_did = (what, k), ("did " + what, k)
        for s, m in enumerate(segments):
            last = first[s] + m - 1
            for w in warps:
                add(("rows", w, s), [("end", 0, s - 1), ("end", 1, s - 1), ("reset", s - 1)] if w == 0 else [("end", 0, s - 1), ("end", 1, s - 1)])
                add(("read", w, s), [("p", w, last), ("did pv", last)])
                add(("end", w, s), [("read", w, s)])
            add(("reset", s), [("end", 0, s), ("end", 1, s)])
        for x in graphlib.TopologicalSorter({x: [y for y in pre if y in self.todo] for x, pre in self.todo.items()}).static_order():
            self.done[x] = frozenset().union(*(self.done[y] | {y} for y in self.todo[x] if y in self.todo))

    def after(self, late, early):
        assert late not in self.todo or early not in self.todo or early in self.done[late], "%s does not wait for %s" % (late, early)


def cuts():
    rng = random.Random(5)
    yield [1] * 24
    yield [24]
    yield [2] * 12
    yield [3, 1, 1, 1, 1, 1, 5, 1, 2, 1, 1, 1, 1]
    for _ in range(6):
        yield [rng.choice((1, 1, 1, 2, 3, 6)) for _ in range(10)]


@pytest.mark.parametrize("dual", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("segments", list(cuts()), ids=str)
def test_nothing_is_overtaken(dim, dual, segments):
    e = Events(segments, dim, dual)
    flags, tells = constant("kFlags"), constant("kTells")
    told = int(re.search(r"s_told\[(\d+)\];", TEXT).group(1))
    below = int(re.search(r"s_below\[(\d+)\]\[kKeys\];", TEXT).group(1))
    assert "s_bad[kFlags]" in TEXT and "s_tell[kTells]" in TEXT and TEXT.count("s_bad[seg % kFlags]") == 3
    for k in range(e.n):
        for w in (0, 1):
            for late in range(k + 1, e.n):  # a segment's flag is cleared before a later one's values are cleaned
                if e.seg[late] >= e.seg[k] + flags:
                    e.after(("clean", w, late), ("reset", e.seg[late] - flags))
            for v in (0, 1):
                e.after(("tell", w, k + told), ("below", v, k))  # no wait by parity meets two phases
                e.after(("tell", w, k + below), ("below", v, k))
                e.after(("tell", w, k + tells), ("p", v, k))
            turn = 1 if dual else 2
            e.after(("did qk", k + turn), ("scores", w, k))
            e.after(("p", w, k + turn), ("pv", k))
            if not dual and e.seg[k] == (e.seg[k - 1] if k else -1):  # the product of the tile before, where O is rescaled
                e.after(("pv wait", w, k), ("did pv", k - 3))  # its barrier's phase before is over
                e.after(("did pv", k + 1), ("pv wait", w, k))
