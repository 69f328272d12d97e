"""Orders inside the attention kernels that no run on a GPU is sure to show, read from their sources (CPU)."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_moe_gb300", "csrc")


def source(name, begin, end):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return text[text.index(begin):text.index(end)]


# ---------------------------------------------------------------- a flag shared by the warps of a segment
def protocol():
    """What a consumer warp of the mma.sync kernel does with s_bad in one segment: its sets, reads, clears and barriers
    in order, each with the flag it touches (0 or 1, turned by the segment's parity where the source turns it)."""
    text = source("tree_attn.cu", "consumers\n  const int cw", "// ---------------------------------------------------------------- join")
    at = r"s_bad(?:\[(?P<%s>[^\]]+)\])?"
    rules = [("wait", r"bar_sync_n\(1, 32 \* kCons\)"), ("set", r"if \(bad\) " + at % "a" + r" = 1"),
             ("clear", r"if \(ct == 0\) " + at % "b" + r" = 0"), ("read", r"isbad = " + at % "c")]
    events = []
    for m in re.finditer("|".join("(?P<%s>%s)" % r for r in rules), text):
        kind = next(k for k, _ in rules if m.group(k))
        which = next((m.group(g) for g in "abc" if m.group(g)), None)
        events.append((kind, {None: None, "turn": 0, "turn ^ 1": 1}[which]))
    assert [k for k, _ in events if k != "wait"].count("set") == 1 and "read" in dict(events)
    return events


def lost_flags(events, bad):
    """Segments in which some warp reads another value than "any warp of the segment was bad", over every interleaving.
    bad[s] = the warps that set the flag in segment s; warp 0 clears."""
    warps = 1 + max([w for b in bad for w in b] + [1])
    steps = [(s, e) for s in range(len(bad)) for e in events]
    waits = [sum(e[0] == "wait" for _, e in steps[:i]) for i in range(len(steps) + 1)]
    lost, seen, todo = set(), set(), [((0,) * warps, (0, 0))]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        pcs, flags = state
        for w, pc in enumerate(pcs):
            if pc == len(steps):
                continue
            s, (kind, which) = steps[pc]
            # a barrier lets a warp through once every warp has reached it
            if kind == "wait" and any(waits[p] < waits[pc] or (waits[p] == waits[pc] and steps[p][1][0] != "wait")
                                      for p in pcs if p < len(steps)):
                continue
            f, i = list(flags), 0 if which is None else which ^ (s & 1)
            if kind == "set" and w in bad[s]:
                f[i] = 1
            if kind == "clear" and w == 0:
                f[i] = 0
            if kind == "read" and f[i] != bool(bad[s]):
                lost.add(s)
            todo.append((pcs[:w] + (pc + 1,) + pcs[w + 1:], tuple(f)))
    return lost


def test_the_model_finds_a_flag_cleared_late():
    late = [("set", None), ("wait", None), ("read", None), ("wait", None), ("clear", None)]
    assert lost_flags(late, [(), (1,)]) == {1}
    early = [("set", 0), ("wait", None), ("read", 0), ("clear", 1), ("wait", None)]
    assert lost_flags(early, [(1,), (), (1,)]) == set()


@pytest.mark.parametrize("bad", [[(), (1,)], [(1,), ()], [(0,), (1,), ()], [(1,), (), (0, 1), ()], [(0, 2), (1,), (2,)]])
def test_no_segment_loses_the_flag_of_a_value_that_is_not_finite(bad):
    assert lost_flags(protocol(), bad) == set()


# ---------------------------------------------------------------- tensor memory read after another warpgroup's wait
def test_outputs_in_tensor_memory_are_read_behind_fences():
    """With one row tile each warpgroup waits for its own last product and reads both accumulators: between the barrier
    through which it learns of the other's and its first load there is a fence after the barrier's, and the other's wait
    is fenced before it."""
    out = source("tree_attn_tc.cu", "// ---- output:", "cudaError_t launch_one")
    names = r"tc_fence_before\(\)|tc_fence_after\(\)|bar_sync_n\(1, 256\)|tmem_ld32\(|mbar_wait_fast\("
    order = [m.group(0) for m in re.finditer(names, out)]
    first = order.index("tmem_ld32(")
    assert order[first - 3:first] == ["tc_fence_before()", "bar_sync_n(1, 256)", "tc_fence_after()"]
    assert order.index("mbar_wait_fast(") < first - 3 and order.count("bar_sync_n(1, 256)") == 2
