"""The graphs of events of test_codes_order.py and test_prompt_order.py are models kept by hand: only numbers of slots and flags
follow the sources, and a wait that a kernel loses stays in its model.  Here: that each of their properties can fail (a ring made
smaller, a wait dropped from the model), and that the tables of a tile's own powers are not written over before they are read."""
from __future__ import annotations

import graphlib
import re

import pytest

from tests import test_codes_order as codes, test_prompt_order as prompts

SHAPES = [(dim, dual) for dim in (64, 128) for dual in (False, True)]


def without(events, drop):
    """The model less the waits (late, early) that `drop` tells of."""
    e = events
    e.todo = {x: [y for y in pre if y in e.todo and not drop(x, y)] for x, pre in e.todo.items()}
    e.done = {}
    for x in graphlib.TopologicalSorter(e.todo).static_order():
        e.done[x] = frozenset().union(*(e.done[y] | {y} for y in e.todo[x]))
    return e


def some_fail(check, cases):
    for case in cases:
        try:
            check(*case)
        except AssertionError as e:
            assert "does not wait for" in str(e)
            return True
    return False


def codes_fail():
    return some_fail(codes.test_nothing_is_overtaken, [(dim, dual, s) for dim, dual in SHAPES for s in codes.cuts()])


def prompts_fail():
    return some_fail(prompts.test_nothing_is_overtaken, [(dim, s) for dim in (64, 128) for s in prompts.cuts()])


def test_the_models_as_they_are():
    assert not codes_fail() and not prompts_fail()


@pytest.mark.parametrize("ring,text,less", [
    ("flags", "constexpr int kFlags = %d", 4), ("tells", "constexpr int kTells = %d", 2), ("told", "s_told[%d];", 2), ("below", "s_below[%d][kKeys];", 2)])
def test_smaller_rings(monkeypatch, ring, text, less):
    pattern = re.escape(text).replace("%d", r"(\d+)")
    assert len(re.findall(pattern, codes.TEXT)) == 1
    monkeypatch.setattr(codes, "TEXT", re.sub(pattern, lambda m: text % less, codes.TEXT))
    assert codes_fail()


@pytest.mark.parametrize("late,early", [
    ("rows", "reset"),      # the flag is cleared before the warpgroups go on
    ("widen k", "did qk"),  # K is widened into a place that has been read
    ("pv", "p"),            # the product follows the weights
    ("scores", "did qk"), ("p", "pv wait"), ("pv wait", "scores")])
def test_waits_dropped_codes(monkeypatch, late, early):
    real = codes.Events
    monkeypatch.setattr(codes, "Events", lambda *a: without(real(*a), lambda x, y: x[0] == late and y[0] == early))
    assert codes_fail()


@pytest.mark.parametrize("late,early", [
    ("begin", "did qk"),   # the flag and Q's place
    ("cleaned", "clean"),  # the MMA warp takes V once it is clean
    ("copy v", "did pv"),  # V is copied into a place that has been read
    ("asked", "dirty"),    # the cleaning warp is a block ahead at most
    ("pv", "p"), ("scores", "did qk")])
def test_waits_dropped_prompts(monkeypatch, late, early):
    real = prompts.Events
    monkeypatch.setattr(prompts, "Events", lambda *a: without(real(*a), lambda x, y: x[0] == late and y[0] == early))
    assert prompts_fail()


@pytest.mark.parametrize("dim,dual", SHAPES)
def test_tables_of_own_powers(dim, dual):
    """A tile's own powers are written where its largest ones are told, and read up to its weights."""
    own, back = (int(re.search(r"%s\[(\d+)\]\[kKeys\];" % name, codes.TEXT).group(1)) for name in ("s_own", "s_back"))
    assert own == back == 8 and "smem_u32(&s_own[tell & 7]" in codes.TEXT and "smem_u32(&s_back[tell & 7]" in codes.TEXT
    assert codes.TEXT.count("s_own[tile & 7]") == codes.TEXT.count("s_back[tile & 7]") == 1
    for segments in codes.cuts():
        e = codes.Events(segments, dim, dual)
        for k in range(e.n):
            for w in (0, 1):
                for v in (0, 1):
                    e.after(("tell", w, k + own), ("p", v, k))
