"""A loop with a vote of the whole warp is left by all its lanes at one vote: a lane that read a flag for itself and
left would wait at the next vote for lanes that wait for it at this one.  (No call makes a wait run out, so the source is read.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_13_gb300", "csrc")
VOTE = re.compile(r"__(any|all|ballot)_sync")


def loops(text):
    """(first line, body) of every for / while loop with braces."""
    for m in re.finditer(r"\b(?:for|while) \(", text):
        i, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        if not text[i:].lstrip().startswith("{"):
            continue
        j = text.index("{", i) + 1
        depth, k = 1, j
        while depth:
            depth += {"{": 1, "}": -1}.get(text[k], 0)
            k += 1
        yield text.count("\n", 0, m.start()) + 1, text[m.start():k]


def alone(text):
    """Lines of loops whose own head or body votes, where a lane may leave on its own look at a flag that other warps set."""
    text = re.sub(r"//[^\n]*", "", text)
    return [n for n, body in loops(text)
            if VOTE.search(body) and re.search(r"if \((?:(?!__any_sync|__all_sync)[^;{])*\*sAbort[^;{]*\)\s*(\{[^{}]*)?break", body)]


def test_it_sees_such_a_loop():
    bad = "for (; __any_sync(0xffffffffu, todo); --left) {\n if (left == 0 || *sAbort) {\n *sAbort = 1;\n break;\n }\n}"
    good = "for (;; --left) {\n if (!__any_sync(0xffffffffu, todo)) break;\n if (__any_sync(0xffffffffu, left == 0 || *sAbort)) {\n *sAbort = 1;\n break;\n }\n}"
    assert alone(bad) == [1] and alone(good) == []


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cuh", ".cu"))))
def test_votes_are_left_together(name):
    with open(os.path.join(CSRC, name)) as f:
        assert alone(f.read()) == []
