"""How warps that share a barrier give up.

Every wait of the kernels is bounded, and two warps that wait for the same thing may
end differently: one just before it comes, one just after.  Warps that share a named
barrier (bar.sync over their threads) must therefore vote on how a wait ended before
they come to any barrier, and leave together: a warp that left alone would never be
counted at it again, and the others would wait without a limit.

Checked on the text of the epilogues, whose four-warp turns are what shares barriers:
from a wait that may give up, the next barrier is a vote."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_moe_route_04_gb300", "csrc")
KERNELS = ["moe_gemm.cu", "moe_mxfp4_gemm.cu", "moe_train_gemm.cu", "moe_int8_gemm.cu"]
WAIT = r"(?P<wait>\b(?:mbar_wait(?:<\w+>)?|ring_get|ring_take)\s*\()"
VOTE = r"(?P<vote>\bvote_any\w*(?:<[^>]*>)?\s*\()"


def function_body(text, start):
    """From the first brace behind `start` to the one that closes it."""
    i = text.index("{", start)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i:j + 1]
    raise ValueError("unbalanced braces")


def epilogue(text):
    """The epilogue's loop over the tiles."""
    text = re.sub(r"//(?! -+ epilogue)[^\n]*", "", text)
    return function_body(text, text.index("for (uint32_t n = 0;;", text.index("- epilogue")))


def events(body):
    """Waits, votes and barriers in the order of the text: what a lambda does counts
    where it is called, and a wait that ignores the abort flag drains what is behind a
    vote."""
    inside = {}
    for m in re.finditer(r"auto (\w+) = \[&\]\([^)]*\) ", body):
        block = function_body(body, m.end())
        inside[m.group(1)] = block
        body = body.replace(block, " " * len(block), 1)
    body = re.sub(r"mbar_wait\([^;]*&no_abort[^;]*;", ";", body)
    calls = "|".join(r"\b%s\(" % n for n, b in inside.items() if "named_barrier_sync" in b) or r"(?!)"
    found = []
    for m in re.finditer("%s|%s|(?P<barrier>named_barrier_sync|%s)" % (WAIT, VOTE, calls), body):
        found.append((m.lastgroup, body.count("\n", 0, m.start())))
    return found


def barriers_behind_unvoted_waits(body):
    open_wait, bad = False, []
    for kind, line in events(body):
        if kind == "wait":
            open_wait = True
        elif kind == "vote":
            open_wait = False
        elif open_wait:
            bad.append(line)
    return bad


def test_the_search_finds_what_it_is_for():
    early = """{ auto staging_free = [&]() { named_barrier_sync(3, 128); };
      bool ok = ring_get(ring, n, c);
      if (ok) staging_free();
      ok = mbar_wait(&full[a], 0, flag, status);
      if (vote_any(!ok, turn)) break; }"""
    assert barriers_behind_unvoted_waits(early) == [2]
    voted = "{ ok = ring_get(r); if (vote_any(!ok)) break; named_barrier_sync(3, 128); }"
    assert barriers_behind_unvoted_waits(voted) == []
    piece = "{ if (vote_any(!ok, 0)) break;\n mbar_wait(&in[0], 0, flag, s);\n named_barrier_sync(3, 128); }"
    assert barriers_behind_unvoted_waits(piece) == [2]
    drained = "{ if (vote_any(!ok)) { mbar_wait(&in[0], 0, &no_abort, s); break; }\n named_barrier_sync(3, 128); }"
    assert barriers_behind_unvoted_waits(drained) == []


@pytest.mark.parametrize("name", KERNELS)
def test_a_wait_is_voted_on_before_the_next_barrier(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        body = epilogue(f.read())
    kinds = [k for k, _ in events(body)]
    assert "wait" in kinds and "vote" in kinds and "barrier" in kinds
    assert barriers_behind_unvoted_waits(body) == []
