"""Static check of the tensor-core kernel's waits that needs no GPU.

Each lane of a warp polls a barrier on its own, and may give up on its own.  Behind a wait that a
whole warp makes stand instructions that all 32 lanes have to execute together (elect.sync,
tcgen05.ld, aligned barriers): such a wait ends with a vote, so that no lane goes on without the
others."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "combine_get_layout_gb300", "csrc", "expert_mm.cu")


def functions(text):
    """{name: body} of the functions that start at the beginning of a line."""
    out = {}
    for m in re.finditer(r"^[\w:<>&* ]*\b(\w+)\([^;{}]*\)\s*\{(.*?)^\}", text, re.M | re.S):
        out[m.group(1)] = m.group(2)
    return out


def unvoted(text):
    text = re.sub(r"//[^\n]*", "", text)
    bodies = functions(text)
    bad = [n for n in ("warp_wait", "wait_for_steps", "wait_for_sums")
           if "__all_sync" not in bodies.get(n, "")]
    kernel = text[text.index("expert_mm_kernel("):]
    # a wait whose result a warp goes by: one of the three
    return bad + re.findall(r"\bok = (mbar_wait\w*)\(", kernel)


def test_waits_of_a_warp_end_with_a_vote():
    assert not unvoted(open(SOURCE).read())


def test_lint_catches_the_pattern():
    good = open(SOURCE).read()
    assert unvoted(good.replace("ok = warp_wait(&sm.full[at.s], at.phase)",
                                "ok = mbar_wait(&sm.full[at.s], at.phase, kWaitTimeoutNs)"))
    assert unvoted(good.replace("__all_sync", "bool"))
