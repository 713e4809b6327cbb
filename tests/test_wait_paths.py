"""A wait inside an attention kernel that runs out must not leave warps behind at a
barrier: the warps that share one come to it whatever their waits said.  No wait can
be made to run out in these kernels without a fault, so the sources are read."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dsa_indexer_indexshare_gb300",
                    "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _softmax_roles(text):
    """The code of the warps that meet at named barrier 1, per kernel: from their
    declaration of the softmax denominators to the CTA's last barrier."""
    return [text[m.start():text.index("tmem_dealloc", m.start())] for m in re.finditer(r"float lpart\[HW\];", text)]


def _loops(role):
    """(start, end) of every for loop's body."""
    found = []
    for m in re.finditer(r"\bfor \(", role):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(role[at], 0)
            at += 1
        if role[at:].lstrip().startswith("{"):
            start = end = role.index("{", at)
            depth = 0
            while True:
                depth += {"{": 1, "}": -1}.get(role[end], 0)
                end += 1
                if not depth:
                    break
            found.append((start, end))
    return found


@pytest.mark.parametrize("name,kernels", [("sparse_mla.cu", 2), ("sparse_mla_int4.cu", 1)])
def test_softmax_warps_come_to_every_barrier_together(name, kernels):
    roles = _softmax_roles(_source(name))
    assert len(roles) == kernels
    for role in roles:
        assert role.count("named_bar_sync(1, NST)") >= 3
        # no loop in which they share a barrier is left, or gone round early, before its end: what a
        # failed wait leaves out is inside loops and branches of its own
        for m in re.finditer(r"\b(break|continue|return);", role):
            inner = [(e - s, s, e) for s, e in _loops(role) if s < m.start() < e]
            assert inner, role[max(0, m.start() - 200):m.end()]
            start, end = min(inner)[1:]
            held = role[m.start():end] if m.group(1) == "continue" else role[start:end]
            assert "named_bar" not in held, role[max(0, m.start() - 200):m.end()]
        # nor is a loop's count a matter of a wait
        for m in re.finditer(r"\bfor \(([^;]*);([^;]*);", role):
            assert not re.search(r"\b(alive|dead|ok)\b|wait", m.group(2)), m.group(0)
