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


@pytest.mark.gpu
def test_the_wait_limit_leaves_time_for_what_is_in_flight():
    """A CTA that gives up waits for its own copies and products with the same limit, so a
    limit below a millisecond is taken as one: a wait for nothing takes that long."""
    torch = pytest.importorskip("torch")
    dsa = pytest.importorskip("dsa_indexer_indexshare_gb300")
    ws = dsa.workspace(256, torch.device("cuda:0"))
    try:
        for ns in (0, 1, 1000):
            dsa.set_wait_timeout_ns(ns)
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            torch.cuda.synchronize()
            a.record()
            dsa.dsa_selftest_wait_timeout(ws)
            b.record()
            with pytest.raises(dsa.DsaError) as e:
                dsa.status_fetch(ws)
            assert e.value.status == dsa.DSA_ERR_TIMEOUT
            torch.cuda.synchronize()
            assert a.elapsed_time(b) >= 0.99
    finally:
        dsa.set_wait_timeout_ns(2_000_000_000)
