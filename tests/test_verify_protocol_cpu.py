"""Host model of the verification's cluster: no CTA stores to one that has not started, or that has left.

A CTA's shared memory may be stored to by the cluster's others from when it has
started until it ends.  The model takes from the kernel's source where it
arrives at the cluster's barrier and where it waits, runs clusters of CTAs whose
steps interleave at random (one may start when the others are steps ahead), and
checks every store's target, that a CTA arrives once before each wait, and that
every CTA comes to its end.  A kernel without its first wait, or without the one
of a walk that makes no pass, must be caught.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_20_gb300", "csrc", "fa_verify.cuh")


def body(text, name):
    """The function's text from its name on to the line that closes it."""
    at = re.search(r"\b" + name + r"\([^;{]*\) \{\n", text)
    return text[at.end():text.index("\n}\n", at.end())]


def protocol():
    """What the source does with the cluster's barrier: {arrives at the start, waits before the first store, waits without a
    pass, joins at the end}."""
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernel, quick, exchange = (body(text, x) for x in ("verify_kernel", "row_quick", "exchange"))
    assert exchange.index("store_to(") < exchange.index("cluster_sync()") and "cluster_wait" not in exchange
    before, loop = kernel.split("while (cur >= 0)")
    assert "row_quick(row, p, s, phase, rank, size, kept == 1)" in loop or "row_quick(row, p, s, phase, rank, size)" in loop
    loop, end = loop.split("if (writer) p.n_kept")
    # nothing else stores to another CTA ahead of the first pass
    assert "exchange" not in before and "row_sum" not in loop[:loop.index("row_quick")] and "store_to" not in kernel
    return dict(arrives="if (size > 1) cluster_started();" in before,
                waits="if (first && size > 1) cluster_wait();" in quick[:quick.index("exchange(")],
                without="if (kept == 0) cluster_wait();" in end, joins="cluster_sync();" in end)


def cta(me, size, passes, does, st):
    """One CTA's steps, as a generator: a yield is where others may run."""
    st["started"].add(me)
    if does["arrives"]:
        st["arrived"][me] += 1
    yield
    for i in range(passes):
        yield  # the pass over the row
        if i == 0 and does["waits"]:
            yield from wait(me, st)
        for to in range(size):
            if to not in st["started"] or to in st["left"]:
                raise LookupError(f"CTA {me} stores to {to}, which is not there")
            yield
        st["arrived"][me] += 1
        yield from wait(me, st)
    if passes == 0 and does["without"]:
        yield from wait(me, st)
    if does["joins"]:
        st["arrived"][me] += 1
        yield from wait(me, st)
    st["left"].add(me)


def wait(me, st):
    st["waited"][me] += 1
    assert st["arrived"][me] == st["waited"][me]  # a thread arrives once before each wait
    while min(st["arrived"]) < st["waited"][me]:
        yield


def run(size, passes, does, seed):
    r = random.Random(seed)
    st = dict(started=set(), left=set(), arrived=[0] * size, waited=[0] * size)
    todo = [cta(i, size, passes, does, st) for i in range(size)]
    slow = r.randrange(size)  # one that starts late, most of the time
    steps = 0
    while todo:
        steps += 1
        assert steps < 100000, "CTAs wait for one another for ever"
        pick = r.choice(todo)
        if pick is todo[min(slow, len(todo) - 1)] and r.random() < 0.9:
            continue
        try:
            next(pick)
        except StopIteration:
            todo.remove(pick)
    assert len(st["left"]) == size


@pytest.mark.parametrize("passes", [0, 1, 2, 5])
@pytest.mark.parametrize("size", [2, 4, 16])
def test_stores_reach_ctas_that_are_there(size, passes):
    does = protocol()
    for seed in range(40):
        run(size, passes, does, seed)


@pytest.mark.parametrize("missing,passes", [(dict(arrives=False, waits=False, without=False), 2), (dict(waits=False), 2),
                                            (dict(without=False), 0)])
def test_a_missing_barrier_is_caught(missing, passes):
    does = dict(protocol(), **missing)
    with pytest.raises((LookupError, AssertionError)):
        for seed in range(200):
            run(4, passes, does, seed)
