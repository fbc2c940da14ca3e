"""The packed forward's products in tensor memory: which accesses to the same columns nothing puts in order.

A query tile's issuer waits for P of step s - 1, issues O += P V (s - 1) and
S (s) = Q K^T, and commits; the softmax warps wait for the commit of S (s),
read S, rescale O and write P, in two halves of which the first is handed
over before the second where the kernel says so.  A product runs from its
issue until a commit behind it has been waited for.  Two products are in
order by themselves where they have the same accumulator and shape.  The
model goes through the steps of two items and lists pairs of accesses to the
same columns, one of them writing, with nothing between them.
"""
import pytest

from tests import packed_host

STEPS = 4


def columns(d, t):
    f = packed_host.lib().packed_tmem
    s, p, o = (f(d, which, t) for which in range(3))
    return set(range(s, s + 128)), [set(range(p, p + 32)), set(range(p + 32, p + 64))], set(range(o, o + d))


def unordered(s_cols, p_cols, o_cols, d, halves):
    issued, found = [], []
    issuer, softmax = set(), set()  # products known to be done

    def touch(name, reads, writes, known, acc=None, shape=None):
        for i, (other, o_reads, o_writes, o_acc, o_shape) in enumerate(issued):
            if i in known or (acc is not None and (acc, shape) == (o_acc, o_shape)):
                continue
            if reads & o_writes or writes & (o_reads | o_writes):
                found.append((other, name, o_shape, shape))

    def issue(name, reads, writes, acc, shape):
        touch(name, reads, writes, issuer, acc, shape)
        issued.append((name, reads, writes, acc, shape))

    def pv(half):
        issue("PV", p_cols[half] | o_cols, o_cols, "O", (128, d))

    def write_p(half):
        touch("P", set(), p_cols[half], softmax)

    for _ in range(2):
        for s in range(STEPS + 1):
            if s > 0:
                if halves:
                    write_p(0)
                    issuer |= softmax  # the first half's hand-over
                    pv(0)
                    write_p(1)
                    issuer |= softmax
                    pv(1)
                else:
                    write_p(0), write_p(1)
                    issuer |= softmax
                    pv(0), pv(1)
            if s < STEPS:
                issue("S", set(), s_cols, "S", (128, 128))
            softmax |= set(range(len(issued)))  # the commit behind S, or behind the item's last P V
            if s < STEPS:
                touch("reads S", s_cols, set(), softmax)
            touch("rescales or reads O", o_cols, o_cols, softmax)
    return found


@pytest.mark.parametrize("t", [0, 1])
def test_head_size_64_rests_on_no_order_of_different_products(t):
    s, p, o = columns(64, t)
    assert not (s & (p[0] | p[1])) and not (o & (p[0] | p[1])) and not (s & o)
    assert unordered(s, p, o, 64, bool(packed_host.lib().packed_halves(64))) == []


@pytest.mark.parametrize("t", [0, 1])
def test_head_size_128_rests_on_the_order_of_products_of_one_shape(t):
    s, p, o = columns(128, t)
    found = unordered(s, p, o, 128, bool(packed_host.lib().packed_halves(128)))
    assert {(a, b) for a, b, _, _ in found} == {("PV", "S")} and all(x == y for _, _, x, y in found)


def test_the_model_sees_p_over_s():
    s, _, o = columns(64, 0)
    over = [set(range(32)), set(range(32, 64))]
    assert {(a, b) for a, b, _, _ in unordered(s, over, o, 64, True)} == {("PV", "S")}


def test_tiles_and_accumulators_share_no_columns():
    for d in (64, 128):
        used = [s | p[0] | p[1] | o for s, p, o in (columns(d, 0), columns(d, 1))]
        assert not used[0] & used[1] and max(used[0] | used[1]) < 512
