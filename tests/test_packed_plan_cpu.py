"""The packed forward's division of work on the host: every key tile of every item is done once, and parts fit together.

The ranges are walked as the kernel's cursor walks them, and the dealt items
as it deals them.
"""
import ctypes
import random

import pytest

from tests import packed_host

KEYS, MIN_PART, MOST_PARTS = 128, 8, 8


def plan(lens, hkv, tpt, causal, ctas):
    """(kind, work): `work` is each CTA's list of (s, h, b, from, to, part), part = (slot, slot0, count, k) or None."""
    n = len(lens)
    info, ranges, pairs = (ctypes.c_int * 4)(), (ctypes.c_int * (14 * 160))(), (ctypes.c_int * (2 * 2048))()
    packed_host.lib().packed_plan((ctypes.c_int * n)(*lens), n, hkv, tpt, int(causal), ctas, info, ranges, pairs)
    grid, dealt, slots, split = info
    assert 0 <= grid <= ctas
    work = [[] for _ in range(grid)]
    if dealt:
        assert grid == ctas and slots == 0 and split == 0 and dealt % hkv == 0
        for c in range(grid):
            for i in range(-(-dealt // grid)):
                at = i * grid + (grid - 1 - c if i % 2 else c)
                if at < dealt:
                    s, b = pairs[at // hkv * 2], pairs[at // hkv * 2 + 1]
                    work[c].append((s, at % hkv, b, 0, steps(lens[s], b, tpt, causal), None))
        return "dealt", work, slots, split
    for c in range(grid):
        s, h, b, n_items, begin, end, *parts = ranges[14 * c:14 * c + 14]
        first, last = tuple(parts[:4]), tuple(parts[4:])
        assert n_items >= 1
        for i in range(n_items):
            if i > 0:
                b += 1
                if b * 2 * tpt >= lens[s]:
                    b, h = 0, h + 1
                    if h == hkv:
                        h, s = 0, s + 1
                        while lens[s] == 0:
                            s += 1
            whole = steps(lens[s], b, tpt, causal)
            k0, k1 = begin if i == 0 else 0, end if i == n_items - 1 else whole
            part = None
            if (k0, k1) != (0, whole):
                part = first if i == 0 else last
                assert part[0] >= 0
            work[c].append((s, h, b, k0, k1, part))
        # what is said to be a part is one
        assert (first[0] >= 0) == (work[c][0][5] == first)
        assert (last[0] >= 0) == (n_items > 1 and work[c][-1][5] == last)
    return "ranges", work, slots, split


def steps(n, b, tpt, causal):
    return -(-(min(n, (2 * b + 2) * tpt) if causal else n) // KEYS)


def check(lens, hkv, tpt, causal, ctas):
    kind, work, slots, split = plan(lens, hkv, tpt, causal, ctas)
    done, parts = {}, {}
    for todo in work:
        for s, h, b, k0, k1, part in todo:
            assert 0 <= k0 < k1
            done.setdefault((s, h, b), []).append((k0, k1))
            if part:
                parts.setdefault((s, h, b), []).append((k0, k1, part))
    want = {(s, h, b) for s, n in enumerate(lens) for h in range(hkv) for b in range(-(-n // (2 * tpt)))}
    assert set(done) == want
    for (s, h, b), pieces in done.items():
        at = 0
        for k0, k1 in sorted(pieces):
            assert k0 == at
            at = k1
        assert at == steps(lens[s], b, tpt, causal)
        assert len(pieces) == 1 or all(k1 - k0 >= MIN_PART for k0, k1 in pieces)
    assert len(parts) == split and sorted(p[2][3] for v in parts.values() for p in v[:1]) == list(range(split))
    used = []
    for pieces in parts.values():
        pieces.sort()
        assert 2 <= len(pieces) <= MOST_PARTS
        slot0, count, k = pieces[0][2][1:]
        assert count == len(pieces)
        assert [p[2] for p in pieces] == [(slot0 + i, slot0, count, k) for i in range(count)]  # in key order
        used += range(slot0, slot0 + count)
    assert sorted(used) == list(range(slots))
    return kind, max((len(v) for v in parts.values()), default=0)


def ragged(rng):
    top = rng.choice([1, 40, 300, 1500, 5000, 20000, 100000])
    n = rng.choice([1, 1, 2, 3, 8, 30, 200, 1024])
    while n > 1 and n * top > 400000:
        n //= 2
    lens = [rng.choice([0, 1, top, rng.randint(0, top)]) for _ in range(n)] if rng.random() < 0.7 else [top] * n
    return lens


@pytest.mark.parametrize("seed", range(30))
def test_random_plans_cover_every_step_once(seed):
    rng = random.Random(seed)
    for _ in range(25):
        hkv = rng.choice([1, 1, 2, 3, 4, 8, 16])
        tpt = 128 // rng.choice([1, 1, 2, 3, 4, 5, 8, 16, 40, 128])
        lens = ragged(rng)
        if sum(lens) * hkv // tpt > 60000:
            lens, hkv = lens[:1], 1
        check(lens, hkv, tpt, rng.random() < 0.7, rng.choice([152, 152, 148, 160, 8, 1]))


def test_each_way_of_dividing_is_met():
    assert check([1800, 3, 0, 900, 700, 1, 1500], 8, 32, True, 152) == ("dealt", 0)
    assert check([4096], 1, 32, True, 152)[0] == "ranges"
    assert check([100000], 1, 128, False, 8)[0] == "ranges"
    assert check([40000], 1, 128, False, 152)[1] >= 2
    assert check([], 4, 32, True, 152) == ("ranges", 0)
    assert check([0, 0], 4, 32, True, 152) == ("ranges", 0)


def test_an_item_of_many_parts():
    assert check([10635], 1, 128, True, 152)[1] == 6
    assert max(check([n], 1, 128, False, 152)[1] for n in range(4000, 20000, 97)) >= 5
