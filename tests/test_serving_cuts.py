"""The attention kernel's division of work, by its own integer arithmetic: every tile of every item is taken once, parts of
an item lie where its join looks for them, and the divisions by multiplication are exact."""
import random

import pytest

HEAD, MIN_UNITS = 3, 3


def segments(items, c, blocks):
    """Block c's segments (item, t0, t1, one past its last unit), and T and G."""
    units = [n + HEAD for n in items]
    total = sum(units)
    g = max(1, min(total // MIN_UNITS, blocks))
    if c >= g or total == 0:
        return [], total, g
    unit = total * c // g
    left = total * (c + 1) // g - unit
    at, m = 0, 0
    while not at <= unit < at + units[m]:
        at += units[m]
        m += 1
    off, got = unit - at, []
    while left > 0 and m < len(items):
        take = min(items[m] + HEAD - off, left)
        head, t0, t1 = off == 0, max(off - HEAD, 0), max(off + take - HEAD, 0)
        unit, left, off, m = unit + take, left - take, 0, m + 1
        if t1 > t0 or (items[m - 1] == 0 and head):
            got.append((m - 1, t0, t1, unit))
    return got, total, g


@pytest.mark.parametrize("seed", range(400))
def test_tiles_parts_and_joins(seed):
    rng = random.Random(seed)
    items = [rng.choice([0, 0, 1, 2, rng.randint(0, 60)]) for _ in range(rng.randint(1, 40))]
    blocks = rng.randint(1, 20)
    whole, slots, joins = {}, {}, {}
    for c in range(blocks):
        got, total, g = segments(items, c, blocks)
        for i, t0, t1, unit in got:
            nt = items[i]
            if t0 == 0 and t1 == nt:
                assert i not in whole
                whole[i] = 1
                continue
            slot = 2 * c + (t0 == 0)
            assert slot not in slots
            holder = lambda u: ((u + 1) * g - 1) // total  # noqa: E731
            slots[slot] = (i, t0, t1)
            joins[slot] = (i, c if t0 == 0 else holder(unit - t1), holder(unit - 1 + nt - t1))
    joined = {}
    for slot, (i, first, last) in joins.items():
        parts = [slots[2 * k + (k == first)] for k in range(first, last + 1)]
        assert all(p[0] == i for p in parts) and first <= slot // 2 <= last
        assert parts[0][1] == 0 and parts[-1][2] == items[i]
        assert all(a[2] == b[1] for a, b in zip(parts, parts[1:]))
        joined[i] = joined.get(i, 0) + (slot // 2 == first)
    for i in range(len(items)):
        assert (i in whole) != (joined.get(i, 0) == 1)


def test_division_by_multiplication():
    rng = random.Random(1)
    for d in list(range(1, 1500)) + [rng.randrange(1, 1 << 31) for _ in range(3000)] + [(1 << 31) - 1, 1 << 30, (1 << 30) + 1]:
        log = 0
        while log < 31 and (1 << log) < d:
            log += 1
        m = (1 << 32) * ((1 << log) - d) // d + 1
        assert m < 1 << 32
        for n in [0, 1, d - 1, d, 2 * d - 1, (1 << 31) - 1, ((1 << 31) - 1) // d * d, rng.randrange(1 << 31)]:
            if 0 <= n < 1 << 31:
                assert ((m * n >> 32) + n) >> log == n // d and (m * n >> 32) + n < 1 << 32
