"""page_tables against the tables made by hand, request after request: whole numbers, all equal."""
import random

import pytest
import torch

import serving_util as u
import sparse_attention_kv_csa_gb300 as csa

pytestmark = pytest.mark.gpu


def run(before, after, ratio, page, free, table, capacity, taken=None, stride=0, in_place=False):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    width = len(table[0]) if table else 0
    t = torch.full((len(table), width + stride), -9, dtype=torch.int32, device="cuda")
    if table and width:
        t[:, :width] = i32(table)
    t = t[:, :width]
    got = csa.page_tables(i32(before), i32(after), ratio, page, i32(free), t, capacity,
                          taken=None if taken is None else i32([taken]), out=t if in_place else None)
    assert (got[0] is t) == in_place
    return [x.tolist() for x in got]


def check(before, after, ratio, page, free, table, capacity, taken=None, **kw):
    want = u.pages_plain(before, after, ratio, page, free, table, capacity, taken or 0)
    got = run(before, after, ratio, page, free, table, capacity, taken, **kw)
    for w, g, name in zip(want, got, ("table", "cu_rows", "slots", "counts")):
        assert list(w) == g, name


def made(rng, n, most, new, ratio, page, width, spare):
    after = [rng.randint(0, most) for _ in range(n)]
    before = [max(0, a - rng.randint(0, new)) for a in after]
    ids = list(range(n * (most // ratio // page + 2) + spare))
    rng.shuffle(ids)
    table = []
    for b in before:
        held = -(-(b // ratio) // page)
        row = [ids.pop() for _ in range(held)]
        table.append((row + [rng.randint(-5, 10 ** 6) for _ in range(width)])[:width])
    return before, after, ids, table


@pytest.mark.parametrize("n,most,new,ratio,page,width", [
    (1, 0, 0, 1, 1, 1), (1, 1, 1, 1, 1, 1), (1, 1000, 1000, 4, 16, 20), (7, 300, 4, 4, 16, 5), (64, 5000, 1, 4, 64, 20),
    (513, 700, 300, 3, 7, 40), (100, 900, 900, 1, 1, 900), (33, 2000, 100, 128, 100, 1), (3, 40000, 20000, 1, 64, 700),
    (1500, 64, 5, 16, 2, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables(n, most, new, ratio, page, width, in_place):
    rng = random.Random(n * 1000 + most)
    before, after, ids, table = made(rng, n, most, new, ratio, page, width, 8)
    total = sum(max(a // ratio - b // ratio, 0) for a, b in zip(after, before))
    for capacity in {total + 5, max(0, total - 3), 0}:
        check(before, after, ratio, page, ids, table, capacity, in_place=in_place)


def test_free_pages_run_out_and_offsets():
    rng = random.Random(5)
    before, after, ids, table = made(rng, 50, 400, 400, 4, 8, 14, 0)
    for free, taken in ((ids[:7], None), (ids[:7], 3), (ids[:7], 7), (ids[:7], 9), ([], None), (ids, 11)):
        check(before, after, 4, 8, free, table, 5000, taken=taken)


def test_table_narrower_than_the_need_lengths_that_shrink_and_strides():
    check([0, 0], [100, 40], 1, 4, list(range(90)), [[-1] * 3, [-1] * 3], 150)
    check([50, 9, -3], [20, -1, 5], 1, 4, list(range(90)), [[7] * 20, [8] * 20, [9] * 20], 6, stride=5)


def test_no_requests_and_no_columns():
    got = run([], [], 4, 16, [1], [], 3)
    assert got[1] == [0] and got[2] == [-1] * 3 and got[3] == [0, 0, 0, 0]
    check([0], [9], 1, 4, [1, 2, 3], [[]], 9)


def test_most_requests():
    rng = random.Random(9)
    before, after, ids, table = made(rng, 14000, 40, 4, 4, 4, 3, 0)
    check(before, after, 4, 4, ids, table, 14100)


def test_graph_replay_takes_pages_step_by_step():
    """The count of pages taken stays on the device: a captured step, replayed, serves a growing request."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    before, after, taken = i32([0]), i32([5]), i32([0])
    table, free = i32([[-1] * 8]), i32([4, 2, 7, 1, 0, 3])
    csa.page_tables(before, after, 1, 2, free, table.clone(), 8, taken=taken)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, cu, slots, counts = csa.page_tables(before, after, 1, 2, free, table, 8, taken=taken, out=table)
        taken += counts[1:2]
        before.copy_(after)
        after += 3
    want_table, used, b, a = [[-1] * 8], 0, 0, 5
    for _ in range(3):
        want_table, _, want_slots, c = u.pages_plain([b], [a], 1, 2, free.tolist(), want_table, 8, used)
        used, b, a = used + c[1], a, a + 3
        g.replay()
        torch.cuda.synchronize()
        assert table.tolist() == want_table and slots.tolist() == want_slots and counts.tolist() == c
