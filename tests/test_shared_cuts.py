"""The division of a shared prefix's work over pairs of blocks, the code itself compiled for the host (shared_cuts_host.cpp): every
tile of every item is taken once, its parts lie in slots of their own, in order, where the join looks for them."""
import ctypes
import os
import random
import subprocess

import pytest

TESTS = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(TESTS), "sparse_attention_kv_csa_gb300", "csrc")


@pytest.fixture(scope="module")
def cuts(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("cuts") / "shared_cuts.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I" + CSRC, os.path.join(TESTS, "shared_cuts_host.cpp"), "-o", so])
    lib = ctypes.CDLL(so)
    i32, i64 = ctypes.c_int, ctypes.c_longlong
    lib.cuts_cut.argtypes, lib.cuts_cut.restype = [i64, i32, i32], i64
    lib.cuts_holder.argtypes, lib.cuts_sharing.argtypes = [i64, i64, i32], [i64, i32]
    lib.cuts_segment.argtypes = [i32, i32, i64, ctypes.POINTER(i32)]
    return lib


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_once_and_parts_where_they_are_looked_for(cuts, seed):
    rng = random.Random(seed)
    # groups of (tiles, items); a group without a shared prefix has no items
    groups = [(rng.choice([1, 2, rng.randint(1, 60), rng.randint(1, 3000)]), rng.choice([0, 1, rng.randint(1, 40)])) for _ in range(rng.randint(1, 30))]
    if seed % 5 == 0:
        groups.append((rng.randint(20000, 60000), rng.randint(30, 80)))  # more than 2^20 units
    items = [(g, t) for g, (t, n) in enumerate(groups) for _ in range(n)]
    head, clusters, out = cuts.cuts_head(), rng.choice([1, 2, 70, 76]), (ctypes.c_int * 3)()
    total = sum(t + head for _, t in items)
    blocks = cuts.cuts_sharing(total, clusters)
    assert 1 <= blocks <= clusters
    begins, at = [], 0
    for _, t in items:
        begins.append(at)
        at += t + head
    done, slots = {}, {}
    m, unit = 0, 0
    for c in range(blocks):
        assert cuts.cuts_cut(total, c, blocks) == unit
        left = cuts.cuts_cut(total, c + 1, blocks) - unit
        while left > 0:
            off = unit - begins[m]
            cuts.cuts_segment(items[m][1], off, left, out)
            take, t0, t1 = out
            assert take > 0
            if t1 > t0:
                assert done.get(m, 0) == t0  # in order, none left out
                done[m] = t1
                slot = m + c
                assert slot not in slots and slot < len(items) + clusters
                slots[slot] = m
            unit, left = unit + take, left - take
            if unit == begins[m] + items[m][1] + head:
                m += 1
    assert unit == total and all(done[i] == t for i, (_, t) in enumerate(items))
    for i, (_, t) in enumerate(items):
        first = begins[i] + head
        c0 = cuts.cuts_holder(first, total, blocks)
        n = cuts.cuts_holder(first + t - 1, total, blocks) - c0 + 1
        assert [slots.get(i + c0 + k) for k in range(n)] == [i] * n
        assert sum(v == i for v in slots.values()) == n
