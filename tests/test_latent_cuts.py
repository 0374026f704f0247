"""The attention kernel's division of work, the code itself compiled for the host (latent_cuts_host.cpp): every tile of every
item is taken once, parts lie where the join looks for them, sizes past 2^20 and 2^31 units among them."""
import ctypes
import os
import random
import subprocess

import pytest

TESTS = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(TESTS), "sparse_attention_kv_csa_gb300", "csrc")


@pytest.fixture(scope="module")
def cuts(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("cuts") / "cuts.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I" + CSRC,
                           os.path.join(TESTS, "latent_cuts_host.cpp"), "-o", so])
    lib = ctypes.CDLL(so)
    i32, i64, u32 = ctypes.c_int, ctypes.c_longlong, ctypes.c_uint
    lib.cuts_cut.argtypes, lib.cuts_cut.restype = [i64, i32, i32], i64
    lib.cuts_holder.argtypes, lib.cuts_sharing.argtypes = [i64, i64, i32], [i64, i32]
    lib.cuts_segment.argtypes = [i32, i32, i64, ctypes.POINTER(i32)]
    for f in (lib.cuts_quotient, lib.cuts_remainder):
        f.argtypes, f.restype = [u32, u32], u32
    return lib


def segments(cuts, items, c, blocks):
    """Block c's segments (item, t0, t1, one past its last unit), and T and G, as the kernel walks them."""
    units = [n + cuts.cuts_head() for n in items]
    total = sum(units)
    g = cuts.cuts_sharing(total, blocks)
    if c >= g or total == 0:
        return [], total, g
    unit = cuts.cuts_cut(total, c, g)
    left = cuts.cuts_cut(total, c + 1, g) - unit
    at, m = 0, 0
    while not at <= unit < at + units[m]:
        at += units[m]
        m += 1
    off, got, out = unit - at, [], (ctypes.c_int * 3)()
    while left > 0 and m < len(items):
        some = cuts.cuts_segment(items[m], off, left, out)
        take, t0, t1 = out
        assert take > 0
        unit, left, off, m = unit + take, left - take, 0, m + 1
        if some:
            got.append((m - 1, t0, t1, unit))
    return got, total, g


SIZES = {"small": (40, 60, 20), "device": (700, 400, 304), "past 20 bits": (40, 90000, 304), "past 31 bits": (200, 33_000_000, 304)}


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("seed", range(40))
def test_tiles_parts_and_joins(cuts, size, seed):
    rng = random.Random(seed)
    many, most, wide = SIZES[size]
    items = [rng.choice([0, 0, 1, 2, rng.randint(0, most)]) for _ in range(rng.randint(1, many))]
    blocks = rng.randint(1, wide)
    if size.startswith("past"):
        bits = int(size.split()[1])
        items += [most] * ((1 << bits) // most + 1)
        rng.shuffle(items)
        assert sum(items) > 1 << bits
    whole, slots, joins = {}, {}, {}
    for c in range(blocks):
        got, total, g = segments(cuts, items, c, blocks)
        for i, t0, t1, unit in got:
            nt = items[i]
            if t0 == 0 and t1 == nt:
                assert i not in whole
                whole[i] = 1
                continue
            slot = 2 * c + (t0 == 0)
            assert slot not in slots
            slots[slot] = (i, t0, t1)
            first = c if t0 == 0 else cuts.cuts_holder(unit - t1, total, g)
            joins[slot] = (i, first, cuts.cuts_holder(unit - 1 + nt - t1, total, g))
    joined = {}
    for slot, (i, first, last) in joins.items():
        joined.setdefault(i, (first, last, []))
        assert joined[i][:2] == (first, last) and first <= slot // 2 <= last
        joined[i][2].append(slot // 2 == first)
    for i, (first, last, firsts) in joined.items():
        assert sum(firsts) == 1 and len(firsts) == last - first + 1
        parts = [slots[2 * k + (k == first)] for k in range(first, last + 1)]
        assert all(p[0] == i for p in parts)
        assert parts[0][1] == 0 and parts[-1][2] == items[i]
        assert all(a[2] == b[1] for a, b in zip(parts, parts[1:]))
    for i in range(len(items)):
        assert (i in whole) != (i in joined)


@pytest.mark.parametrize("total", [1, 2, 5, 1000, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, 123456789, (1 << 31) + 7, 1 << 39])
def test_cuts_and_holders_are_the_exact_quotients(cuts, total):
    rng = random.Random(total)
    for g in (1, 2, 7, 151, 152, 304, 4095):
        for c in {0, 1, g // 2, g - 1, g}:
            assert cuts.cuts_cut(total, c, g) == total * c // g
        for unit in {0, total // 2, total - 1, *(rng.randrange(total) for _ in range(50))}:
            c = cuts.cuts_holder(unit, total, g)
            assert total * c // g <= unit < total * (c + 1) // g
    for blocks in (1, 152, 304):
        assert cuts.cuts_sharing(total, blocks) == max(1, min(total // cuts.cuts_least(), blocks))


def test_division_by_multiplication(cuts):
    rng = random.Random(1)
    for d in list(range(1, 600)) + [rng.randrange(1, 1 << 31) for _ in range(500)] + [(1 << 31) - 1, 1 << 30, (1 << 30) + 1]:
        for n in [0, 1, d - 1, d, 2 * d - 1, (1 << 31) - 1, ((1 << 31) - 1) // d * d, rng.randrange(1 << 31)]:
            if 0 <= n < 1 << 31:
                assert cuts.cuts_quotient(n, d) == n // d and cuts.cuts_remainder(n, d) == n % d
