"""The rings through which a shared prefix's rows go, with the split and the choice of the filling warp compiled from the kernel's
header: whatever the order in which the warps run and in which the barriers' arrivals become visible, no wait on a barrier's parity
passes before the phase that it stands for is over."""
import ctypes
import os
import random
import subprocess

import pytest

TESTS = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(TESTS), "sparse_attention_kv_csa_gb300", "csrc")


@pytest.fixture(scope="module")
def rings(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rings") / "shared_rings.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I" + CSRC, os.path.join(TESTS, "shared_rings_host.cpp"), "-o", so])
    return ctypes.CDLL(so)


def run(slots, filler, fills, rng, reorder):
    """Two warps fill `fills` units into a ring of `slots`, one reader takes them in order.  A slot's empty barrier counts phases; a
    wait for phase k (its unit's use of the slot is over) passes as the hardware's does: when the phase in progress has another
    parity than k.  reorder: how many later arrivals may become visible before one that was made earlier."""
    full = [0] * slots       # units that lie or lay in a slot
    phase = [0] * slots      # of its empty barrier, as it is visible
    at = [0, 0]              # the next unit that each warp looks at
    read, hidden = 0, []     # units read, and those whose arrivals are not visible yet
    for _ in range(400 * fills):
        moves = [("fill", w) for w in (0, 1) if at[w] < fills]
        if read < fills and full[read % slots] > read // slots:
            moves.append(("read", 0))
        if hidden:
            moves.append(("show", 0))
        if not moves:
            break
        what, w = rng.choice(moves)
        if what == "read":
            hidden.append(read)
            read += 1
        elif what == "show":
            unit = hidden.pop(rng.randrange(min(len(hidden), 1 + reorder)))
            phase[unit % slots] += 1
        else:
            unit = at[w]
            slot, round_ = unit % slots, unit // slots
            if filler(slot, unit) == w:
                if round_ > 0 and phase[slot] % 2 == (round_ - 1) % 2:
                    continue  # the wait does not pass yet
                if phase[slot] < round_:
                    return "unit %d over unit %d" % (unit, unit - slots)
                full[slot] += 1
            at[w] += 1
    return None if at == [fills, fills] and read == fills else "stuck"


SHAPES = sorted({(nk, vch) for nk in range(2, 10) for vch in range(1, 5) if 2 * vch <= nk})


@pytest.mark.parametrize("nk,vch", SHAPES)
def test_no_slot_is_filled_before_it_is_free(rings, nk, vch):
    cw = min(vch, 2)
    out = (ctypes.c_int * 2)()
    rng = random.Random(nk * 10 + vch)
    for slots in range(4, 17):  # (as many as fit: 7 for rows of 576 columns, 16 at most)
        rings.rings_split(slots, -(-nk // cw), 2 * -(-vch // cw), 2, out)
        assert sum(out) == slots and min(out) >= 2
        for n in out:
            for _ in range(4):
                assert run(n, lambda slot, unit: rings.rings_filler(slot), 5 * n, rng, n) is None


def test_turns_would_not_do():
    # the model sees what it is for: warps that take units in turn meet every other phase of a slot where their number is odd
    rng = random.Random(1)
    assert any(run(3, lambda slot, unit: unit % 2, 60, rng, 3) for _ in range(300))
    assert not any(run(4, lambda slot, unit: unit % 2, 60, rng, 4) for _ in range(300))
