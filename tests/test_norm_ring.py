"""The bookkeeping of the norm's ring of rows, the device code itself compiled for the host (norm_ring_host.cpp): stages are
refilled only when their copy has landed, and no copy is under way when a team ends, after a wait that gave up either."""
import ctypes
import os
import subprocess

import pytest

TESTS = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(TESTS), "sparse_attention_kv_csa_gb300", "csrc")


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("ring") / "ring.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I" + CSRC,
                           os.path.join(TESTS, "norm_ring_host.cpp"), "-o", so])
    lib = ctypes.CDLL(so)
    lib.ring_faults.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                ctypes.POINTER(ctypes.c_int)]
    return lib


@pytest.mark.parametrize("stages", [1, 2, 3, 8])
@pytest.mark.parametrize("arrays", [1, 2, 3])
def test_every_copy_is_waited_for(ring, stages, arrays):
    fills = ctypes.c_int()
    for n_rows, step in ((1, 1), (2, 1), (7, 1), (8, 1), (9, 1), (40, 1), (40, 3), (41, 7), (3, 5)):
        rows = -(-n_rows // step)
        assert ring.ring_faults(stages, n_rows, step, arrays, -1, 0, fills) == 0 and fills.value == rows
        for stuck in range(rows):
            for late in (0, 1):
                assert ring.ring_faults(stages, n_rows, step, arrays, stuck, late, fills) == 0, (n_rows, step, stuck, late)
                assert fills.value == min(rows, stuck + stages)  # none after the wait that gave up
