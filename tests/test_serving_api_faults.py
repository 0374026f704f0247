"""What the serving operators' entry points do when a CUDA call below them fails: the entry points compiled for the host over fakes
(serving_api_host.cpp), no GPU."""
import ctypes
import os
import subprocess

import pytest

from sparse_attention_kv_csa_gb300 import _build

TESTS = os.path.dirname(os.path.abspath(__file__))
CUDA_INVALID, CUDA_NO_MEMORY = 1, 2


@pytest.fixture(scope="module")
def api(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("api") / "serving_api.so")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc())))
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I" + _build.CSRC, "-I" + _build.INCLUDE, "-I" + os.path.join(cuda, "include"),
                           "-x", "c++", os.path.join(_build.CSRC, "csa_serving_api.cu"), os.path.join(TESTS, "serving_api_host.cpp"), "-o", so])
    lib = ctypes.CDLL(so)
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    lib.csa_shared_attention.argtypes = [P, i64, i64, P, i32, i64, i32, i32, i32, P, i64, i32, P, i64, i32, P, i64, i32,
                                         P, P, P, i32, i32, f32, P, P, P, P]
    return lib


def shared(api, shared_result=0, malloc_result=0):
    """The status of one call, and how often what was called."""
    a = 4096  # (an address that nothing reads)
    api.fake_reset(shared_result, malloc_result)
    rc = api.csa_shared_attention(a, 64 * 512, 512, a, 64, 64, 64, 512, 512, a, 512, 0, None, 100, 64, a, 90, 90, a, a, a, 1, 1, 1.0, None, a, None,
                                  None)
    n = (ctypes.c_int * 7)()
    api.fake_counts(n)
    return rc, dict(zip(("shared", "latent", "plain", "mallocs", "frees", "cleared", "last"), n))


def test_ordinary_call(api):
    rc, n = shared(api)
    assert rc == 0 and n["shared"] == 1 and n["latent"] == 0


def test_no_room_for_the_parts_of_a_shared_prefix_is_read_by_request(api):
    rc, n = shared(api, CUDA_NO_MEMORY)
    assert rc == 0 and n["shared"] == 1 and n["latent"] == 1 and n["mallocs"] == n["frees"] == 1
    assert n["last"] == 0  # the next caller of CUDA does not meet the error


def test_no_room_at_all_and_other_errors_are_reported(api):
    rc, n = shared(api, CUDA_NO_MEMORY, CUDA_NO_MEMORY)
    assert rc != 0 and n["latent"] == 0
    rc, n = shared(api, CUDA_INVALID)
    assert rc != 0 and n["latent"] == 0
