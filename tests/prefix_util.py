"""The choice between reading prefixes apart and request by request, compiled from the kernels' header, for tests that are meant for
one of the two ways."""
import ctypes
import functools
import os
import subprocess
import tempfile

TESTS = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(TESTS), "sparse_attention_kv_csa_gb300", "csrc")


@functools.lru_cache(None)
def choice():
    so = os.path.join(tempfile.mkdtemp(), "prefix_choice.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I" + CSRC, os.path.join(TESTS, "prefix_choice_host.cpp"), "-o", so])
    lib = ctypes.CDLL(so)
    for f in (lib.choice_apart, lib.choice_image_rows):
        f.argtypes = [ctypes.c_longlong, ctypes.POINTER(ctypes.c_int), ctypes.c_longlong] + ([ctypes.c_int] if f is lib.choice_apart else [])
    return lib


def _call(tokens, heads, requests, groups, dim, v_dim, bits8, pages, page, width):
    return tokens, (ctypes.c_int * 8)(heads, requests, groups, dim, v_dim, bits8, page, width), pages


def apart(*call, sms=152):
    """call: tokens, heads, requests, groups, head_dim, v_dim, bits8, pages of the cache, rows of a page, pages of a table."""
    return bool(choice().choice_apart(*_call(*call), sms))


def image_rows(*call):
    return choice().choice_image_rows(*_call(*call))


def read_apart(a, v_dim=None):
    """Whether shared_attention(**a) reads prefixes apart on the current device."""
    import torch
    q, cache = a["q"], a["cache"]
    sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return apart(q.shape[0], q.shape[1], a["seq_lens"].numel(), a["shared_rows"].numel(), q.shape[2], q.shape[2] if v_dim is None else v_dim,
                 cache.dtype != torch.bfloat16, cache.shape[0], cache.shape[1], a["block_table"].shape[1], sms=sms)
