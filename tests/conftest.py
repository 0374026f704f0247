import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (runs the libcsa kernels)")


def pytest_collection_modifyitems(config, items):
    # GPU tests need a device; on a machine without one they are skipped rather
    # than failed, so that `-m "not gpu"` and a plain run both work there.
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)


@pytest.fixture(scope="module", autouse=True)
def status_word(request):
    """Every module that ran on the GPU leaves the device's status word clear (no bounded wait gave up)."""
    yield
    if "torch" not in sys.modules:
        return
    import torch
    if torch.cuda.is_available() and torch.cuda.is_initialized():
        import sparse_attention_kv_csa_gb300 as csa
        torch.cuda.synchronize()
        assert csa.csa_device_status() == 0, csa.csa_last_error_message()
