"""csa_torch is a short way, not a condition: the package imports and the helpers work where it cannot be built or loaded."""
import os
import subprocess
import sys

import pytest

import sparse_attention_kv_csa_gb300 as csa
from sparse_attention_kv_csa_gb300 import _build, serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_package_imports_beside_a_torch_without_headers(tmp_path):
    """A torch newer than the binding and without C++ headers: the Compressor's entry points need neither."""
    os.makedirs(tmp_path / "torch")
    for name in ("__init__.py", "version.py"):
        (tmp_path / "torch" / name).write_text("")
    code = "import sparse_attention_kv_csa_gb300 as csa, sys; csa.csa_version(); assert 'torch' not in sys.modules"
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT]))
    got = subprocess.run([sys.executable, "-c", code], env=env, cwd=str(tmp_path), capture_output=True, text=True)
    assert got.returncode == 0, got.stderr


def test_helpers_do_without(monkeypatch):
    torch = pytest.importorskip("torch")

    def fails(*_):
        raise RuntimeError("g++ failed for csa_torch:\nmany lines")

    monkeypatch.setattr(_build, "build_binding", fails)
    for name in ("_torch", "_short", "_e4m3"):
        monkeypatch.setattr(serving, name, None)
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="csa_torch is not to be had .g.. failed for csa_torch:.:"):
        with pytest.raises(ValueError):
            csa.rms_norm_forward(x)
    assert serving._short is None
    with pytest.raises(ValueError):
        csa.rms_norm_backward(x, x, None, torch.zeros(4))
    with pytest.raises(ValueError):
        csa.page_tables(i, i, 4, 16, i, i.view(2, 1), 4)
    with pytest.raises(ValueError):
        csa.latent_attention(x.view(4, 1, 8), x.view(2, 2, 8), i.view(2, 1), i, i[:1], 4, 1.0)


def test_build_reports_the_library_first_and_the_binding_too(monkeypatch):
    pytest.importorskip("torch")

    def binding(*_):
        raise RuntimeError("binding")

    def library(*_):
        raise RuntimeError("library")

    monkeypatch.setattr(_build, "binding_stale", lambda: True)
    monkeypatch.setattr(_build, "build_binding", binding)
    with pytest.raises(RuntimeError, match="binding"):
        _build.build()
    monkeypatch.setattr(_build, "build_library", library)
    with pytest.raises(RuntimeError, match="library"):
        _build.build()
