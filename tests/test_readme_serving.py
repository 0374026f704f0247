"""README's lines on shared prefixes, rotated rows and layer norms, run as they stand: through the helpers' own checks without a GPU
(the entry points below them left out), and for real."""
import os
import re
import types

import pytest
import torch

import sparse_attention_kv_csa_gb300 as csa
from sparse_attention_kv_csa_gb300 import serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def lines():
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    text = text[text.index("have operators of their own:"):]
    return "\n".join(line.strip() for line in re.match(r"[^\n]*\n\n((?:    [^\n]*\n)+)", text).group(1).splitlines())


def names(device):
    """What the lines take as given: 3 requests behind a common prompt in pages of 64 rows, ratio 4, one new token and row each."""
    int32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
    randn = lambda *a: torch.randn(a, device=device)  # noqa: E731
    n = dict(csa=types.SimpleNamespace(**{k: getattr(csa, k) for k in serving.__all__}), n_positions=2000, scale=512 ** -0.5)
    n["csa"].rotation_table = lambda *a: csa.rotation_table(*a, device=device)
    n.update(cache=randn(12, 64, 512).bfloat16(), rows=randn(3, 512).bfloat16(), positions=int32(199, 200, 210),
             slots=torch.tensor([4 * 64 + 7, 5 * 64 + 8, 6 * 64 + 18], device=device), q=randn(3, 64, 512).bfloat16(),
             q_positions=int32(799, 803, 843), table=int32([0, 1, 2, 4], [0, 1, 2, 5], [0, 1, 2, 6]), cu_q=int32(0, 1, 2, 3),
             lens=int32(800, 804, 844), cu_groups=int32(0, 3), shared_rows=int32(192))
    n.update(x=randn(5, 96).bfloat16(), r=randn(5, 96).bfloat16(), weight=randn(96), bias=randn(96), grad_out=randn(5, 96).bfloat16(),
             g=randn(5, 96).bfloat16())
    return n


class Entries:
    """Entry points that do nothing, and which of them were called."""

    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        return lambda *a: self.called.append(name) or 0


def test_the_helpers_take_the_lines_arguments(monkeypatch):
    entries = Entries()
    monkeypatch.setattr(serving, "_lib", entries)
    for name, value in (("_torch", torch), ("_Tensor", torch.Tensor), ("_e4m3", torch.float8_e4m3fn)):
        monkeypatch.setattr(serving, name, value)
    for code, dtype in enumerate((torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn)):
        monkeypatch.setitem(serving._CODES, dtype, code)
    monkeypatch.setattr(serving, "_short", None)
    monkeypatch.setattr(serving, "_check_device", lambda t, name: t.get_device())
    monkeypatch.setattr(serving, "_handle", lambda stream, device: 0)
    n = names("cpu")
    exec(lines(), n)
    assert entries.called == ["csa_append_rows", "csa_shared_attention", "csa_rotate", "csa_layer_norm_fwd", "csa_layer_norm_bwd"]
    assert n["back"].shape == (3, 64, 64) and n["lse"].shape == (3, 64)


@pytest.mark.gpu
def test_the_lines_run():
    n = names("cuda")
    before = n["q"].clone()
    exec(lines(), n)
    torch.cuda.synchronize()
    assert csa.csa_device_status() == 0
    assert torch.equal(n["q"][..., :448], before[..., :448]) and not torch.equal(n["q"], before)
    want, lse = csa.latent_attention(n["q"], n["cache"], n["table"], n["cu_q"], n["lens"], 4, n["scale"])
    assert torch.equal(n["lse"], lse) and n["back"].shape == (3, 64, 64)
    assert all(n[k].isfinite().all() for k in ("back", "grad_x", "grad_weight", "grad_bias"))
