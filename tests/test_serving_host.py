"""The serving operators without a GPU: refusals of the C entry points (before any CUDA call) and of the helpers, and
the plain forms that the GPU tests compare with."""
import pytest
import torch

import serving_util as u
import sparse_attention_kv_csa_gb300 as csa

A = 1 << 20  # an aligned fake address; validation fails before it is used


def norm_fwd(**kw):
    a = dict(x=A, xs=512, res=A, rs=512, w=A, n=4, dim=512, eps=1e-6, dt=0, slots=None, ns=0, out=A, os=512, odt=0,
             scales=None, group=0, total=A, rstd=A)
    a.update(kw)
    csa.csa_rms_norm_fwd(a["x"], a["xs"], a["res"], a["rs"], a["w"], a["n"], a["dim"], a["eps"], a["dt"], a["slots"],
                         a["ns"], a["out"], a["os"], a["odt"], a["scales"], a["group"], a["total"], a["rstd"], stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(dim=0), 2), (dict(dim=16385), 2), (dict(dt=3), 2), (dict(odt=2), 2),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(group=64, odt=3, scales=A), 2), (dict(xs=511), 1),
    (dict(rs=511), 1), (dict(os=511), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(odt=3), 1), (dict(x=A + 1), 3),
    (dict(w=A + 2), 3), (dict(slots=A + 4, ns=8), 3), (dict(slots=A, ns=-1), 1), (dict(rstd=A + 2), 3),
    (dict(group=128, odt=3, scales=A, xs=513), 3), (dict(group=128, odt=3, scales=A, out=A + 4), 3),
    (dict(group=128, dim=576, xs=576, rs=576, os=576, odt=3, scales=A), 2),
])
def test_norm_refusals(kw, status):
    with pytest.raises(csa.CSAError) as e:
        norm_fwd(**kw)
    assert e.value.status == status and csa.csa_last_error_message()


def test_no_rows_needs_nothing():
    norm_fwd(n=0, x=None, res=None, out=None, w=None, total=None, rstd=None)
    csa.csa_rms_norm_bwd(None, 8, None, 8, None, 0, None, None, 0, 8, 0, None, None, stream=0)
    csa.csa_latent_attention(None, 64, 64, None, 0, 0, 1, 64, 64, None, 64, 0, None, 0, 1, None, 0, 0, None, 1, 1.0,
                             None, None, None, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(dim=0), 2), (dict(dt=3), 2), (dict(hs=7), 1), (dict(gs=7), 1), (dict(h=None), 1),
    (dict(g=None), 1), (dict(rstd=None), 1), (dict(dx=None), 1), (dict(h=A + 1), 3), (dict(dw=A + 2), 3),
    (dict(res=A, rs=7), 1),
])
def test_norm_gradient_refusals(kw, status):
    a = dict(h=A, hs=8, g=A, gs=8, res=None, rs=0, w=A, rstd=A, n=4, dim=8, dt=0, dx=A, dw=A)
    a.update(kw)
    with pytest.raises(csa.CSAError) as e:
        csa.csa_rms_norm_bwd(a["h"], a["hs"], a["g"], a["gs"], a["res"], a["rs"], a["w"], a["rstd"], a["n"], a["dim"],
                             a["dt"], a["dx"], a["dw"], stream=0)
    assert e.value.status == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(ratio=0), 1), (dict(page=0), 1), (dict(nf=-1), 1), (dict(width=-1), 1), (dict(cap=-1), 1),
    (dict(n=14001), 2), (dict(stride=3), 1), (dict(before=None), 1), (dict(after=None), 1), (dict(free=None), 1),
    (dict(table=None), 1), (dict(out=None), 1), (dict(cu=None), 1), (dict(slots=None), 1), (dict(counts=None), 1),
    (dict(slots=A + 4), 3), (dict(taken=A + 1), 3), (dict(out=A, stride=5), 1),
])
def test_page_table_refusals(kw, status):
    a = dict(before=A, after=A, n=2, ratio=4, page=16, free=A, nf=3, taken=None, table=A, stride=4, width=4, cap=8,
             out=A + 4096, cu=A, slots=A, counts=A)
    a.update(kw)
    with pytest.raises(csa.CSAError) as e:
        csa.csa_page_tables(a["before"], a["after"], a["n"], a["ratio"], a["page"], a["free"], a["nf"], a["taken"],
                            a["table"], a["stride"], a["width"], a["cap"], a["out"], a["cu"], a["slots"], a["counts"],
                            stream=0)
    assert e.value.status == status


@pytest.mark.parametrize("kw,status", [
    (dict(r=-1), 1), (dict(n=-1), 1), (dict(h=0), 1), (dict(page=0), 1), (dict(ratio=0), 1), (dict(d=4), 2),
    (dict(d=1032), 2), (dict(d=60), 2), (dict(v=72), 2), (dict(v=0), 2), (dict(v=12), 2), (dict(dt=1), 2),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(h=4097), 4),
    (dict(n=1 << 30, h=4), 4), (dict(pages=1 << 26, page=64), 4), (dict(width=1 << 26, stride=1 << 26, page=64), 4),
    (dict(qt=32), 1), (dict(qh=32), 1), (dict(cs=32), 1), (dict(stride=1), 1), (dict(qt=68), 3), (dict(cs=68), 3),
    (dict(dt=3, cs=72, rs=A), 3), (dict(q=None), 1), (dict(cu=None), 1), (dict(lens=None), 1), (dict(cache=None), 1),
    (dict(table=None), 1), (dict(dt=3), 1), (dict(out=None), 1), (dict(q=A + 2), 3), (dict(out=A + 4), 3),
    (dict(sink=A + 1), 3), (dict(lse=A + 2), 3),
])
def test_attention_refusals(kw, status):
    a = dict(q=A, qt=64, qh=64, cu=A, r=1, n=2, h=1, d=64, v=64, cache=A, cs=64, dt=0, rs=None, pages=4, page=16, table=A,
             stride=2, width=2, lens=A, ratio=4, scale=1.0, sink=None, out=A, lse=A)
    a.update(kw)
    with pytest.raises(csa.CSAError) as e:
        csa.csa_latent_attention(a["q"], a["qt"], a["qh"], a["cu"], a["r"], a["n"], a["h"], a["d"], a["v"], a["cache"],
                                 a["cs"], a["dt"], a["rs"], a["pages"], a["page"], a["table"], a["stride"], a["width"],
                                 a["lens"], a["ratio"], a["scale"], a["sink"], a["out"], a["lse"], stream=0)
    assert e.value.status == status


def test_helpers_refuse_host_tensors_and_wrong_types():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        csa.rms_norm_forward(x)
    with pytest.raises(TypeError):
        csa.rms_norm_forward(None)
    with pytest.raises(ValueError):
        csa.rms_norm_forward(x.double())
    with pytest.raises(ValueError):
        csa.rms_norm_backward(x, x, None, torch.zeros(4))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        csa.page_tables(i, i, 4, 16, i, i.view(2, 1), 4)
    with pytest.raises(ValueError):
        csa.page_tables(i.long(), i, 4, 16, i, i.view(2, 1), 4)
    with pytest.raises(ValueError):
        csa.latent_attention(x.view(4, 1, 8), x.view(2, 2, 8), i.view(2, 1), i, i[:1], 4, 1.0)


def test_plain_attention_by_hand():
    # two visible rows with equal logits: the mean of the values; the sink halves it
    q = torch.zeros(1, 1, 8, dtype=torch.bfloat16)
    cache = torch.arange(16, dtype=torch.float32).view(1, 2, 8).bfloat16()
    table, cu = torch.zeros(1, 1, dtype=torch.int32), torch.tensor([0, 1])
    out, lse, *_ = u.attention64(q, cache, table, cu, torch.tensor([8]), 4, 1.0, 8)
    assert torch.equal(out[0, 0], torch.arange(8) + 4.0) and abs(lse.item() - 0.6931471805599453) < 1e-12
    out, *_ = u.attention64(q, cache, table, cu, torch.tensor([4]), 4, 1.0, 8, sink=torch.zeros(1))
    assert torch.equal(out[0, 0], torch.arange(8) / 2.0)
    out, lse, *_ = u.attention64(q, cache, table, cu, torch.tensor([3]), 4, 1.0, 8)
    assert out.abs().max() == 0 and lse.item() == float("-inf")


def test_plain_pages_by_hand():
    table, cu, slots, counts = u.pages_plain([0, 8], [9, 12], 4, 2, [5, 6, 7], [[-1, -1], [3, -1]], 4)
    assert table == [[5, -1], [3, 6]] and cu == [0, 2, 3] and slots == [10, 11, 12, -1] and counts == [3, 2, 0, 2]
