"""The layer norm, the append, the rotation and the shared attention without a GPU: refusals of the C entry points (before any
CUDA call) and of the helpers."""
import pytest
import torch

import sparse_attention_kv_csa_gb300 as csa

A = 1 << 20  # an aligned fake address; validation fails before it is used
WIDE = 1 << 32


def layer_fwd(**kw):
    a = dict(x=A, x_stride=512, residual=A, residual_stride=512, weight=A, bias=A, n_rows=4, dim=512, eps=1e-5, dtype=0, out=A,
             out_stride=512, residual_out=A, mean=A, rstd=A, stream=0)
    csa.csa_layer_norm_fwd(**{**a, **kw})


def layer_bwd(**kw):
    a = dict(h=A, h_stride=8, grad_out=A, grad_out_stride=8, grad_residual=A, grad_residual_stride=8, weight=A, mean=A, rstd=A,
             n_rows=4, dim=8, dtype=0, grad_x=A, grad_weight=A, grad_bias=A, stream=0)
    csa.csa_layer_norm_bwd(**{**a, **kw})


def append(**kw):
    a = dict(rows=A, row_stride=512, row_dim=512, rotary=A, rotary_stride=64, rot_dim=64, positions=A, n_rows=4, dtype=0, rotation=A,
             n_positions=10, interleaved=0, slots=A, n_slots=9, out=A, out_stride=576, out_dtype=0, scales=None, q=A, q_token_stride=1024,
             q_head_stride=64, q_positions=A, n_tokens=3, n_heads=16, q_out=A, q_out_token_stride=1024, q_out_head_stride=64, stream=0)
    csa.csa_append_rows(**{**a, **kw})


def rotate(**kw):
    a = dict(x=A, x_token_stride=1024, x_head_stride=64, positions=A, n_tokens=3, n_heads=16, rot_dim=64, dtype=0, rotation=A,
             n_positions=10, interleaved=1, inverse=0, out=A, out_token_stride=1024, out_head_stride=64, stream=0)
    csa.csa_rotate(**{**a, **kw})


def shared(**kw):
    a = dict(q=A, q_token_stride=64, q_head_stride=64, cu_q=A, n_req=1, n_tokens=2, n_heads=1, head_dim=64, v_dim=64, cache=A,
             cache_stride=64, cache_dtype=0, row_scales=None, n_pages=4, page_size=16, block_table=A, table_stride=2, width=2,
             seq_lens=A, cu_groups=A, shared_rows=A, n_groups=1, ratio=4, scale=1.0, sink=None, out=A, lse=A, stream=0)
    csa.csa_shared_attention(**{**a, **kw})


CASES = [
    *[(layer_fwd, kw, s) for kw, s in [
        (dict(n_rows=-1), 1), (dict(n_rows=1 << 31), 1), (dict(dim=0), 2), (dict(dim=16385), 2), (dict(dtype=3), 2), (dict(eps=-1.0), 1),
        (dict(eps=float("nan")), 1), (dict(x_stride=511), 1), (dict(residual_stride=511), 1), (dict(out_stride=511), 1), (dict(x=None), 1),
        (dict(out=None), 1), (dict(x=A + 1), 3), (dict(weight=A + 2), 3), (dict(bias=A + 2), 3), (dict(mean=A + 1), 3), (dict(rstd=A + 2), 3),
        (dict(residual_out=A + 1), 3)]],
    *[(layer_bwd, kw, s) for kw, s in [
        (dict(n_rows=-1), 1), (dict(dim=0), 2), (dict(dtype=3), 2), (dict(h_stride=7), 1), (dict(grad_out_stride=7), 1),
        (dict(grad_residual_stride=7), 1), (dict(h=None), 1), (dict(grad_out=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1),
        (dict(grad_x=None), 1), (dict(h=A + 1), 3), (dict(grad_weight=A + 2), 3), (dict(grad_bias=A + 1), 3), (dict(mean=A + 2), 3)]],
    *[(append, kw, s) for kw, s in [
        (dict(n_rows=-1), 1), (dict(n_rows=1 << 31), 1), (dict(n_slots=-1), 1), (dict(dtype=3), 2), (dict(out_dtype=2), 2), (dict(rot_dim=63), 2),
        (dict(rot_dim=0), 2), (dict(rot_dim=1026, rotary_stride=1026), 2), (dict(row_dim=0), 2), (dict(row_dim=1024, row_stride=1024), 2),
        (dict(rotary=None, row_dim=62), 2), (dict(row_stride=511), 1), (dict(rotary_stride=63), 1), (dict(out_stride=575), 1),
        (dict(n_positions=-1), 1), (dict(n_tokens=-1), 1), (dict(n_heads=0), 1), (dict(n_tokens=1 << 30), 4), (dict(rows=None), 1),
        (dict(positions=None), 1), (dict(slots=None), 1), (dict(rotation=None), 1), (dict(out=None), 1), (dict(out_dtype=3), 1),
        (dict(q=None), 1), (dict(q_positions=None), 1), (dict(q_out=None), 1), (dict(rows=A + 1), 3), (dict(rotary=A + 1), 3),
        (dict(slots=A + 4), 3), (dict(positions=A + 2), 3), (dict(rotation=A + 2), 3), (dict(q=A + 1), 3), (dict(q_out=A + 1), 3),
        (dict(q_token_stride=63), 1), (dict(q_head_stride=63), 1), (dict(q_out_token_stride=63), 1), (dict(q_out_head_stride=63), 1),
        (dict(out_dtype=3, scales=A + 2), 3)]],
    *[(rotate, kw, s) for kw, s in [
        (dict(n_tokens=-1), 1), (dict(n_heads=0), 1), (dict(rot_dim=65), 2), (dict(dtype=3), 2), (dict(n_tokens=1 << 31, n_heads=1), 4),
        (dict(n_tokens=1 << 62, n_heads=4), 4), (dict(x=None), 1), (dict(out=None), 1), (dict(positions=None), 1), (dict(rotation=None), 1),
        (dict(x_head_stride=63), 1), (dict(out_token_stride=2), 1), (dict(x=A + 1), 3), (dict(out=A + 1), 3), (dict(positions=A + 1), 3)]],
    *[(shared, kw, s) for kw, s in [
        (dict(n_groups=-1), 1), (dict(n_groups=14001), 4), (dict(cu_groups=None), 1), (dict(shared_rows=None), 1), (dict(cu_groups=A + 2), 3),
        (dict(shared_rows=A + 1), 3), (dict(n_req=-1), 1), (dict(n_heads=4097), 4), (dict(n_req=14001), 4), (dict(head_dim=60), 2),
        (dict(cache_dtype=1), 2), (dict(q=None), 1), (dict(out=A + 4), 3), (dict(scale=0.0), 1), (dict(cu_groups=None, n_groups=0, q=A + 2), 3),
        (dict(n_tokens=1 << 60, n_heads=16), 4)]],
]


@pytest.mark.parametrize("call,kw,status", CASES)
def test_refusals(call, kw, status):
    with pytest.raises(csa.CSAError) as e:
        call(**kw)
    assert e.value.status == status and csa.csa_last_error_message()


def test_nothing_to_do_needs_nothing():
    layer_fwd(n_rows=0, x=None, residual=None, out=None, weight=None, bias=None, residual_out=None, mean=None, rstd=None)
    layer_bwd(n_rows=0, h=None, grad_out=None, grad_residual=None, weight=None, mean=None, rstd=None, grad_x=None, grad_weight=None, grad_bias=None)
    append(n_rows=0, n_tokens=0, rows=None, rotary=None, positions=None, rotation=None, slots=None, out=None, q=None, q_positions=None, q_out=None)
    append(n_slots=0, out=None, n_tokens=0)
    rotate(n_tokens=0, x=None, positions=None, rotation=None, out=None)
    shared(n_tokens=0, q=None, cu_q=None, cache=None, block_table=None, seq_lens=None, cu_groups=None, shared_rows=None, n_groups=0, out=None)


@pytest.mark.parametrize("call,name", [
    *[(layer_fwd, n) for n in ("dim", "dtype")], (layer_bwd, "dim"), *[(append, n) for n in ("row_dim", "rot_dim", "dtype", "out_dtype", "n_heads")],
    *[(rotate, n) for n in ("n_heads", "rot_dim", "dtype")], *[(shared, n) for n in ("n_req", "page_size", "width", "n_groups", "ratio", "head_dim")]])
@pytest.mark.parametrize("sign", [1, -1])
def test_numbers_past_32_bits(call, name, sign):
    with pytest.raises(ValueError, match=name):
        call(**{name: sign * WIDE + 64})


@pytest.mark.parametrize("call,name", [(layer_fwd, "n_rows"), (layer_bwd, "h_stride"), (append, "n_slots"), (append, "q_out_head_stride"),
                                       (rotate, "n_tokens"), (rotate, "out_token_stride"), (shared, "n_pages")])
def test_numbers_past_64_bits(call, name):
    with pytest.raises(ValueError, match=name):
        call(**{name: (1 << 64) + 64})


def test_helpers_refuse_host_tensors_and_wrong_types():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    i, v = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError):
        csa.layer_norm_forward(x)
    with pytest.raises(TypeError):
        csa.layer_norm_forward(None)
    with pytest.raises(ValueError):
        csa.layer_norm_backward(x, x, None, v, v)
    with pytest.raises(ValueError):
        csa.append_rows(x, i, torch.zeros(3, 4), i.long(), x)
    with pytest.raises(ValueError):
        csa.rotate(x.view(4, 1, 8), i, torch.zeros(3, 8))
    with pytest.raises(ValueError):
        csa.rotate(x, i, torch.zeros(3, 8))
    with pytest.raises(TypeError):
        csa.rotate(None, i, torch.zeros(3, 8))
    with pytest.raises(ValueError):
        csa.shared_attention(x.view(4, 1, 8), x.view(2, 2, 8), i.view(4, 1), i, i[:1], i[:2], i[:1], 4, 1.0)


def test_rotation_table_on_the_host():
    t = csa.rotation_table(5, 4, 100.0, device="cpu")
    at = torch.arange(5).double()
    want = torch.stack([at.cos(), (at / 10).cos(), at.sin(), (at / 10).sin()], 1)
    assert t.dtype == torch.float32 and (t.double() - want).abs().max() <= 2.0 ** -25
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(n_positions=-1), dict(base=0.0)):
        with pytest.raises(ValueError):
            csa.rotation_table(**{**dict(n_positions=2, rot_dim=4, device="cpu"), **bad})
