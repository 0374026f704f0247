"""Numbers that pass the entry points' integers, without a GPU: refused, not wrapped."""
import pytest

import sparse_attention_kv_csa_gb300 as csa

A = 1 << 20  # an aligned fake address; validation fails before it is used


@pytest.mark.parametrize("tokens,heads", [(1 << 60, 16), (1 << 62, 4), ((1 << 60) + 1, 16), (1 << 31, 1), (1 << 30, 2)])
def test_tokens_times_heads_does_not_wrap(tokens, heads):
    with pytest.raises(csa.CSAError) as e:
        csa.csa_latent_attention(None, 64 * heads, 64, A, 1, tokens, heads, 64, 64, A, 64, 0, None, 4, 16, A, 2, 2, A, 4, 1.0,
                                 None, A, A, stream=0)
    assert e.value.status == 4, csa.csa_last_error_message()


WIDE = 1 << 32  # what 32 bits would cut off


def attention(**kw):
    a = dict(q=A, q_token_stride=64, q_head_stride=64, cu_q=A, n_req=1, n_tokens=2, n_heads=1, head_dim=64, v_dim=64, cache=A,
             cache_stride=64, cache_dtype=0, row_scales=None, n_pages=4, page_size=16, block_table=A, table_stride=2, width=2,
             seq_lens=A, ratio=4, scale=1.0, sink=None, out=A + 4, lse=A, stream=0)  # out is refused, so nothing is launched
    csa.csa_latent_attention(**{**a, **kw})


def norm(**kw):
    a = dict(x=A + 1, x_stride=8, residual=None, residual_stride=0, weight=None, n_rows=2, dim=8, eps=1e-6, dtype=0, slots=None,
             n_slots=0, out=A, out_stride=8, out_dtype=0, scales=None, scale_group=0, residual_out=None, rstd=None, stream=0)
    csa.csa_rms_norm_fwd(**{**a, **kw})


def norm_gradient(**kw):
    a = dict(h=A + 1, h_stride=8, grad_out=A, grad_out_stride=8, grad_residual=None, grad_residual_stride=0, weight=None, rstd=A,
             n_rows=2, dim=8, dtype=0, grad_x=A, grad_weight=None, stream=0)
    csa.csa_rms_norm_bwd(**{**a, **kw})


def pages(**kw):
    a = dict(before=A, after=A, n_req=2, ratio=4, page_size=16, free_pages=A, n_free=3, taken=None, table=A, table_stride=4, width=4,
             capacity=8, table_out=A + 4096, cu_rows=A, slots=A + 4, counts=A, stream=0)
    csa.csa_page_tables(**{**a, **kw})


@pytest.mark.parametrize("call,name", [
    *[(attention, n) for n in ("n_req", "n_heads", "head_dim", "v_dim", "cache_dtype", "page_size", "width", "ratio")],
    *[(norm, n) for n in ("dim", "dtype", "out_dtype", "scale_group")], (norm_gradient, "dim"), (norm_gradient, "dtype"),
    *[(pages, n) for n in ("n_req", "ratio", "page_size", "n_free", "width")]])
@pytest.mark.parametrize("sign", [1, -1])
def test_numbers_past_32_bits(call, name, sign):
    with pytest.raises(csa.CSAError):
        call()  # as it stands the call is refused for a misaligned address
    with pytest.raises(ValueError, match=name):
        call(**{name: sign * WIDE + 64})


@pytest.mark.parametrize("call,name", [
    (attention, "n_tokens"), (attention, "n_pages"), (attention, "cache_stride"), (norm, "n_rows"), (norm, "x_stride"),
    (norm_gradient, "n_rows"), (pages, "capacity"), (pages, "table_stride")])
def test_numbers_past_64_bits(call, name):
    with pytest.raises(ValueError, match=name):
        call(**{name: (1 << 64) + 64})


def test_helpers_take_no_number_past_32_bits():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="ratio"):
        csa.page_tables(i, i, WIDE + 4, 16, i, i.view(2, 1), 4)
    with pytest.raises(ValueError, match="page_size"):
        csa.page_tables(i, i, 4, WIDE + 16, i, i.view(2, 1), 4)
    with pytest.raises(ValueError, match="ratio"):
        csa.latent_attention(q, q.view(1, 2, 64), i[:1].view(1, 1), i, i[:1], WIDE + 1, 1.0)
    with pytest.raises(ValueError, match="v_dim"):
        csa.latent_attention(q, q.view(1, 2, 64), i[:1].view(1, 1), i, i[:1], 1, 1.0, v_dim=WIDE + 64)
