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
