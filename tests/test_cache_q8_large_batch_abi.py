"""Batches whose queries' images pass 2^40 bytes: the call refuses them, and so does the size of its workspace (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def hsp():
    from hidden_state_projection_gb300 import build
    build.build()
    import hidden_state_projection_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("heads,kv,dk,dv,latent", [(128, 1, 576, 512, True), (512, 1, 512, 512, True), (4096, 64, 128, 128, False)])
def test_a_batch_that_is_too_large(hsp, heads, kv, dk, dv, latent):
    per = 2 * heads * dk                                     # (64 heads to a tile: no more than its own bytes and a unit each)
    assert hsp.paged_attention_q8_workspace_bytes(2 ** 39 // per, heads, kv, dk, dv, latent) > 2 ** 38
    for batch in (2 ** 40 // per + 1, 2 ** 31 - 1):
        with pytest.raises(hsp.ProjError) as e:
            hsp.paged_attention_q8_workspace_bytes(batch, heads, kv, dk, dv, latent)
        assert e.value.status_name == "PROJ_ERR_UNSUPPORTED_SHAPE" and "too large" in str(e.value)
        assert hsp.lib().proj_paged_attention_q8_workspace_bytes(batch, heads, kv, dk, dv, int(latent)) == 0
