"""The same sequences in a table that just holds them (one launch) and in one as wide as a server's (cut and joined):
both within the bounds of test_attention_gpu."""
import pytest
import torch

from test_attention_gpu import check, hsp, make  # noqa: F401  (hsp: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("latent,dk,dv", [(True, 576, 512), (True, 512, 512), (False, 128, 128), (False, 64, 64)])
@pytest.mark.parametrize("lens", [[1], [64], [77], [200], [0], [250, 0, 1, 63, 65, 129]])
def test_narrow_and_wide_tables(hsp, latent, dk, dv, lens):  # noqa: F811
    heads, kv = (16, 1) if latent else (8, 2)
    q, k, v, table, ln = make(lens, heads, kv, dk, latent, 16, 60 + len(lens))
    narrow = table[:, :16]
    assert narrow.shape[1] * 16 <= 256
    wide = torch.full((len(lens), 4096), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    n = hsp.launch_count()
    check(hsp, (q, k, v, narrow, ln), 0.07, dv)
    assert hsp.launch_count() == n + 1
    check(hsp, (q, k, v, wide, ln), 0.07, dv)
    assert hsp.launch_count() == n + 3
