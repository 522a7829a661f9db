"""proj_paged_attention_q8 over scales that are no powers of two, of keys and of values, up to the ends of their range; bounds as in
test_attention_q8_sums_gpu.py."""
import pytest
import torch

from test_attention_q8_gpu import F8, hsp, make  # noqa: F401  (hsp: the fixture)
from test_attention_q8_sums_gpu import KINDS, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("latent,dk,dv,heads,kv", KINDS)
@pytest.mark.parametrize("page,block,lens", [(16, 1, [300, 0, 5000]), (64, 16, [129, 1, 3000]), (128, 128, [2000, 77])])
def test_scales_of_any_value(hsp, latent, dk, dv, heads, kv, page, block, lens):
    args = make(lens, heads, kv, dk, latent, page, 200 + page, block=block, std=2.0 ** -3)
    g = torch.Generator(device="cuda").manual_seed(page)
    for s in args[3:5]:
        if s is not None:
            s.mul_(1 + torch.rand(s.shape, generator=g, device="cuda"))
    check(hsp, args, 0.1, dv)


@pytest.mark.parametrize("d,heads,kv", [(64, 8, 4), (128, 36, 2)])
@pytest.mark.parametrize("exponent", [-60, 59])
def test_scales_at_the_ends_of_the_range(hsp, d, heads, kv, exponent):
    """All values' scales next to 2^-60 or 2^60; all keys' next to 2^-60 under queries of 2^50 (scores of about one)."""
    args = list(make([700, 40], heads, kv, d, False, 16, 7, block=4, spread=0))
    g = torch.Generator(device="cuda").manual_seed(d)
    m = 1 + torch.rand(args[4].shape, generator=g, device="cuda") * 0.99
    args[4].copy_(m * 2.0 ** exponent)
    check(hsp, args, 0.1, d)
    args[3].copy_(m.flip(0) * 2.0 ** -60)
    args[0] = args[0] * 2.0 ** 50
    check(hsp, args, 0.5, d)


@pytest.mark.parametrize("latent,dk,dv,heads,kv", KINDS)
def test_queries_at_the_end_of_their_range(hsp, latent, dk, dv, heads, kv):
    """Queries of 2^120 over keys of 2^-54 and less: q . codes passes fp32's range, the scores are about one."""
    args = list(make([700, 40], heads, kv, dk, latent, 16, 9, block=4, spread=0, std=2.0 ** -48))
    args[0] = (args[0].float().clamp(-3, 3) * 2.0 ** 120).to(args[0].dtype)
    check(hsp, args, 2.0 ** -74, dv)
