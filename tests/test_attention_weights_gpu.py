"""The rounding of the softmax weights in proj_paged_attention.

The product with the values takes bf16 weights.  Divided by the sum of the same rounded weights, the rounding of
a token that has nearly all the weight cancels: with weights p1 (1 + e1) and p0 (1 + e0), |e| <= 2^-8,
    o = v p1 (1 + e1) / (p1 (1 + e1) + p0 (1 + e0))
is off by at most |e1 - e0| p0 / (p0 + p1) <= 2^-7 * 2^-6 = 2^-13 relative where p1 > 2^6 p0, besides the rounding
of the result (half a bf16 step) and 2^-18 for the fp32 scores and sums.
"""
import math

import pytest
import torch

from test_attention_gpu import BF, hsp, make, reference  # noqa: F401  (hsp: the module's fixture)

pytestmark = pytest.mark.gpu


def half_step(x):
    """Half the distance of neighbouring bf16 values around x (fp64), rounded up to the next binade at its border."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -120))) - 8)


# (first token, second token, length): in one part of an uncut call, and in the 51st of 152 parts
@pytest.mark.parametrize("low,high,n", [(3, 70, 130), (200 * 64 + 5, 201 * 64 + 9, 152 * 256)])
@pytest.mark.parametrize("latent,dk,dv", [(True, 576, 512), (False, 128, 128), (False, 64, 64)])
def test_a_token_with_all_the_weight_comes_out_as_it_is(hsp, latent, dk, dv, low, high, n):  # noqa: F811
    """Two tokens have scores far above all others, the second 6.1 to 7.9 (in log2) above the first, so that the
    first stays the reference point of the running softmax and the second has a weight of 2^6.1 to 2^7.9."""
    heads, page = 16, 64
    q, k, v, table, lens = make([n], heads, 1, dk, latent, page, 11)
    ids = table[0, : -(-n // page)].long()
    pool = k if latent else v
    kk = k[ids].flatten(0, 1)
    kk[:n] = 0
    vals = torch.randn(dv, generator=torch.Generator("cuda").manual_seed(5), device="cuda").to(BF)
    # the last column carries the scores (no value column of a latent cache of 576)
    kk[low, 0, dk - 1], kk[high, 0, dk - 1] = 64.0, 72.0
    if latent:
        kk[high, 0, :dv] = vals
    k[ids] = kk.view(-1, page, 1, dk)
    if not latent:
        vv = v[ids].flatten(0, 1)
        vv[:n] = 0
        vv[high, 0] = vals
        v[ids] = vv.view(-1, page, 1, dv)
    assert pool is not None
    q.zero_()
    q[0, :, dk - 1] = torch.linspace(6.1 / 8, 7.9 / 8, heads, device="cuda").to(BF)
    scale = math.log(2.0)                                   # scores in log2: 48.8 to 63.2 and 6.1 to 7.9 more
    out, lse = hsp.paged_attention(q, k, v, table, lens, scale, v_dim=dv, return_lse=True)
    hsp.check_device_error()
    ref, rlse, _, ltol = reference(q, k, v, table, lens, scale, dv)
    tol = half_step(ref) * (1 + 2.0 ** -8) + ref.abs() * (2.0 ** -13 + 2.0 ** -18)
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), f"{int((err > tol).sum())} of {err.numel()} off, by up to {float((err / tol).max()):.2f} of the bound"
    assert ((lse.double() - rlse).abs() <= ltol).all()
