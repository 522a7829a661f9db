"""cache_append_q8 into blocks whose scale another writer left, a power of two or not: the documented rule, code by code.

The scale stays where the new tokens ask for no more: code = x / s rounded once, ties to the even code (with s = 1.5 * 2^i many quotients of bf16
numbers are ties).  Where it grows, codes in front are rounded once from code * old / new.
"""
import numpy as np
import pytest
import torch

from test_cache_q8_gpu import BF, Cache8, append, hsp, ints, new_rows, numbers  # noqa: F401  (hsp: the fixture)

pytestmark = pytest.mark.gpu
SHORT = [1.5, 1.25, 1.75, 1.0, 1.875, 1.3125]


def cache(rows, page, block, kv, dk, dv, seed, short, top=3):
    """Scales of about 2^top, mantissas of a few bits or any."""
    c = Cache8(rows, 2, page, block, kv, dk, dv, seed)
    for s in (c.ks, c.vs):
        if s is not None:
            m = torch.tensor(SHORT, device="cuda")[torch.randint(0, len(SHORT), s.shape, generator=c.g, device="cuda")]
            if not short:
                m = 1 + torch.rand(s.shape, generator=c.g, device="cuda")
            s.copy_(m * 2.0 ** torch.randint(top - 3, top, s.shape, generator=c.g, device="cuda"))
    return c


def whole(c, n, kv, dim):
    """Small whole numbers: quotients by short scales that are ties between codes, or codes."""
    return torch.randint(-255, 256, (n, kv, dim), generator=c.g, device="cuda").to(BF)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("short", [True, False])
@pytest.mark.parametrize("dk,kv,dv,rot", [(576, 1, None, 64), (512, 1, None, 0), (128, 3, 128, 128), (80, 2, 48, 16)])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 4), (64, 64)])
def test_a_scale_that_stays(hsp, dk, kv, dv, rot, page, block, short, interleaved):
    c = cache(6, page, block, kv, dk, dv, 5 + block + dk, short)
    start = block // 4                                       # (tokens in front)
    n = block - start
    c.lens.copy_(ints([block] * 6))
    rows, pos = [r for r in range(6) for _ in range(n)], [start + i for _ in range(6) for i in range(n)]
    for make in (whole, lambda c, n, kv, dim: new_rows(c.g, n, kv, dim, spread=0.5)):
        keep = c.ks.clone()
        append(hsp, c, rows, pos, dk, kv, dv, rot, interleaved, kn=make(c, len(rows), kv, dk),
               vn=make(c, len(rows), kv, dv) if dv else None)
        assert torch.equal(keep, c.ks)                       # none of these grew


def test_units_shared_by_clusters(hsp):
    """So many latent tokens, a few long runs: several CTAs share a run, under scales that stay and scales that grow."""
    c = cache(60, 64, 64, 1, 576, None, 9, True)
    c.lens.copy_(ints([47] * 60))
    rows, pos = [r for r in range(60) for _ in range(40)], [7 + i for _ in range(60) for i in range(40)]
    append(hsp, c, rows, pos, 576, 1, None, 64, True, heads=2, kn=whole(c, 2400, 1, 576))
    append(hsp, c, rows, pos, 576, 1, None, 64, False, heads=2, kn=new_rows(c.g, 2400, 1, 576, spread=5.0) * 64)


@pytest.mark.parametrize("short", [True, False])
@pytest.mark.parametrize("dk,kv,dv,rot", [(576, 1, None, 64), (128, 8, 128, 0)])
def test_a_scale_that_grows(hsp, dk, kv, dv, rot, short):
    """Codes in front under a new power of two: products of 28 bits, next to the borders of codes too."""
    c = cache(8, 64, 64, kv, dk, dv, 7, short, top=-2)
    c.lens.copy_(ints([60] * 8))
    append(hsp, c, list(range(8)), [59] * 8, dk, kv, dv, rot, kn=whole(c, 8, kv, dk) * 4, vn=whole(c, 8, kv, dv) * 2 if dv else None)
    # scales by which a code falls behind a border by less than fp32 shows
    p = c.table[:, 0].long()
    odd = np.float32(1.0625) + np.float32(2.0) ** -23 * np.arange(1, 9, dtype=np.float32)
    c.ks[p, 0] = torch.tensor(odd, device="cuda")[:, None].expand(8, kv).contiguous()
    c.k.view(torch.uint8)[p, :59] = torch.randint(0x38, 0x7e, (8, 59, kv, dk), generator=c.g, device="cuda").to(torch.uint8)
    append(hsp, c, list(range(8)), [59] * 8, dk, kv, dv, rot, kn=whole(c, 8, kv, dk) * 64, vn=whole(c, 8, kv, dv) * 2 if dv else None)
