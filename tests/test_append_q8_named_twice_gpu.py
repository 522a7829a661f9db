"""cache_append_q8 with a place named twice by neighbours: the block's scale is the documented one over both rows, the place holds numbers of
either under it."""
import numpy as np
import pytest
import torch

from test_cache_q8_gpu import Cache8, hsp, ints, nearest, new_rows, numbers  # noqa: F401  (hsp: the fixture)

pytestmark = pytest.mark.gpu


def exponent(most):
    e = -60
    while e < 60 and most > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("larger", [0, 1])
@pytest.mark.parametrize("page,block,start", [(16, 8, 8), (16, 8, 11), (64, 64, 5), (32, 1, 7)])
def test_the_scale_is_that_of_both_rows(hsp, page, block, start, larger, sign):
    """The larger row first or last, its largest number above or below zero; with and without tokens in front."""
    for old in (2.0 ** -8, 2.0 ** 12):
        c = Cache8(1, 2, page, block, 2, 64, 64, 21)
        c.lens.copy_(ints([2 * page]))
        for s in (c.ks, c.vs):
            s.fill_(old)
        kn, vn = new_rows(c.g, 2, 2, 64), new_rows(c.g, 2, 2, 64)
        for x in (kn, vn):
            x.clamp_(-3, 3)
            x[larger] *= 64
            x[larger, :, 5] = 500.0 * sign
        hsp.cache_append_q8(kn, vn, c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=ints([0, 0]), positions=ints([start, start]))
        hsp.check_device_error()
        p, line = int(c.table[0, start // page]), start % page
        for new, codes, scales in ((kn, c.k, c.ks), (vn, c.v, c.vs)):
            x = numbers(new)
            for h in range(2):
                want = exponent(np.abs(x[:, h]).max())
                if line % block > 0:
                    want = max(want, old)
                assert float(scales[p, line // block, h]) == want
                got = numbers(codes.view(torch.uint8)[p, line, h].view(codes.dtype))
                either = nearest(x[:, h] / want)
                assert ((got == either[0]) | (got == either[1])).all()
