"""cache_append_q8 at the end of its range: turned keys that lie beside 448 * 2^60 by less than an fp32 sum of their products shows.

Up to there a number counts for the scale, which is then 2^60, and has the largest code; beyond it is NaN and does not count.
"""
import numpy as np
import pytest
import torch

from test_cache_q8_gpu import BF, Cache8, hsp, ints, numbers, turned, write  # noqa: F401  (hsp: the fixture)

pytestmark = pytest.mark.gpu
TOP = 448 * 2.0 ** 60


def sums_at_the_end(n, seed):
    """bf16 numbers a, b and fp32 numbers c, s such that a c - b s lies within 2^-24 of TOP, the exact sum and its fp32 form (fused
    with either product) on different sides of it or at it."""
    rng = np.random.default_rng(seed)
    got = []
    while len(got) < n:
        m = 400000
        a = np.ldexp((128 + rng.integers(0, 128, m)) / 128.0, 69)
        b = np.ldexp((128 + rng.integers(0, 128, m)) / 128.0, 67) * rng.choice([-1.0, 1.0], m)
        s = rng.uniform(0.3, 1.0, m).astype(np.float32)
        c = ((TOP + b * s.astype(np.float64)) / a).astype(np.float32)
        c = np.where(rng.random(m) < 0.5, np.nextafter(c, np.float32(2)), c)
        exact = a * c.astype(np.float64) - b * s.astype(np.float64)      # (fewer than 53 bits)
        p = (b * s.astype(np.float64)).astype(np.float32).astype(np.float64)
        fast = (a * c.astype(np.float64) - p).astype(np.float32).astype(np.float64)
        pick = ((fast > TOP) != (exact > TOP)) & (np.abs(exact / TOP - 1) < 2.0 ** -24)
        got += list(zip(a[pick], b[pick], c[pick], s[pick]))
    return got[:n]


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("page,block,rot", [(16, 1, 16), (16, 16, 16), (64, 64, 64)])
def test_sums_beside_the_end(hsp, page, block, rot, interleaved):
    """One such pair to a token, the first numbers of it at the end; every column of it there in some tokens."""
    pages, half = 3, rot // 2
    n, dim = pages * page, rot + 16
    c = Cache8(1, pages, page, block, 1, dim, None, 4)
    c.lens.copy_(ints([n]))
    found = sums_at_the_end(n * half, page + block)
    kn = torch.zeros(n, 1, dim, dtype=BF)
    cs = torch.zeros(n, rot)
    for t in range(n):
        for i in range(half if t % 3 == 0 else 1):
            a, b, co, si = found[t * half + i]
            one, two = (16 + 2 * i, 16 + 2 * i + 1) if interleaved else (16 + i, 16 + half + i)
            kn[t, 0, one], kn[t, 0, two] = float(a), float(b)
            cs[t, i], cs[t, half + i] = float(co), float(si)
    kn, cs = kn.cuda(), cs.cuda()
    x = turned(numbers(kn), numbers(cs), np.arange(n), interleaved)
    assert (x == TOP).sum() + (x > TOP).sum() > 0 and (x < TOP).sum() > 0
    m = c.model()
    hsp.cache_append_q8(kn, None, c.k, None, c.ks, None, c.table, c.lens, rows=ints([0] * n), positions=ints(list(range(n))), cos_sin=cs,
                        interleaved=interleaved)
    hsp.check_device_error()
    at = c.table.cpu().numpy()[0, np.arange(n) // page]
    write(m["k"], m["ks"], x, at, np.arange(n) % page, block)
    c.same(m)
