"""cache_read_q8 rounds code * scale once, whatever the scale: products that fp32 does not hold, next to the middle between two bf16
numbers, where a rounding to fp32 first would fall on the middle and then to the even one."""
import numpy as np
import pytest
import torch

from test_cache_q8_gpu import F8, GRID, Cache8, hsp, ints, numbers  # noqa: F401  (hsp: the fixture)

pytestmark = pytest.mark.gpu


def bf16_of(x):
    """Nearest bf16 number of positive normal 64-bit numbers, ties to the even one (code * scale has 28 bits: exact there)."""
    bits = x.view(np.uint64)
    drop = 52 - 7
    low, half = bits & np.uint64((1 << drop) - 1), np.uint64(1 << (drop - 1))
    up = (low > half) | ((low == half) & ((bits >> np.uint64(drop)) & np.uint64(1) == 1))
    return (((bits >> np.uint64(drop)) + up.astype(np.uint64)) << np.uint64(drop)).view(np.float64)


def near_middles(code, n=64):
    """fp32 scales whose exact product with `code` lies behind a middle between two bf16 numbers by less than half of fp32's last
    bit, so that fp32's product is the middle."""
    rng = np.random.default_rng(int(code * 1024))
    mid = (128 + rng.integers(0, 128, 200000) + 0.5) * 2.0 ** rng.integers(-20, 10, 200000)
    s = (mid / code).astype(np.float32)
    s = np.concatenate([s, np.nextafter(s, np.float32(0)), np.nextafter(s, np.float32(np.inf))])
    exact = s.astype(np.float64) * code
    twice = bf16_of((s * np.float32(code)).astype(np.float64))
    return s[twice != bf16_of(exact)][:n]


def test_products_next_to_a_middle(hsp):
    c = Cache8(1, 40, 64, 1, 1, 64, None, 5)
    codes, scales = [], []
    for g in (1.125, 1.375, 1.625, 1.875, 13.0, 208.0, 0.6875):
        assert g in GRID
        s = near_middles(g)
        codes += [g] * len(s)
        scales += s.tolist()
    n = len(codes)
    assert n > 200                                            # (there are such scales for codes of four bits)
    n = min(n, 40 * 64)
    c.lens.copy_(ints([n]))
    t = torch.arange(n, device="cuda")
    page, line = c.table[0].long()[t // 64], t % 64
    x = torch.tensor(codes[:n], device="cuda")
    sign = torch.where(torch.arange(64, device="cuda") % 2 == 0, 1.0, -1.0)
    c.k.view(torch.uint8)[page, line, 0] = (x[:, None] * sign).to(F8).view(torch.uint8)
    c.ks[page, line, 0] = torch.tensor(scales[:n], device="cuda", dtype=torch.float32)
    k, _ = hsp.cache_read_q8(c.k, None, c.ks, None, c.table, c.lens, rows=ints([0] * n), positions=t.to(torch.int32))
    hsp.check_device_error()
    want = bf16_of(np.array(scales[:n], dtype=np.float64) * np.array(codes[:n]))[:, None] * sign.cpu().numpy()
    assert np.array_equal(numbers(k)[:, 0], want)


@pytest.mark.parametrize("block", [1, 16])
def test_any_code_under_any_scale(hsp, block):
    """All codes, NaN among them, under scales over the whole range: the definition's number."""
    c = Cache8(2, 8, 64, block, 3, 256, None, 6)
    c.lens.copy_(ints([512, 300]))
    c.k.copy_(torch.arange(256, device="cuda").to(torch.uint8).view(F8).expand(c.k.shape))
    e = torch.randint(-60, 60, c.ks.shape, generator=c.g, device="cuda")
    c.ks.copy_((1 + torch.rand(c.ks.shape, generator=c.g, device="cuda")) * 2.0 ** e)
    c.ks[0, 0] = 2.0 ** 60
    t = torch.arange(512, device="cuda")
    k, _ = hsp.cache_read_q8(c.k, None, c.ks, None, c.table, c.lens, rows=ints([0] * 512), positions=t.to(torch.int32))
    hsp.check_device_error()
    page, line = c.table[0].long()[t // 64].cpu().numpy(), (t % 64).cpu().numpy()
    x = numbers(c.k.view(torch.uint8).view(F8))[page, line] * numbers(c.ks)[page, line // block][..., None]
    want = np.copysign(np.where(x == 0, 0.0, bf16_of(np.where(np.isnan(x) | (x == 0), 1.0, np.abs(x)))), x)
    want = np.where(np.isnan(x), np.nan, want)
    assert np.array_equal(numbers(k), want, equal_nan=True)
