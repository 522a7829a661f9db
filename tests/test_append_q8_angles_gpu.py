"""cache_append_q8 where the angles end before the positions do: such tokens are reported and written nowhere, and nothing behind the
table of angles is read (a page that begins there has no angle at all)."""
import numpy as np
import pytest
import torch

from test_cache_q8_gpu import BF, Cache8, angles, hsp, ints, new_rows, numbers, turned, write  # noqa: F401  (hsp: the fixture)

pytestmark = pytest.mark.gpu


def run(hsp, c, rows, pos, dk, kv, dv, cs, interleaved, heads=2):
    n, most = len(rows), cs.shape[0]
    kn, vn = new_rows(c.g, n, kv, dk), new_rows(c.g, n, kv, dv) if dv else None
    q = torch.randn(n, heads, dk, generator=c.g, device="cuda").to(BF)
    kept = torch.full_like(q, 7.0)
    m, table = c.model(), c.table.cpu().numpy()
    hsp.cache_append_q8(kn, vn, c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=ints(rows), positions=ints(pos), cos_sin=cs,
                        interleaved=interleaved, q=q, q_out=kept)
    with pytest.raises(hsp.ProjError) as e:
        hsp.check_device_error()
    assert e.value.status_name == "PROJ_ERR_BAD_INDEX"
    at = np.array([table[r, p // c.page] if p < most else -1 for r, p in zip(rows, pos)])
    line = np.array(pos) % c.page
    cs64 = cs.cpu().numpy().astype(np.float64)
    write(m["k"], m["ks"], turned(numbers(kn), cs64, np.minimum(pos, most - 1), interleaved), at, line, c.block)
    if dv:
        write(m["v"], m["vs"], numbers(vn), at, line, c.block)
    c.same(m)
    far = torch.tensor([p >= most for p in pos], device="cuda")
    assert bool((kept[far] == 7).all())                      # queries without angles stay as they are


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dk,kv,dv,rot,page,block", [(576, 1, None, 64, 64, 64), (128, 3, 128, 128, 16, 16), (64, 2, 64, 32, 32, 1)])
def test_angles_that_end_inside_a_page(hsp, dk, kv, dv, rot, page, block, interleaved):
    """The table ends in the middle of a page: a run of tokens on both sides of the end, and pages without any angle behind."""
    most = page + page // 2 + 3
    c = Cache8(2, 5, page, block, kv, dk, dv, 3)
    c.lens.copy_(ints([5 * page, 4 * page]))
    pos = list(range(page // 2, 4 * page - 1))
    run(hsp, c, [0] * len(pos), pos, dk, kv, dv, angles(most, rot), interleaved)
    run(hsp, c, [0, 1, 1], [5 * page - 1, most, most - 1], dk, kv, dv, angles(most, rot), interleaved)


@pytest.mark.parametrize("dk,kv,dv,rot", [(576, 1, None, 64), (128, 8, 128, 128)])
def test_positions_far_behind_the_angles(hsp, dk, kv, dv, rot):
    """Tables as long as 2^28 tokens, 16 angles: few tokens, and as many as fill the GPU (chunks, clusters)."""
    page = 64
    c = Cache8(1, 4, page, 64, kv, dk, dv, 8)
    wide = c.table.repeat(1, 2 ** 20).contiguous()           # four pages again and again: 2^28 positions
    c.table, c.lens = wide, ints([2 ** 28])
    for n in (1, 9, 2200):
        pos = [2 ** 28 - n + i for i in range(n)]
        m = c.model()
        kn, vn = new_rows(c.g, n, kv, dk), new_rows(c.g, n, kv, dv) if dv else None
        hsp.cache_append_q8(kn, vn, c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=ints([0] * n), positions=ints(pos), cos_sin=angles(16, rot))
        with pytest.raises(hsp.ProjError):
            hsp.check_device_error()
        c.same(m)
    pos = [2 ** 28 - 1, 3, 15, 2 ** 27]                      # and between them tokens that have theirs
    run(hsp, c, [0] * 4, pos, dk, kv, dv, angles(16, rot), True)
