"""The paged cache's calls stay inside the workspaces that their size queries ask for: the bytes in front of and behind a
workspace of exactly that size keep their pattern, and the results are those of a call that takes its own."""
import pytest
import torch

from test_attention_gpu import make
from test_cache_gpu import hsp  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu
GUARD, PATTERN = 4096, 0x5A


def guarded(need):
    buf = torch.full((need + 2 * GUARD,), PATTERN, dtype=torch.uint8, device="cuda")
    return buf, buf[GUARD:GUARD + need]


def untouched(buf):
    assert (buf[:GUARD] == PATTERN).all() and (buf[-GUARD:] == PATTERN).all()
    assert (buf[GUARD:-GUARD] != PATTERN).any()


# every instance of the kernel (columns; 16, 32 and 64 heads), and more heads than one tile holds
@pytest.mark.parametrize("group", [1, 16, 20, 32, 50, 64, 100, 200])
@pytest.mark.parametrize("dk,dv,kv", [(576, 512, 1), (512, 512, 2), (128, 128, 2), (64, 64, 3)])
def test_attention(hsp, dk, dv, kv, group):  # noqa: F811
    lens = [4000, 9, 2500, 0, 64, 700, 65, 1300, 1, 5100]
    args = make(lens, kv * group, kv, dk, dv == 512, 64, 40 + group)
    assert args[3].shape[1] * 64 > 256                      # sequences may be cut
    buf, ws = guarded(hsp.paged_attention_workspace_bytes(kv * group, kv, dk, dv, dv == 512))
    want = hsp.paged_attention(*args, 0.07, return_lse=True)
    n = hsp.launch_count()
    got = hsp.paged_attention(*args, 0.07, return_lse=True, workspace=ws)
    assert hsp.launch_count() == n + 2
    hsp.check_device_error()
    untouched(buf)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    bare = hsp.paged_attention(*args, 0.07, workspace=ws)   # without lse: the parts hold less
    assert torch.equal(bare, want[0])
    untouched(buf)


def cache(rows, width, pages, page):
    pool = torch.randint(-9, 9, (1, pages, page, 8), device="cuda").to(torch.int16)
    return (torch.full((rows, width), -1, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda"),
            torch.zeros(pages, dtype=torch.int32, device="cuda")), pool


@pytest.mark.parametrize("rows,pages", [(300, 5000), (1025, 5001), (40, 4097), (1, 9000)])
def test_resize(hsp, rows, pages):  # noqa: F811
    """Every row of the table grows on a page that another one holds, and takes two more: two launches."""
    page = 16
    a, pool = cache(2 * rows, 4, pages, page)
    first, second = (torch.arange(k * rows, (k + 1) * rows, dtype=torch.int32, device="cuda") for k in (0, 1))
    assert not hsp.cache_resize(*a, first, torch.full_like(first, 5), page, [pool]).any()
    assert not hsp.cache_fork(*a, first, second, page).any()
    state = [t.clone() for t in (*a, pool)]
    new = torch.full_like(first, 40)
    hsp.cache_resize(*a, second, new, page, [pool])
    want = [t.clone() for t in (*a, pool)]
    for t, o in zip((*a, pool), state):
        t.copy_(o)
    buf, ws = guarded(hsp.cache_workspace_bytes(a[0], pages, rows))
    n = hsp.launch_count()
    assert not hsp.cache_resize(*a, second, new, page, [pool], workspace=ws).any()
    assert hsp.launch_count() == n + 2
    hsp.check_device_error()
    untouched(buf)
    assert all(torch.equal(x, y) for x, y in zip((*a, pool), want))


@pytest.mark.parametrize("pages", [2, 3, 128, 4096, 5001])
def test_compact(hsp, pages):  # noqa: F811
    """The upper half of the pages is live: as many moves as there can be."""
    page, live = 16, pages // 2
    a, pool = cache(1, pages, pages, page)
    a[0][0, :live] = torch.arange(pages - live, pages, device="cuda")
    a[1][0] = live * page
    a[2][pages - live:] = 1
    kept = pool[0, pages - live:].clone()
    buf, ws = guarded(hsp.cache_workspace_bytes(a[0], pages, 0))
    assert hsp.cache_compact(*a, page, [pool], workspace=ws).tolist() == [live]
    hsp.check_device_error()
    untouched(buf)
    assert a[0][0, :live].tolist() == list(range(live)) and torch.equal(pool[0, :live], kept)
