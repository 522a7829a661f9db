"""Calls of the paged cache that meet what a step cannot look at before: a growth that failed, arrays that are the
same tensor."""
import numpy as np
import pytest
import torch

from test_cache_gpu import BF, Cache, hsp  # noqa: F401  (hsp: the module's fixture)

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def expect_bad_index(hsp):  # noqa: F811
    import hidden_state_projection_gb300 as m
    with pytest.raises(m.ProjError) as ei:
        hsp.check_device_error()
    assert ei.value.status_name == "PROJ_ERR_BAD_INDEX"


@pytest.mark.parametrize("captured", [False, True])
def test_append_after_a_growth_that_failed(hsp, captured):  # noqa: F811
    """Row 1, forked from row 0 and cut back, grows again on the page that both hold, and no page is free for its copy;
    row 2 wants a new page; row 3 grows inside its own.  The step appends to all of them at the new lengths."""
    page, dk = 16, 64
    k = torch.randn(1, 5, page, 1, dk, device="cuda").to(BF)
    v = torch.randn(1, 5, page, 1, dk, device="cuda").to(BF)
    table = torch.full((4, 3), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    a, pools = (table, lens, refs), [k, v]
    assert hsp.cache_resize(*a, ints([0, 2, 3]), ints([30, 32, 5]), page, pools).tolist() == [0, 0, 0]
    assert hsp.cache_fork(*a, ints([0]), ints([1]), page).tolist() == [0]
    assert hsp.cache_resize(*a, ints([1]), ints([20]), page, pools).tolist() == [0]
    rows, status = ints([1, 2, 3]), torch.full((3,), 9, dtype=torch.int32, device="cuda")
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    kn = torch.randn(3, dk, device="cuda").to(BF)

    def step():
        torch.add(lens[rows.long()], 1, out=new)
        hsp.cache_resize(*a, rows, new, page, pools, status=status)
        hsp.cache_append(kn, kn, k[0], v[0], table, lens, rows=rows, positions=new - 1)

    before = [t.clone() for t in pools]
    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        saved = [t.clone() for t in (*a, *pools)]
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        expect_bad_index(hsp)
        for t, o in zip((*a, *pools), saved):
            t.copy_(o)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        g.replay()
    else:
        step()
    expect_bad_index(hsp)
    assert status.tolist() == [1, 1, 0] and lens.tolist() == [30, 20, 32, 6]
    for t, b in zip(pools, before):
        b[0, table[3, 0].long(), 5, 0] = kn[2]              # row 3's token, and no other
        assert torch.equal(t, b)


def test_append_at_and_behind_the_end(hsp):  # noqa: F811
    page = 16
    k = torch.zeros(3, page, 1, 576, dtype=BF, device="cuda")
    table = torch.tensor([[2, 0], [1, -1]], dtype=torch.int32, device="cuda")
    kn = torch.ones(2, 576, dtype=BF, device="cuda")
    hsp.cache_append(kn, None, k, None, table, ints([17, 3]), rows=ints([0, 1]), positions=ints([16, 2]))
    hsp.check_device_error()
    assert (k != 0).any(-1).nonzero().tolist() == [[0, 0, 0], [1, 2, 0]]
    k.zero_()
    hsp.cache_append(kn, None, k, None, table, ints([16, 3]), rows=ints([0, 1]), positions=ints([16, 3]))
    expect_bad_index(hsp)
    assert not k.any()


@pytest.mark.parametrize("rows,pages", [(200, 900), (3000, 9000)])
def test_new_lengths_that_lie_in_the_lengths(hsp, rows, pages):  # noqa: F811
    """rows[i] gets the length that row i had: every length is read before any is changed, in one launch and in two."""
    c = Cache(hsp, rows, 4, pages, 16, rows)
    rng = np.random.RandomState(rows)
    c.resize(range(rows), rng.randint(0, 65, rows))
    for step in range(8):
        who = rng.permutation(rows)
        n = rows if step % 2 else rows - 1
        st = hsp.cache_resize(c.table, c.lens, c.refs, c.t(who[:n]), c.lens[:n], 16, c.pools)
        assert st.tolist() == c.model.resize(list(who[:n]), list(c.model.lens[:n]))
        c.check()
    hsp.check_device_error()
