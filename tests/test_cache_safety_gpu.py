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


@pytest.mark.parametrize("with_positions", [False, True])
def test_append_to_a_page_that_others_hold(hsp, with_positions):  # noqa: F811
    """Row 1 is a fork of row 0 whose growth found no free page; rows 2 and 3 have pages of their own.  With the holder
    counts the shared page stays as it is, also where the call writes each row's last token."""
    page = 16
    k = torch.randn(1, 4, page, 2, 64, device="cuda").to(BF)
    v = torch.randn_like(k)
    table = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    a, pools = (table, lens, refs), [k, v]
    assert not hsp.cache_resize(*a, ints([0, 2, 3]), ints([30, 10, 7]), page, pools).any()
    assert not hsp.cache_fork(*a, ints([0]), ints([1]), page).any()
    assert hsp.cache_resize(*a, ints([1, 2, 3]), ints([31, 11, 7]), page, pools).tolist() == [1, 0, 0]
    rows, kn = ints([1, 2, 3]), torch.randn(3, 2, 64, device="cuda").to(BF)
    pos = lens[rows.long()] - 1 if with_positions else None
    args = dict(rows=rows, positions=pos)
    before, old = [t.clone() for t in pools], lens.clone()
    if pos is None:
        lens_of = torch.zeros(3, dtype=torch.int32, device="cuda")      # (without rows and positions: rows 0 .. 2 of a table)
        lens_of.copy_(lens[1:])
        hsp.cache_append(kn, kn, k[0], v[0], table[1:], lens_of, ref_counts=refs)
    else:
        hsp.cache_append(kn, kn, k[0], v[0], table, lens, ref_counts=refs, **args)
    expect_bad_index(hsp)
    assert torch.equal(lens, old)
    for t, b in zip(pools, before):
        b[0, table[2, 0].long(), 10] = kn[1]
        b[0, table[3, 0].long(), 6] = kn[2]
        assert torch.equal(t, b)
    # rows of their own alone: nothing to report
    hsp.cache_append(kn[1:], kn[1:], k[0], v[0], table, lens, rows=rows[1:], ref_counts=refs)
    hsp.check_device_error()
