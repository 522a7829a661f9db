"""The pages of a cache: append with the rotary turn, resize, fork, compact, copy, and a decode run of them
together with the projection and the attention.

Page calls move and count, so they are checked exactly, against a plain model in Python that follows the
documented rules one row after the other.  The rotary turn: two fp32 products and a sum, 3 * 2^-24 of
|a cos| + |b sin|, then one rounding to bf16, at most 2^-8 of the result.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def hsp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import hidden_state_projection_gb300 as m
    m.lib()
    m.set_options(pdl=True, wait_limit_us=0, skip_stage=None)
    return m


# ---- the rules, one row after the other ------------------------------------------------------------

class Model:
    def __init__(self, rows, width, pages, page, pools):
        self.table = np.full((rows, width), -1, np.int64)
        self.lens = np.zeros(rows, np.int64)
        self.refs = np.zeros(pages, np.int64)
        self.page = page
        self.pools = [p.copy() for p in pools]

    def resize(self, rows, new):
        R, W = self.table.shape
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        shared = self.refs.copy()
        status, seen, wanted = [], set(), 0
        copies = []
        for r, n in zip(rows, new):
            if not 0 <= r < R or r in seen or not 0 <= n <= W * self.page:
                status.append(2)
                if 0 <= r < R:
                    seen.add(r)
                continue
            seen.add(r)
            old = self.lens[r]
            have, want = -(-old // self.page), -(-n // self.page)
            cow = n > old and old % self.page != 0 and shared[self.table[r, have - 1]] > 1
            need = max(0, want - have) + cow
            first, wanted = wanted, wanted + need
            if need and wanted > len(free):
                status.append(1)
                continue
            status.append(0)
            take = free[first:first + need]
            if cow:
                src, dst = self.table[r, have - 1], take.pop(0)
                copies.append((src, dst))
                self.refs[src] -= 1
                self.refs[dst] = 1
                self.table[r, have - 1] = dst
            for j in range(have, want):
                self.table[r, j] = take[j - have]
                self.refs[take[j - have]] = 1
            for j in range(want, have):
                self.refs[self.table[r, j]] -= 1
                self.table[r, j] = -1
            self.lens[r] = n
        for src, dst in copies:
            for p in self.pools:
                p[:, dst] = p[:, src]
        return status

    def fork(self, parents, children):
        R, status = self.table.shape[0], []
        for i, (p, c) in enumerate(zip(parents, children)):
            if not (0 <= p < R and 0 <= c < R) or c in children[:i] or p in children or self.lens[c] != 0:
                status.append(2)
                continue
            n = -(-self.lens[p] // self.page)
            self.table[c, :n] = self.table[p, :n]
            for id in self.table[p, :n]:
                self.refs[id] += 1
            self.lens[c] = self.lens[p]
            status.append(0)
        return status

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] == 0]
        tails = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        for h, t in zip(holes, tails):
            for p in self.pools:
                p[:, h] = p[:, t]
            self.refs[h], self.refs[t] = self.refs[t], 0
            for r in range(len(self.lens)):
                n = -(-self.lens[r] // self.page)
                self.table[r, :n][self.table[r, :n] == t] = h
        return live


class Cache:
    """The same cache on the GPU and in the model."""

    def __init__(self, hsp, rows, width, pages, page, seed, layers=(2, 1), cols=(24, 8)):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hsp, self.page = hsp, page
        self.pools = [torch.randint(-30000, 30000, (l, pages, page, c), generator=g, device="cuda").to(torch.int16)
                      for l, c in zip(layers, cols)]
        wide = torch.full((rows, width + 3), -77, dtype=torch.int32, device="cuda")     # rows further apart than they are long
        wide[:, :width] = -1
        self.wide, self.table = wide, wide[:, :width]
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.model = Model(rows, width, pages, page, [p.cpu().numpy() for p in self.pools])

    def t(self, v):
        return torch.tensor(list(v), dtype=torch.int32, device="cuda")

    def resize(self, rows, new, **kw):
        st = self.hsp.cache_resize(self.table, self.lens, self.refs, self.t(rows), self.t(new), self.page, self.pools, **kw)
        assert st.tolist() == self.model.resize(list(rows), list(new))

    def fork(self, parents, children):
        st = self.hsp.cache_fork(self.table, self.lens, self.refs, self.t(parents), self.t(children), self.page)
        assert st.tolist() == self.model.fork(list(parents), list(children))

    def compact(self):
        live = self.hsp.cache_compact(self.table, self.lens, self.refs, self.page, self.pools)
        assert live.tolist() == [self.model.compact()]

    def check(self):
        m = self.model
        assert np.array_equal(self.table.cpu().numpy(), m.table)
        assert np.array_equal(self.lens.cpu().numpy(), m.lens)
        assert np.array_equal(self.refs.cpu().numpy(), m.refs)
        for p, q in zip(self.pools, m.pools):
            assert np.array_equal(p.cpu().numpy(), q)
        assert (self.wide[:, self.table.shape[1]:] == -77).all()


def test_resize_grows_cuts_and_frees(hsp):
    c = Cache(hsp, 5, 6, 20, 16, 1)
    c.resize([2], [1])
    c.resize([0, 1, 4], [16, 17, 96])
    c.check()
    c.resize([1, 0, 4, 2], [0, 40, 33, 16])
    c.resize([3, 4], [96, 34])
    c.resize([0], [40])                                       # as it is
    c.check()
    hsp.check_device_error()


def test_resize_refusals_and_a_full_cache(hsp):
    import hidden_state_projection_gb300 as m
    c = Cache(hsp, 6, 4, 7, 16, 2)
    c.resize([0, 1, 2], [64, 40, 16])                          # seven pages wanted and more: the last row must wait
    c.check()
    c.resize([3, 0, 4], [16, 1, 32])                           # nothing is free yet, the row that shrinks still does
    c.check()
    c.resize([4, 3, 5, 5, 4], [32, 48, 1, 16, 64])             # rows named twice count once; first come, first served
    c.resize([0, 1], [-1, 65])
    c.check()
    hsp.check_device_error()
    for rows in ([-1, 0], [0, 6], [2 ** 31 - 1]):
        c.resize(rows, [0] * len(rows))
        with pytest.raises(m.ProjError) as ei:
            hsp.check_device_error()
        assert ei.value.status_name == "PROJ_ERR_BAD_INDEX"
    c.check()


def test_shared_last_page_is_copied_when_a_holder_grows(hsp):
    c = Cache(hsp, 8, 5, 30, 16, 3)
    c.resize([0, 1], [39, 32])
    c.fork([0, 0, 1, 0], [2, 3, 4, 5])
    c.check()
    c.resize([2, 4, 3], [40, 33, 70])                          # row 4 ends on a page border: nothing to copy
    c.check()
    c.resize([0, 5], [40, 41])                                 # both holders of the last shared page: it becomes free
    c.check()
    c.resize([1], [20])                                        # into a page that row 4 holds too
    c.resize([1], [21])
    c.check()
    c.resize([0, 1, 2, 3, 4, 5], [0] * 6)
    c.check()
    assert int(c.refs.sum()) == 0


def test_fork_refusals(hsp):
    import hidden_state_projection_gb300 as m
    c = Cache(hsp, 8, 4, 30, 16, 4)
    c.resize([0, 1], [50, 7])
    c.fork([0, 1, 0, 2, 3, 6], [2, 2, 1, 3, 3, 6])             # twice a child, a full child, a parent that is a child, its own
    c.check()
    c.fork([7], [6])                                           # an empty parent
    c.check()
    hsp.check_device_error()
    c.fork([0, -1, 0, 8], [4, 5, 9, 5])
    c.check()
    with pytest.raises(m.ProjError):
        hsp.check_device_error()


@pytest.mark.parametrize("rows,width,pages,page,seed", [(1, 1, 1, 16, 5), (7, 9, 61, 16, 6), (40, 30, 1300, 32, 7),
                                                        (1500, 3, 4200, 16, 8)])
def test_random_runs_of_all_of_them(hsp, rows, width, pages, page, seed):
    c = Cache(hsp, rows, width, pages, page, seed)
    rng = np.random.RandomState(seed)
    for step in range(12):
        n = rng.randint(1, rows + 1)
        who = rng.permutation(rows)[:n]
        most = width * page
        c.resize(who, np.where(rng.rand(n) < 0.25, 0, rng.randint(0, most + 1, n)))
        empty = np.flatnonzero(c.model.lens == 0)
        full = np.flatnonzero(c.model.lens > 0)
        if len(empty) and len(full):
            k = rng.randint(1, len(empty) + 1)
            c.fork(rng.choice(full, k), rng.permutation(empty)[:k])
        if step % 4 == 2:
            c.compact()
        grow = np.flatnonzero(c.model.lens > 0)
        if len(grow):
            c.resize(grow, np.minimum(c.model.lens[grow] + rng.randint(1, 5, len(grow)), most))
        c.check()
    hsp.check_device_error()


@pytest.mark.parametrize("n", [255, 256, 257])
@pytest.mark.parametrize("pages", [4095, 4096, 4097])
def test_one_launch_or_two(hsp, pages, n):
    """Requests and pools on both sides of the sizes that one launch serves: the same rules, rows named twice and
    rows outside the table among them, a pool that runs out."""
    import hidden_state_projection_gb300 as m
    c = Cache(hsp, 400, 30, pages, 16, pages + n)
    rng = np.random.RandomState(n)
    small = n <= 256 and pages <= 4096
    for step in range(6):
        who = rng.randint(-1, 401, n)
        before = hsp.launch_count()
        c.resize(who, np.where(rng.rand(n) < 0.2, 0, rng.randint(-1, 30 * 16 + 2, n)))
        assert hsp.launch_count() - before == (1 if small else 2)
        c.check()
        empty, full = np.flatnonzero(c.model.lens == 0), np.flatnonzero(c.model.lens > 0)
        c.fork(rng.choice(full, len(empty) // 2), empty[:len(empty) // 2])
        held = rng.permutation(np.flatnonzero(c.model.lens > 0))[:n]
        c.resize(held, np.minimum(c.model.lens[held] + 1, 480))
        c.check()
        if step % 2:
            c.compact()
            c.check()
    with pytest.raises(m.ProjError) as ei:
        hsp.check_device_error()
    assert ei.value.status_name == "PROJ_ERR_BAD_INDEX"


def test_one_launch_moves_as_much_as_two(hsp):
    """Pages of 196,608 bytes over two pools: five copies at most in one launch."""
    for n in (1, 4, 5, 6, 40):
        c = Cache(hsp, 80, 6, 100, 16, n, cols=(2048, 2048))
        c.resize(range(0, 2 * n, 2), [17 + i for i in range(n)])
        c.fork(range(0, 2 * n, 2), range(1, 2 * n, 2))
        before = hsp.launch_count()
        c.resize(range(1, 2 * n, 2), [18 + i for i in range(n)])
        assert hsp.launch_count() - before == (1 if n <= 5 else 2)
        c.check()
    hsp.check_device_error()


def test_compact_an_empty_a_full_and_a_sparse_cache(hsp):
    for pages in (1, 127, 128, 129, 5000):
        c = Cache(hsp, 70, 40, pages, 16, pages, layers=(1,), cols=(8,))
        c.compact()
        c.check()
        c.resize(range(70), [16 * (1 + 37 * i % 40) for i in range(70)])
        c.compact()
        c.check()
        c.resize(range(0, 70, 3), [0] * 24)
        c.resize(range(1, 70, 3), [16] * 23)
        c.compact()
        c.compact()
        c.check()
    hsp.check_device_error()


def test_pages_of_an_unusual_size(hsp):
    """Pages that are not a whole number of 16 KB pieces, and pools that are parts of wider tensors."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for cols in (8, 1032, 1024, 520):
        wide = torch.randint(-9, 9, (3, 20, 3, 16, cols), generator=g, device="cuda").to(torch.int16)
        pool = wide[1:, :, 1]
        before = wide.clone()
        hsp.cache_copy_pages([pool], [0, 5, 0], [7, 19, 3])
        torch.cuda.synchronize()
        want = before.clone()
        want[1:, [7, 19, 3], 1] = before[1:, [0, 5, 0], 1]
        assert torch.equal(wide, want)


@pytest.mark.parametrize("n", [1, 64, 65, 2048])
def test_copy_pages(hsp, n):
    pool = torch.randint(-9, 9, (2, 4100, 16, 8), device="cuda").to(torch.int16)
    other = torch.randn(1, 4100, 16, 4, device="cuda")
    ids = torch.randperm(4100)[:2 * n].to(torch.int32)
    src, dst = ids[:n].contiguous(), ids[n:].contiguous()
    want = [pool.clone(), other.clone()]
    for w in want:
        w[:, dst.long().cuda()] = w[:, src.long().cuda()]
    hsp.cache_copy_pages([pool, other], src, dst)
    assert torch.equal(pool, want[0]) and torch.equal(other, want[1])
    hsp.cache_copy_pages([pool], [], [])


def test_pages_past_four_gigabytes(hsp):
    pages, page = 36000, 64
    pool = torch.empty(1, pages, page, 1024, dtype=BF, device="cuda")        # 4.7 GB, 2^31 elements and more
    pool[0, [3, pages - 1]] = torch.randn(2, page, 1024, device="cuda").to(BF)
    hsp.cache_copy_pages([pool], [3, pages - 1], [pages - 7, 5])
    assert torch.equal(pool[0, pages - 7], pool[0, 3]) and torch.equal(pool[0, 5], pool[0, pages - 1])
    table = torch.tensor([[pages - 1, pages - 7, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[pages - 1] = refs[pages - 7] = 1
    kept = pool[0, [pages - 1, pages - 7]].clone()
    assert hsp.cache_compact(table, lens, refs, page, [pool]).tolist() == [2]
    assert sorted(table[0, :2].tolist()) == [0, 1] and torch.equal(pool[0, table[0, :2].long()], kept)
    assert refs.nonzero().flatten().tolist() == [0, 1]
    hsp.check_device_error()


def test_page_calls_captured_and_replayed(hsp):
    """A beam step captured once: free the children, fork, grow; replayed with other parents."""
    c = Cache(hsp, 10, 8, 60, 16, 9)
    c.resize([0, 1], [50, 33])
    parents, children = c.t([0, 0, 1]), c.t([4, 7, 2])
    zero, new = c.t([0, 0, 0]), c.t([0, 0, 0])
    a = (c.table, c.lens, c.refs)

    def step():
        hsp.cache_resize(*a, children, zero, 16, c.pools)
        hsp.cache_fork(*a, parents, children, 16)
        torch.add(c.lens[parents.long()], 1, out=new)
        hsp.cache_resize(*a, children, new, 16, c.pools)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    saved = [t.clone() for t in (*a, *c.pools)]
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    for t, o in zip((*a, *c.pools), saved):
        t.copy_(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for p in ([0, 0, 1], [1, 1, 1], [0, 1, 0]):
        parents.copy_(c.t(p))
        g.replay()
        c.model.resize([4, 7, 2], [0, 0, 0])
        c.model.fork(p, [4, 7, 2])
        c.model.resize([4, 7, 2], [int(c.model.lens[x]) + 1 for x in p])
        torch.cuda.synchronize()
        c.check()
    hsp.check_device_error()


# ---- append -----------------------------------------------------------------------------------------

def turned(x, cs, rot, inter):
    """(value, bound) of the last `rot` columns of x [n, heads, d] turned, in 64 bits."""
    y = x.double().clone()
    t = torch.zeros_like(y)
    if rot == 0:
        return y, t
    d = x.shape[-1]
    c, s = cs[:, None, :rot // 2].double(), cs[:, None, rot // 2:].double()
    i = torch.arange(rot // 2, device=x.device)
    one, two = (d - rot + 2 * i, d - rot + 2 * i + 1) if inter else (d - rot + i, d - rot // 2 + i)
    a, b = x.double()[..., one], x.double()[..., two]
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    eps = 3 * 2.0 ** -24
    t[..., one] = eps * ((a * c).abs() + (b * s).abs()) + y[..., one].abs() * 2.0 ** -8
    t[..., two] = eps * ((b * c).abs() + (a * s).abs()) + y[..., two].abs() * 2.0 ** -8
    return y, t


APPEND = [(1, 16, 1, 576, 512, True, 64, 64, True), (8, 128, 1, 576, 512, True, 64, 64, False), (5, 0, 1, 512, 512, True, 16, 0, True),
          (3, 7, 1, 512, 512, True, 128, 48, True), (13, 32, 8, 128, 128, False, 16, 128, False), (300, 3, 1, 64, 64, False, 32, 32, True),
          (64, 20, 5, 64, 64, False, 1024, 16, False), (1, 1, 1, 64, 64, False, 16, 64, True), (700, 0, 2, 128, 128, False, 64, 128, False)]


@pytest.mark.parametrize("n,heads,kv,dk,dv,latent,page,rot,inter", APPEND)
def test_append(hsp, n, heads, kv, dk, dv, latent, page, rot, inter):
    g = torch.Generator(device="cuda").manual_seed(n + dk)
    width = -(-900 // page) + 1
    seqs = min(n, 9)
    pages = seqs * width + 2
    table = torch.randperm(pages, generator=g, device="cuda")[:seqs * width].view(seqs, width).to(torch.int32)
    which = torch.randperm(seqs * 900, generator=g, device="cuda")[:n]         # row and position, all different
    rows, pos = (which // 900).to(torch.int32), (which % 900).to(torch.int32)
    k = torch.randn(pages, page, kv, dk, generator=g, device="cuda").to(BF)
    v = None if latent else torch.randn(pages, page, kv, dv, generator=g, device="cuda").to(BF)
    kn = torch.randn(n, kv * dk + 8, generator=g, device="cuda").to(BF)[:, :kv * dk]   # columns of a wider projection
    vn = None if latent else torch.randn(n, kv, dv, generator=g, device="cuda").to(BF)
    q = torch.randn(n, heads, dk, generator=g, device="cuda").to(BF) if heads else None
    ang = torch.rand(1000, max(rot // 2, 1), generator=g, device="cuda") * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).contiguous() if rot else None
    k0, v0 = k.clone(), None if latent else v.clone()
    lens = torch.full((seqs,), 900, dtype=torch.int32, device="cuda")
    got = hsp.cache_append(kn, vn, k, v, table, lens, rows=rows, positions=pos, cos_sin=cs, interleaved=inter, q=q)
    hsp.check_device_error()
    at, off = table[rows.long(), (pos // page).long()].long(), (pos % page).long()
    csr = cs[pos.long()] if rot else None
    y, t = turned(kn.reshape(n, kv, dk), csr, rot, inter)
    assert ((k[at, off].double() - y).abs() <= t).all()
    k0[at, off] = k[at, off]
    assert torch.equal(k, k0)                                                  # and nothing else
    if not latent:
        v0[at, off] = vn
        assert torch.equal(v, v0)
    if heads:
        y, t = turned(q, csr, rot, inter)
        assert ((got.double() - y).abs() <= t).all()
        same = q.clone()
        assert hsp.cache_append(kn, vn, k, v, table, lens, rows=rows, positions=pos, cos_sin=cs, interleaved=inter, q=same,
                                q_out=same) is same
        assert torch.equal(same, got)


def test_append_at_the_last_place_and_far_positions(hsp):
    page, far = 16, 65535
    table = torch.zeros(3, 4096, dtype=torch.int32, device="cuda")
    table[0, 4095], table[1, 0], table[2, 1] = 2, 1, 3
    lens = torch.tensor([far + 1, 1, 18], dtype=torch.int32, device="cuda")
    k = torch.zeros(4, page, 1, 576, dtype=BF, device="cuda")
    kn = torch.randn(3, 576, device="cuda").to(BF)
    ang = torch.arange(far + 1, dtype=torch.float64, device="cuda")[:, None] * torch.logspace(0, -4, 32, dtype=torch.float64, device="cuda")
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    hsp.cache_append(kn, None, k, None, table, lens, cos_sin=cs)
    hsp.check_device_error()
    y, t = turned(kn.view(3, 1, 576), cs[[far, 0, 17]], 64, True)
    got = torch.stack([k[2, 15], k[1, 0], k[3, 1]])
    assert ((got.double() - y).abs() <= t).all()
    assert int((k != 0).any(-1).sum()) == 3


def test_append_reports_what_lies_outside(hsp):
    import hidden_state_projection_gb300 as m
    page = 16
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 5], dtype=torch.int32, device="cuda")
    kn = torch.ones(2, 64, device="cuda", dtype=BF)
    cs = torch.ones(40, 64, device="cuda")

    def expect(table, **kw):
        k = torch.zeros(4, page, 1, 64, dtype=BF, device="cuda")
        v = torch.zeros_like(k)
        hsp.cache_append(kn, kn, k, v, table, kw.pop("lens", lens), **{x: torch.tensor(y, dtype=torch.int32, device="cuda")
                                                               if x in ("rows", "positions") else y for x, y in kw.items()})
        with pytest.raises(m.ProjError) as ei:
            hsp.check_device_error()
        assert ei.value.status_name == "PROJ_ERR_BAD_INDEX"
        return int((k != 0).any(-1).sum())

    assert expect(table, rows=[0, 2]) == 1
    assert expect(table, rows=[-1, 1]) == 1
    assert expect(table, positions=[-1, 0]) == 1
    assert expect(table, positions=[32, 0]) == 1
    assert expect(table, positions=[0, 31], cos_sin=cs[:31]) == 1
    bad = table.clone()
    bad[0, 0], bad[1, 0] = 4, -2
    assert expect(bad, positions=[0, 1]) == 0
    assert expect(table, lens=torch.tensor([0, 1], dtype=torch.int32, device="cuda")) == 1


# ---- together ---------------------------------------------------------------------------------------

def test_a_decode_run(hsp):
    """Project, grow, append, attend, with a fork on the way, a sequence freed and the cache compacted: after every
    step each sequence's attention equals that over its own history kept densely."""
    from test_attention_gpu import reference
    g = torch.Generator(device="cuda").manual_seed(77)
    K, heads, page, rows, pages = 512, 16, 16, 4, 14
    w = (torch.randn(heads * 576 + 576, K, generator=g, device="cuda") * 0.04).to(BF)
    k = torch.full((2, pages, page, 1, 576), float("nan"), dtype=BF, device="cuda")   # two layers, the second is used
    table = torch.full((rows, 6), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    ang = torch.arange(96, device="cuda")[:, None] * torch.logspace(0, -3, 32, device="cuda")[None]
    cs = torch.cat([ang.cos(), ang.sin()], 1).contiguous()
    history = {}
    active = [0, 2]
    for step in range(40):
        if step == 21:                                       # row 2 becomes the parent of 1 and 3, on a partly filled page
            st = hsp.cache_fork(table, lens, refs, *(torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([2, 2], [1, 3])), page)
            assert st.tolist() == [0, 0]
            history[1], history[3] = list(history[2]), list(history[2])
            active = [0, 1, 2, 3]
        if step == 30:                                       # row 0 ends, its pages go, the others move together
            st = hsp.cache_resize(table, lens, refs, *(torch.tensor([t], dtype=torch.int32, device="cuda") for t in (0, 0)), page, [k])
            assert st.tolist() == [0]
            live = hsp.cache_compact(table, lens, refs, page, [k])
            assert int(live) == int((refs > 0).sum()) and (refs[:int(live)] > 0).all()
            active = [3, 1, 2]
        r = torch.tensor(active, dtype=torch.int32, device="cuda")
        x = torch.randn(len(active), K, generator=g, device="cuda").to(BF)
        q, kv = hsp.fused_gemm(x, w, [heads * 576, 576])
        new = lens[r.long()] + 1
        assert not hsp.cache_resize(table, lens, refs, r, new, page, [k]).any()
        q = hsp.cache_append(kv, None, k[1], None, table, lens, rows=r, positions=new - 1, cos_sin=cs,
                             q=q.view(len(active), heads, 576))
        out, lse = hsp.paged_attention(q, k[1], None, table, lens, 0.07, rows=r, return_lse=True)
        hsp.check_device_error()
        for i, row in enumerate(active):
            # the row as it was just written (its values are test_append's), kept apart from the cache
            p = int(lens[row]) - 1
            written = k[1][table[row, p // page].long(), p % page, 0].clone()
            y, t = turned(kv[i].view(1, 1, 576), cs[p:p + 1], 64, True)
            assert ((written.double() - y.view(576)).abs() <= t.view(576)).all()
            history.setdefault(row, []).append(written)
            n = len(history[row])
            assert n == p + 1
            dense = torch.stack(history[row]).view(1, n, 1, 576)
            ref, rl, tol, ltol = reference(q[i:i + 1], dense, None, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                                           torch.tensor([n]), 0.07, 512)
            assert ((out[i].double() - ref[0]).abs() <= tol[0]).all()
            assert ((lse[i].double() - rl[0]).abs() <= ltol[0]).all()
    assert lens.tolist() == [0, 40, 40, 40]
