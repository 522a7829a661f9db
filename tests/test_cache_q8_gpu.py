"""The paged cache in 8 bits: what cache_append_q8 writes and cache_read_q8 gives back, code by code.

Codes and scales are those of the definition in 64 bits, without tolerance: a scale is a power of two, the products
of the rotary turn (bf16 times fp32: 32 bits) and their sums are exact or rounded far behind the codes' last bit in 64
bits, and the kernel rounds the exact sum once.  Turned queries: two fp32 products and a sum, 3 * 2^-24 of
|a cos| + |b sin|, then one rounding to bf16, at most 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
GRID = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])[:127]


@pytest.fixture(scope="module")
def hsp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import hidden_state_projection_gb300 as m
    m.lib()
    m.set_options(pdl=True, wait_limit_us=0, skip_stage=None)
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def numbers(t):
    return t.float().cpu().numpy().astype(np.float64)


def nearest(x):
    """Nearest e4m3 value, ties to the even code; what is not within 448 is NaN."""
    y = np.abs(x)
    with np.errstate(invalid="ignore"):
        hi = np.searchsorted(GRID, y).clip(1, 126)
        low, up = y - GRID[hi - 1], GRID[hi] - y
        i = np.where((low < up) | ((low == up) & (hi % 2 == 1)), hi - 1, hi)
        return np.where(y <= 448, np.copysign(GRID[i], x), np.nan)


class Cache8:
    """A cache on the GPU: block table, lengths, codes and scales, with something in every place."""

    def __init__(self, rows, width, page, block, kv, dk, dv, seed, spare=3, order="token", packed=False):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        pages = rows * width + spare
        self.page, self.block = page, block
        self.table = torch.randperm(pages, generator=g, device="cuda")[: rows * width].to(torch.int32).view(rows, width).contiguous()
        self.lens = ints([0] * rows)
        nb = page // block

        def side(dim):
            if dim is None:
                return None, None
            if packed:  # codes and scales of a page side by side in a pool of bytes
                size = page * kv * dim
                pool = torch.randint(0, 127, (pages, size + -(-nb * kv * 4 // 16) * 16), generator=g, device="cuda").to(torch.uint8)
                codes = pool[:, :size].view(pages, page, kv, dim).view(F8)
                scales = pool[:, size:].view(torch.float32)[:, : nb * kv].view(pages, nb, kv)
            elif order == "head":
                codes = torch.randint(0, 127, (pages, kv, page, dim), generator=g, device="cuda").to(torch.uint8).view(F8).transpose(1, 2)
                scales = torch.empty(pages, kv, nb, device="cuda").transpose(1, 2)
            else:
                codes = torch.randint(0, 127, (pages, page, kv, dim), generator=g, device="cuda").to(torch.uint8).view(F8)
                scales = torch.empty(pages, nb, kv, device="cuda")
            scales.copy_(2.0 ** torch.randint(-9, -4, (pages, nb, kv), generator=g, device="cuda").float())
            return codes, scales

        self.k, self.ks = side(dk)
        self.v, self.vs = side(dv)

    def model(self):
        m = {"k": numbers(self.k), "ks": numbers(self.ks)}
        if self.v is not None:
            m |= {"v": numbers(self.v), "vs": numbers(self.vs)}
        return m

    def same(self, m):
        for name in m:
            got = numbers(getattr(self, name))
            bad = ~((got == m[name]) | (np.isnan(got) & np.isnan(m[name])))
            assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size}, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {m[name][bad][0]}"


def turned(x, cs, pos, interleaved, minus=-1.0):
    """The turn; with minus = 1 of absolute values: |a cos| + |b sin| and |b cos| + |a sin|."""
    rot = cs.shape[1]
    y = x.copy()
    c, s = cs[pos][:, None, : rot // 2], cs[pos][:, None, rot // 2:]
    i, a = np.arange(rot // 2), x.shape[-1] - rot
    one, two = (a + 2 * i, a + 2 * i + 1) if interleaved else (a + i, a + rot // 2 + i)
    y[..., one] = x[..., one] * c + minus * x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def write(codes, scales, x, at, line, block):
    """The documented rule, one block and head after the other.  at[i] < 0: token i is written nowhere."""
    groups = {}
    for i in range(len(x)):
        if at[i] >= 0:
            groups.setdefault((int(at[i]), int(line[i]) // block), []).append(i)
    for (p, b), tokens in groups.items():
        first = min(int(line[i]) for i in tokens)
        for h in range(x.shape[1]):
            y = np.abs(x[tokens, h])
            y = y[y <= 448 * 2.0 ** 60]
            e = -60
            while e < 60 and y.size and y.max() > 448 * 2.0 ** e:
                e += 1
            s, old = 2.0 ** e, scales[p, b, h]
            if first > b * block and old >= s:
                s = old
            elif first > b * block:
                codes[p, b * block:first, h] = nearest(codes[p, b * block:first, h] * (old / s))
            for i in tokens:
                codes[p, line[i], h] = nearest(x[i, h] / s)
            scales[p, b, h] = s


def angles(n, rot, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.rand(n, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 7
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def new_rows(g, n, kv, dim, spread=1.5):
    size = torch.exp(torch.randn(n, 1, 1, generator=g, device="cuda") * spread)
    return (torch.randn(n, kv, dim, generator=g, device="cuda") * size).to(BF)


def append(hsp, c, rows, pos, dk, kv, dv, rot=0, interleaved=True, heads=0, kn=None, vn=None, bad=(), **kw):
    """One call and the model's; tokens named in `bad` are expected to be written nowhere, and reported."""
    n = len(rows)
    kn = new_rows(c.g, n, kv, dk) if kn is None else kn
    vn = (new_rows(c.g, n, kv, dv) if vn is None else vn) if dv else None
    cs = angles(max(64, int(c.table.shape[1]) * c.page), rot) if rot else None
    q = torch.randn(n, heads, dk, generator=c.g, device="cuda").to(BF) if heads else None
    m = c.model()
    out = hsp.cache_append_q8(kn, vn, c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=ints(rows), positions=ints(pos), cos_sin=cs,
                              interleaved=interleaved, q=q, **kw)
    if bad:
        with pytest.raises(hsp.ProjError) as e:
            hsp.check_device_error()
        assert e.value.status_name == "PROJ_ERR_BAD_INDEX"
    else:
        hsp.check_device_error()
    table = c.table.cpu().numpy()
    at = np.array([-1 if i in bad else table[rows[i], pos[i] // c.page] for i in range(n)])
    line = np.array(pos) % c.page
    x = numbers(kn)
    cs64 = cs.cpu().numpy().astype(np.float64) if rot else None
    write(m["k"], m["ks"], turned(x, cs64, np.maximum(pos, 0), interleaved) if rot else x, at, line, c.block)
    if dv:
        write(m["v"], m["vs"], numbers(vn), at, line, c.block)
    c.same(m)
    if heads:
        x = numbers(q)
        want = turned(x, cs64, pos, interleaved)
        size = turned(np.abs(x), np.abs(cs64), pos, interleaved, 1.0)
        off = np.abs(numbers(out) - want) - (3 * 2.0 ** -24 * size + 2.0 ** -8 * np.abs(want))
        assert off.max() <= 0, f"queries off by {off.max()} more than they may be"
    return m


KINDS = [(576, 1, None, 64), (512, 1, None, 0), (128, 3, 128, 128), (64, 5, 64, 32), (80, 2, 48, 16)]


@pytest.mark.parametrize("dk,kv,dv,rot", KINDS)
@pytest.mark.parametrize("page,block", [(16, 1), (16, 16), (64, 4), (64, 32), (64, 64), (128, 128)])
def test_append(hsp, dk, kv, dv, rot, page, block):
    """Chunks that begin and end inside blocks and pages, then single tokens behind them, whose blocks grow."""
    c = Cache8(4, 4, page, block, kv, dk, dv, 5 + page + block + dk)
    start, n = [0, 3, page + 1, 2 * page - 1], [2 * page + 5, 1, page - 1, page + 2]
    rows = [r for r in range(4) for _ in range(n[r])]
    pos = [start[r] + i for r in range(4) for i in range(n[r])]
    c.lens.copy_(ints([s + k for s, k in zip(start, n)]))
    append(hsp, c, rows, pos, dk, kv, dv, rot, True, heads=3 if rot else 0)
    for step in range(3):
        last = c.lens.tolist()
        c.lens += 1
        append(hsp, c, [2, 0, 3, 1], [last[r] for r in (2, 0, 3, 1)], dk, kv, dv, rot, False, heads=3 if rot else 0,
               kn=new_rows(c.g, 4, kv, dk, spread=4.0))


@pytest.mark.parametrize("page,block,dk,kv", [(16, 16, 128, 8), (64, 64, 576, 1), (64, 1, 64, 2), (1024, 1024, 64, 1)])
def test_append_many(hsp, page, block, dk, kv):
    """More tokens than the CTAs that fit the GPU: chunks, runs that go on behind them."""
    n = 3001
    c = Cache8(2, -(-n // page) + 1, page, block, kv, dk, dk if kv > 1 else None, 11)
    rows, pos = [1] * 1700 + [0] * (n - 1700), list(range(7, 1707)) + list(range(n - 1700))
    c.lens.copy_(ints([n - 1700, 1707]))
    append(hsp, c, rows, pos, dk, kv, dk if kv > 1 else None, rot=32, heads=2)


@pytest.mark.parametrize("order,packed", [("head", False), ("token", True)])
def test_layouts(hsp, order, packed):
    c = Cache8(2, 3, 32, 8, 4, 64, 64, 9, order=order, packed=packed)
    c.lens.copy_(ints([50, 61]))
    append(hsp, c, [0] * 20 + [1] * 33, list(range(30, 50)) + list(range(28, 61)), 64, 4, 64, rot=64, interleaved=False, heads=4)
    k, v = hsp.cache_read_q8(c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=ints([1] * 61), positions=ints(list(range(61))))
    hsp.check_device_error()
    at, line = c.table[1][torch.arange(61, device="cuda") // 32].long(), torch.arange(61, device="cuda") % 32
    for got, codes, scales in ((k, c.k, c.ks), (v, c.v, c.vs)):
        want = codes.float()[at, line] * scales[at, line // 8][..., None]
        assert torch.equal(got, want.to(BF))


def test_any_order_inside_a_block(hsp):
    """Tokens of a block in any order, some of its places left out, a place named twice with the same rows."""
    c = Cache8(2, 2, 32, 16, 2, 64, 64, 21)
    c.lens.copy_(ints([32, 64]))
    append(hsp, c, [0] * 5 + [1] * 4, [9, 3, 12, 4, 5, 40, 37, 39, 33], 64, 2, 64)
    kn = new_rows(c.g, 1, 2, 64).expand(3, 2, 64).contiguous()
    append(hsp, c, [1, 1, 1], [50, 50, 50], 64, 2, 64, kn=kn, vn=kn)


@pytest.mark.parametrize("block", [1, 16])
def test_values_at_the_ends(hsp, block):
    """NaN, infinities, zeros, the largest and smallest bf16 numbers, ties between codes."""
    c = Cache8(1, 2, 16, block, 1, 64, None, 2)
    c.lens.copy_(ints([16]))
    kn = new_rows(c.g, 16, 1, 64)
    kn[0, 0, :3] = torch.tensor([float("nan"), float("inf"), -float("inf")])
    kn[1] = 0
    kn[2, 0, 0] = 3.38e38
    kn[3] = 1e-38
    kn[4] = -0.0
    kn[5, 0] = torch.arange(64, device="cuda") / 64 + 448 - 32           # ties at 440 among them
    kn[6] = float("nan")
    kn[7] = float("inf")
    kn[8, 0, 5] = 448 * 2.0 ** 60
    kn[9, 0, 5] = 450 * 2.0 ** 60
    kn[10] = 2.0 ** -66
    if block == 16:
        kn[8], kn[9, 0, 5] = 1, -1                                         # (their scale would leave nothing of the others)
    append(hsp, c, [0] * 16, list(range(16)), 64, 1, None, kn=kn)
    append(hsp, c, [0] * 16, list(range(16)), 64, 1, None, kn=torch.full_like(kn, float("nan")))


def test_codes_in_front_follow_a_grown_scale(hsp):
    """A small token, then larger ones: every code in front is rounded to the new scale, and a smaller one changes none."""
    c = Cache8(1, 1, 64, 64, 1, 512, None, 4)
    size = [1e-3, 1e-2, 1.0, 0.5, 300.0, 1e4, 1e-8, 1e12]
    for i, s in enumerate(size):
        c.lens.copy_(ints([i + 1]))
        before = c.model()
        append(hsp, c, [0], [i], 512, 1, None, kn=(torch.randn(1, 1, 512, generator=c.g, device="cuda") * s).to(BF))
        page = int(c.table[0, 0])
        if i and s < max(size[:i]):
            assert np.array_equal(before["k"][page, :i], c.model()["k"][page, :i], equal_nan=True)


def test_what_is_not_written(hsp):
    c = Cache8(3, 2, 16, 8, 2, 64, 64, 6)
    c.lens.copy_(ints([20, 9, 32]))
    # behind the row's end, negative, far out: reported, and the rest is written
    append(hsp, c, [0, 0, 0, 1, 1, 2, 2], [18, 19, 20, 8, 9, 31, 0], 64, 2, 64, bad=(2, 4))
    append(hsp, c, [0, 1, 2], [-1, 8, 1 << 30], 64, 2, 64, bad=(0, 2))
    m = c.model()
    kn = new_rows(c.g, 3, 2, 64)
    hsp.cache_append_q8(kn, kn, c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=ints([-1, 3, 1 << 30]), positions=ints([0, 0, 0]))
    with pytest.raises(hsp.ProjError):
        hsp.check_device_error()
    bad = c.table.clone()
    bad[0, 1], bad[1, 0] = -7, 1 << 29
    hsp.cache_append_q8(kn, kn, c.k, c.v, c.ks, c.vs, bad, c.lens, rows=ints([0, 1, 1]), positions=ints([19, 8, 7]))
    with pytest.raises(hsp.ProjError):
        hsp.check_device_error()
    c.same(m)
    # a page that others hold too
    refs = ints([1] * c.k.shape[0])
    refs[c.table[1, 0].long()] = 2
    append(hsp, c, [0, 1, 2], [19, 8, 31], 64, 2, 64, bad=(1,), ref_counts=refs)
    # angles end before the positions do: neither keys nor values
    m, cs = c.model(), angles(16, 32)
    hsp.cache_append_q8(kn[:2], kn[:2], c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=ints([2, 2]), positions=ints([16, 30]), cos_sin=cs)
    with pytest.raises(hsp.ProjError):
        hsp.check_device_error()
    c.same(m)


def test_last_places_without_positions(hsp):
    c = Cache8(3, 2, 16, 4, 2, 64, 64, 8)
    c.lens.copy_(ints([20, 9, 32]))
    m = c.model()
    kn, vn = new_rows(c.g, 3, 2, 64), new_rows(c.g, 3, 2, 64)
    hsp.cache_append_q8(kn, vn, c.k, c.v, c.ks, c.vs, c.table, c.lens)
    table = c.table.cpu().numpy()
    at, line = np.array([table[0, 1], table[1, 0], table[2, 1]]), np.array([3, 8, 15])
    write(m["k"], m["ks"], numbers(kn), at, line, 4)
    write(m["v"], m["vs"], numbers(vn), at, line, 4)
    c.same(m)
    k, v = hsp.cache_read_q8(c.k, c.v, c.ks, c.vs, c.table, c.lens)
    hsp.check_device_error()
    assert np.array_equal(numbers(k), m["k"][at, line] * m["ks"][at, line // 4][..., None])
    assert np.array_equal(numbers(v), m["v"][at, line] * m["vs"][at, line // 4][..., None])


@pytest.mark.parametrize("dk,kv,dv", [(576, 1, None), (128, 8, 128), (64, 5, 64), (80, 2, 48)])
@pytest.mark.parametrize("n", [1, 5, 700, 6007])
def test_read(hsp, dk, kv, dv, n):
    c = Cache8(3, 40, 64, 16, kv, dk, dv, n)
    c.lens.copy_(ints([2560, 1, 999]))
    g = torch.Generator().manual_seed(n)
    rows = torch.randint(0, 3, (n,), generator=g)
    pos = (torch.rand(n, generator=g) * torch.tensor([2560, 1, 999])[rows]).to(torch.int32)
    rows, pos = rows.to(torch.int32).cuda(), pos.cuda()
    # token rows wider than they are, as where keys and values share an output
    wide = torch.full((n, kv * (dk + (dv or 0)) + 8), 7.0, dtype=BF, device="cuda")
    ko, vo = wide[:, : kv * dk], wide[:, kv * dk: kv * (dk + dv)] if dv else None
    k, v = hsp.cache_read_q8(c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=rows, positions=pos, k_out=ko, v_out=vo)
    hsp.check_device_error()
    assert k is ko and v is vo and bool((wide[:, -8:] == 7).all())
    at, line = c.table[rows.long(), (pos // 64).long()].long(), (pos % 64).long()
    for got, codes, scales in ((k, c.k, c.ks), (v, c.v, c.vs)):
        if codes is not None:
            want = codes.view(torch.uint8)[at, line].view(F8).float() * scales[at, line // 16][..., None]
            assert torch.equal(got.reshape(want.shape), want.to(BF))


def test_read_outside_the_cache_gives_zeros(hsp):
    c = Cache8(2, 2, 16, 16, 1, 64, None, 3)
    c.lens.copy_(ints([5, 32]))
    c.table[1, 1] = 1 << 20
    k, v = hsp.cache_read_q8(c.k, None, c.ks, None, c.table, c.lens, rows=ints([0, 0, 1, 2, -1, 1, 0]), positions=ints([4, 5, 15, 0, 0, 16, -1]))
    with pytest.raises(hsp.ProjError) as e:
        hsp.check_device_error()
    assert e.value.status_name == "PROJ_ERR_BAD_INDEX" and v is None
    assert bool((k[[1, 3, 4, 5, 6]] == 0).all())
    want = (c.k.view(torch.uint8)[c.table[0, 0].long(), 4].view(F8).float() * c.ks[c.table[0, 0].long(), 0][..., None]).to(BF)
    assert torch.equal(k[0], want)


def test_read_rounds_scales_of_any_value(hsp):
    """A scale that the writer would not make: one rounding of the product."""
    c = Cache8(1, 1, 16, 4, 1, 64, None, 3)
    c.lens.copy_(ints([16]))
    c.ks.copy_(torch.rand(c.ks.shape, generator=c.g, device="cuda") * 3 + 0.1)
    k, _ = hsp.cache_read_q8(c.k, None, c.ks, None, c.table, c.lens, rows=ints([0] * 16), positions=ints(list(range(16))))
    p = int(c.table[0, 0])
    want = numbers(c.k)[p] * np.repeat(numbers(c.ks)[p], 4, 0)[..., None]
    # the fp32 product, 2^-24, then bf16, 2^-8 (relative, of a product within 2^-24 of the exact one)
    assert (np.abs(numbers(k) - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want)).all()


def test_streams_and_graphs(hsp):
    """The same call on another stream, and captured: the same codes."""
    c = Cache8(3, 3, 32, 16, 2, 128, 128, 12)
    c.lens.copy_(ints([40, 50, 61]))
    keep = {n: getattr(c, n).clone() for n in ("k", "v", "ks", "vs")}
    rows, pos = ints([0, 1, 2, 2]), ints([39, 49, 59, 60])
    kn, vn, q, cs = new_rows(c.g, 4, 2, 128), new_rows(c.g, 4, 2, 128), new_rows(c.g, 4, 6, 128), angles(96, 128)

    def call(**kw):
        out = hsp.cache_append_q8(kn, vn, c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=rows, positions=pos, cos_sin=cs, q=q, **kw)
        return (out, *hsp.cache_read_q8(c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=rows, positions=pos, **kw))

    def reset():
        for n, t in keep.items():
            getattr(c, n).copy_(t)

    want = [t.clone() for t in call()]
    codes = [c.k.clone(), c.v.clone(), c.ks.clone(), c.vs.clone()]
    reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(2):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for a, b in zip((c.k, c.v, c.ks, c.vs), codes):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    hsp.check_device_error()


def test_queries_in_place(hsp):
    c = Cache8(2, 2, 16, 8, 1, 576, None, 1)
    c.lens.copy_(ints([3, 20]))
    kn, q, cs = new_rows(c.g, 2, 1, 576), new_rows(c.g, 2, 5, 576), angles(32, 64)
    for inter in (True, False):
        a = hsp.cache_append_q8(kn, None, c.k, None, c.ks, None, c.table, c.lens, cos_sin=cs, interleaved=inter, q=q)
        mine = q.clone()
        assert hsp.cache_append_q8(kn, None, c.k, None, c.ks, None, c.table, c.lens, cos_sin=cs, interleaved=inter, q=mine, q_out=mine) is mine
        assert torch.equal(a, mine)
    hsp.check_device_error()


def test_no_tokens(hsp):
    c = Cache8(2, 2, 16, 8, 1, 64, None, 1)
    m = c.model()
    none = torch.empty(0, 1, 64, dtype=BF, device="cuda")
    assert hsp.cache_append_q8(none, None, c.k, None, c.ks, None, c.table, c.lens, rows=ints([]), positions=ints([])) is None
    k, _ = hsp.cache_read_q8(c.k, None, c.ks, None, c.table, c.lens, rows=ints([]), positions=ints([]))
    assert k.shape == (0, 1, 64)
    c.same(m)


def test_a_place_named_twice(hsp):
    """Neighbours in the call: the same row twice is that row; the scale is that of both."""
    c = Cache8(2, 2, 16, 8, 2, 64, 64, 21)
    c.lens.copy_(ints([20, 9]))
    kn, vn = new_rows(c.g, 4, 2, 64), new_rows(c.g, 4, 2, 64)
    kn[2], vn[2] = kn[1], vn[1]
    append(hsp, c, [0, 0, 0, 1], [16, 18, 18, 3], 64, 2, 64, kn=kn, vn=vn)
    kn[2] *= 64                                                        # (another row: the place holds numbers of either)
    hsp.cache_append_q8(kn, vn, c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=ints([0, 0, 0, 1]), positions=ints([16, 18, 18, 3]))
    hsp.check_device_error()
    got, _ = hsp.cache_read_q8(c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=ints([0]), positions=ints([18]))
    for h in range(2):
        s = float(c.ks[int(c.table[0, 1]), 0, h])
        either = [nearest(numbers(kn)[i, h] / s) * s for i in (1, 2)]
        assert float(numbers(kn)[2, h].max()) <= 448 * s
        x = numbers(got)[0, h]
        assert ((x == either[0]) | (x == either[1])).all()


def test_without_dependent_launches_and_from_threads(hsp):
    """pdl off, then four threads at once, each with a cache and a stream of its own: the same bytes as alone."""
    import threading

    def work(seed, stream):
        with torch.cuda.stream(stream):
            c = Cache8(4, 4, 32, 16, 2, 128, 128, seed)
            c.lens.copy_(ints([128] * 4))
            rows, pos = ints([i // 60 for i in range(240)]), ints([i % 60 + 3 for i in range(240)])
            kn, vn, q, cs = new_rows(c.g, 240, 2, 128), new_rows(c.g, 240, 2, 128), new_rows(c.g, 240, 8, 128), angles(128, 128)
            out = []
            for _ in range(5):
                qt = hsp.cache_append_q8(kn, vn, c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=rows, positions=pos, cos_sin=cs, q=q)
                read = hsp.cache_read_q8(c.k, c.v, c.ks, c.vs, c.table, c.lens, rows=rows, positions=pos)
                att = hsp.paged_attention_q8(qt[::60].contiguous(), c.k, c.v, c.ks, c.vs, c.table, c.lens, 0.09)
                out += [qt, *read, att]
            stream.synchronize()
        return [t.cpu() for t in out]

    hsp.set_options(pdl=False)
    try:
        want = [work(seed, torch.cuda.current_stream()) for seed in range(4)]
    finally:
        hsp.set_options(pdl=True)
    got, streams = [None] * 4, [torch.cuda.Stream() for _ in range(4)]

    def run(i):
        got[i] = work(i, streams[i])

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    hsp.check_device_error()
    for a, b in zip(want, got):
        assert b is not None and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
