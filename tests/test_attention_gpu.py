"""proj_paged_attention against softmax attention in 64 bits.

Tolerances, derived before the first run.  With p_t the exact softmax weights, A = sum_t p_t |v_t| and
s = scale * sum_i |q_i k_i| (the largest over t):
  * a score is an fp32 sum of dk products: off by at most dk * 2^-24 * s, and by 2^-22 of its size for the
    scaling and the exponential; a weight and the sum l are off by that (relative) each, l by len * 2^-24 more;
  * a weight is rounded to bf16 once for the product: at most half a step, 2^-8, relative to the weight, so
    2^-8 * A in the result (l adds the unrounded weights);
  * the fp32 sum over the tokens: len * 2^-24 * A; joining parts: a few 2^-24 * A more;
  * the result is rounded to bf16 once: 2^-8 |o|.
"""
import math

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


def make(lens, heads, kv_heads, dk, latent, page, seed, std=1.0, hnd=False, spare=2):
    """A cache whose pages lie in no order, every place behind a sequence's last token NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    width = max(max(counts), 1) + 1
    table = torch.full((len(lens), width), 2 ** 30, dtype=torch.int32, device="cuda")   # never read past a row's pages
    shape = (pages, kv_heads, page, dk) if hnd else (pages, page, kv_heads, dk)

    def pool():
        t = torch.full(shape, float("nan"), dtype=BF, device="cuda")
        return t.transpose(1, 2) if hnd else t

    k, v = pool(), None if latent else pool()
    at = 0
    for b, n in enumerate(lens):
        ids = perm[at:at + counts[b]]
        at += counts[b]
        table[b, :counts[b]] = ids
        for t in (k, v):
            if t is None or n == 0:
                continue
            rows = (torch.randn(n, kv_heads, dk, generator=g, device="cuda") * std).to(BF)
            tok = torch.arange(n, device="cuda")
            t[ids.long()[tok // page], tok % page] = rows
    q = torch.randn(len(lens), heads, dk, generator=g, device="cuda").to(BF)
    return q, k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def reference(q, k, v, table, lens, scale, dv, rows=None):
    """(out, lse, bound of out, bound of lse) in 64 bits."""
    B, H, dk = q.shape
    page, kv = k.shape[1], k.shape[2]
    G = H // kv
    out = torch.zeros(B, H, dv, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        r = b if rows is None else rows[b]
        n = int(lens[r])
        if n == 0:
            continue
        ids = table[r, : -(-n // page)].long()
        kk = k[ids].flatten(0, 1)[:n].double()
        vv = kk[..., :dv] if v is None else v[ids].flatten(0, 1)[:n].double()
        for h in range(kv):
            at = slice(h * G, (h + 1) * G)
            qq = q[b, at].double()
            x = qq @ kk[:, h].T * scale
            p = torch.softmax(x, -1)
            out[b, at] = p @ vv[:, h]
            lse[b, at] = torch.logsumexp(x, -1)
            s = float((qq.abs() @ kk[:, h].abs().T).max()) * abs(scale)
            rel = dk * 2.0 ** -24 * s + 2.0 ** -22 * (1 + float(x.abs().max()))
            a = p @ vv[:, h].abs()
            tol[b, at] = a * (2.0 ** -8 + 2 * rel + (2 * n + 64) * 2.0 ** -24) + out[b, at].abs() * 2.0 ** -8
            ltol[b, at] = rel + (n + 64) * 2.0 ** -24 + lse[b, at].abs() * 2.0 ** -22
    return out, lse, tol, ltol


def check(hsp, args, scale, dv, **kw):
    q, k, v, table, lens = args
    rows = kw.pop("rows", None)
    out, lse = hsp.paged_attention(q, k, v, table, lens, scale, v_dim=dv, return_lse=True, rows=rows, **kw)
    hsp.check_device_error()
    ref, rlse, tol, ltol = reference(q, k, v, table, lens, scale, dv, None if rows is None else rows.tolist())
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), f"out off by {float((err - tol).max()):.3e}, {int((err > tol).sum())} of {err.numel()}"
    empty = torch.isinf(rlse)
    assert torch.equal(torch.isneginf(lse), empty)
    lerr = (lse.double() - rlse).abs().masked_fill(empty, 0)
    assert (lerr <= ltol).all(), f"lse off by {float((lerr - ltol).max()):.3e}"
    return out, lse


# the smallest first: one tile, then tiles that end inside, pages that end inside a tile, several parts
LATENT = [([1], 16, 64), ([64], 16, 64), ([63], 1, 64), ([65], 7, 16), ([77], 16, 64), ([0], 16, 64),
          ([128, 0, 129, 1], 16, 32), ([300, 17, 1000], 20, 128), ([5, 700], 64, 64), ([130, 64], 128, 16),
          ([2000, 3, 0, 0, 999], 96, 256), ([20011], 16, 64), ([9000, 8000], 65, 1024)]


@pytest.mark.parametrize("dk", [576, 512])
@pytest.mark.parametrize("lens,heads,page", LATENT)
def test_latent(hsp, lens, heads, page, dk):
    check(hsp, make(lens, heads, 1, dk, True, page, 100 + len(lens) + heads), 192 ** -0.5, 512)


GROUPED = [([1], 1, 1, 64), ([64], 4, 4, 64), ([63, 0], 8, 2, 16), ([65], 3, 1, 16), ([129, 5, 640], 32, 8, 16),
           ([2, 1, 3], 40, 5, 32), ([777], 16, 1, 128), ([1000, 300], 64, 2, 64), ([513, 4000], 96, 2, 64),
           ([12345], 8, 8, 1024), ([700, 0, 0, 31], 130, 2, 32)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,heads,kv,page", GROUPED)
def test_grouped(hsp, lens, heads, kv, page, d):
    check(hsp, make(lens, heads, kv, d, False, page, 7 + heads), d ** -0.5, d)


# Every shape of the copy ring (columns, head tiles), over sequences long enough for each CTA to go around it
# several times, next to short ones: what each warp waits for has to be the use of a place that it means.
RAGGED = [64, 64, 63, 1, 1, 63, 7560, 0, 64, 0, 7122, 64, 0, 7560, 2569, 276, 7560, 0, 1, 2123, 65, 1, 65, 2814, 6038, 1954,
          1793, 0, 65, 0, 2096, 1, 6664, 7484, 1, 1930, 63, 4785, 4611]


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("d,kv,group", [(128, 3, 16), (128, 3, 17), (128, 3, 40), (64, 3, 5), (64, 3, 17), (64, 3, 64)])
def test_grouped_rings(hsp, d, kv, group, page):
    args = make(RAGGED, kv * group, kv, d, False, page, 616 + group)
    first = check(hsp, args, -0.1, d)
    for _ in range(20):                                     # other timings, the same bits
        out, lse = hsp.paged_attention(*args, -0.1, v_dim=d, return_lse=True)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    hsp.check_device_error()


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("dk,heads", [(576, 16), (576, 32), (576, 64), (576, 100), (512, 16), (512, 32), (512, 64)])
def test_latent_rings(hsp, dk, heads, page):
    args = make(RAGGED, heads, 1, dk, True, page, 617 + heads)
    first = check(hsp, args, 0.06, 512)
    for _ in range(20):
        out, lse = hsp.paged_attention(*args, 0.06, return_lse=True)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    hsp.check_device_error()


@pytest.mark.parametrize("latent", [True, False])
def test_many_sequences(hsp, latent):
    lens = [(37 * i) % 301 for i in range(391)]            # more sequences than threads, empty ones among them
    dk, dv, heads, kv = (576, 512, 16, 1) if latent else (128, 128, 8, 2)
    check(hsp, make(lens, heads, kv, dk, latent, 16, 3), dk ** -0.5, dv)


@pytest.mark.parametrize("latent", [True, False])
def test_many_short_sequences_are_not_cut(hsp, latent):
    """Tables of at most 256 tokens per row: one launch, no workspace."""
    lens = [(37 * i) % 241 for i in range(700)]
    dk, dv, heads, kv = (512, 512, 70, 1) if latent else (64, 64, 6, 3)
    args = make(lens, heads, kv, dk, latent, 16, 13)
    assert args[3].shape[1] * 16 == 256
    n = hsp.launch_count()
    check(hsp, args, dk ** -0.5, dv)
    assert hsp.launch_count() == n + 1


@pytest.mark.parametrize("latent", [True, False])
def test_a_padded_batch(hsp, latent):
    """A batch padded with empty sequences, before, between and behind the others: zeros there, and the others as
    without them (the CTAs and their cuts are the same)."""
    dk, dv, kv = (576, 512, 1) if latent else (128, 128, 2)
    q, k, v, table, lens = make([900, 0, 77] + [0] * 250 + [1500], 16, kv, dk, latent, 64, 23)
    out, lse = check(hsp, (q, k, v, table, lens), 0.07, dv)
    assert (out[lens == 0] == 0).all() and torch.isneginf(lse[lens == 0]).all()
    rows = torch.tensor([0, 2, 253], dtype=torch.int32, device="cuda")
    packed = hsp.paged_attention(q[rows.long()], k, v, table, lens, 0.07, rows=rows)
    assert torch.equal(packed, out[rows.long()])


@pytest.mark.parametrize("latent", [True, False])
def test_a_cache_past_four_gigabytes(hsp, latent):
    """Pages whose offsets do not fit 32 bits, neither in bytes nor in elements."""
    dk, dv, kv, heads, page = (576, 512, 1, 16, 64) if latent else (128, 128, 4, 8, 64)
    lens = [200, 129]
    q, k, v, table, ln = make(lens, heads, kv, dk, latent, page, 17)
    pages = 2 ** 32 // (page * kv * dk) + 40                        # more than 2^32 elements
    at = pages - 1 - torch.arange(7, device="cuda") * 3
    move = {}

    def far(t):
        big = torch.empty((pages,) + tuple(t.shape[1:]), dtype=BF, device="cuda")
        big[at] = t[:7]
        return big

    assert k.shape[0] <= 9 and int(table[table < 2 ** 30].max()) < 9
    used = sorted(set(table[table < 2 ** 30].tolist()))
    move = {u: int(at[i]) for i, u in enumerate(used)}
    order = torch.tensor(used, device="cuda")
    big_k, big_v = far(k[order]), None if latent else far(v[order])
    far_table = table.clone()
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            far_table[b, j] = move[int(table[b, j])]
    want = hsp.paged_attention(q, k, v, table, ln, 0.07)
    assert torch.equal(hsp.paged_attention(q, big_k, big_v, far_table, ln, 0.07), want)
    # and the new tokens of the next step land there
    kn = torch.randn(2, kv, dk, device="cuda").to(BF)
    hsp.cache_append(kn, None if latent else kn, big_k, big_v, far_table, ln)
    hsp.check_device_error()
    for b, n in enumerate(lens):
        p = int(far_table[b, (n - 1) // page])
        assert p * page * kv * dk >= 2 ** 32 - 40 * page * kv * dk
        assert torch.equal(big_k[p, (n - 1) % page], kn[b])
        assert latent or torch.equal(big_v[p, (n - 1) % page], kn[b])


@pytest.mark.parametrize("latent", [True, False])
def test_heads_before_tokens_and_strided_queries(hsp, latent):
    """Pages that hold head after head, queries and keys that are columns of wider tensors."""
    dk, dv, kv = (576, 512, 2) if latent else (128, 128, 2)
    q, k, v, table, lens = make([130, 70], 8, kv, dk, latent, 64, 5, hnd=True)
    wide = torch.randn(2, 9, dk + 24, device="cuda").to(BF)
    wide[:, :8, 16:16 + dk] = q
    kw = torch.randn(k.shape[0], 64, kv, dk + 64, device="cuda").to(BF)
    kw[..., :dk] = k
    tw = torch.full((2, table.shape[1] + 3), -5, dtype=torch.int32, device="cuda")
    tw[:, :table.shape[1]] = table
    args = (wide[:, :8, 16:16 + dk], kw[..., :dk], v, tw[:, :table.shape[1]], lens)
    a, la = check(hsp, args, 0.07, dv)
    b, lb = check(hsp, (q, k, v, table, lens), 0.07, dv)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_rows_select_and_repeat(hsp):
    args = make([100, 0, 257, 64], 16, 1, 576, True, 64, 9)
    q = torch.randn(6, 16, 576, device="cuda").to(BF)
    rows = torch.tensor([3, 2, 2, 0, 1, 2], dtype=torch.int32, device="cuda")
    check(hsp, (q,) + args[1:], 192 ** -0.5, 512, rows=rows)


@pytest.mark.parametrize("scale", [3.0, -0.2, 0.0])
@pytest.mark.parametrize("latent", [True, False])
def test_scores_that_grow_along_the_sequence(hsp, latent, scale):
    """Every tile exceeds the maximum so far by far, so O is rescaled tile after tile; and a negative and a zero scale."""
    dk, dv = (576, 512) if latent else (64, 64)
    q, k, v, table, lens = make([1500], 16, 1, dk, latent, 64, 21, std=0.05)
    ids = table[0, :24].long()
    ramp = torch.linspace(0.0, 1.0, 1500, device="cuda")
    kk = k[ids].flatten(0, 1)
    kk[:1500, 0] = (kk[:1500, 0].float() + ramp[:, None] * q[0, 0].float()[None]).to(BF)
    k[ids] = kk.view(24, 64, 1, dk)
    check(hsp, (q, k, v, table, lens), scale * dk ** -0.5, dv)


def test_one_token_takes_all_the_weight(hsp):
    q, k, v, table, lens = make([900], 16, 1, 128, False, 16, 2, std=0.01)
    at = 531
    k[table[0, at // 16].long(), at % 16, 0] = (q[0, 3].float() * 4).to(BF)
    out, _ = check(hsp, (q, k, v, table, lens), 1.0, 128)
    assert torch.equal(out[0, 3], v[table[0, at // 16].long(), at % 16, 0])


def test_infinite_and_nan_inputs_stay_where_they_are(hsp):
    """NaN in one query head, and a key that gives -infinity: the other heads are as before."""
    args = list(make([200], 16, 1, 576, True, 64, 4))
    clean = hsp.paged_attention(*args, 0.07)
    args[0] = args[0].clone()
    args[0][0, 5] = float("nan")
    out = hsp.paged_attention(*args, 0.07)
    keep = [h for h in range(16) if h != 5]
    assert torch.equal(out[0, keep], clean[0, keep]) and torch.isnan(out[0, 5]).all()
    q, k, v, table, lens = make([130], 4, 1, 64, False, 16, 4)
    q[...] = 1.0
    k[table[0, 2].long(), 3, 0] = float("-inf")            # score -infinity: weight 0
    out, lse = hsp.paged_attention(q, k, v, table, lens, 0.125, return_lse=True)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    hsp.check_device_error()


def test_repeat_graph_and_side_stream_bitwise(hsp):
    lens = [4000, 65, 0, 2500, 1]
    args = make(lens, 16, 1, 576, True, 64, 31)
    first = hsp.paged_attention(*args, 0.07, return_lse=True)
    again = hsp.paged_attention(*args, 0.07, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = hsp.paged_attention(*args, 0.07, return_lse=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    hsp.set_options(pdl=False)
    try:
        assert torch.equal(hsp.paged_attention(*args, 0.07), first[0])
    finally:
        hsp.set_options(pdl=True)
    # captured: new queries, new lengths, the same addresses; two graphs live at once
    q, k, v, table, ln = args
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(hsp.paged_attention(q, k, v, table, ln, 0.07, return_lse=True))
        graphs.append(g)
    for step, new in enumerate(([4000, 65, 0, 2500, 1], [3999, 1, 0, 64, 0])):
        q.copy_(torch.randn(q.shape, generator=torch.Generator("cuda").manual_seed(step), device="cuda"))
        ln.copy_(torch.tensor(new, dtype=torch.int32))
        want = hsp.paged_attention(q, k, v, table, ln, 0.07, return_lse=True)
        for g, o in zip(graphs, outs):
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want))
    hsp.check_device_error()


def test_two_streams_at_once(hsp):
    a, b = make([3000, 40], 16, 1, 576, True, 64, 1), make([700] * 9, 8, 2, 128, False, 16, 2)
    wa, wb = hsp.paged_attention(*a, 0.07), hsp.paged_attention(*b, 0.09)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        with torch.cuda.stream(s1):
            x = hsp.paged_attention(*a, 0.07)
        with torch.cuda.stream(s2):
            y = hsp.paged_attention(*b, 0.09)
        got.append((x, y))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in got)


def test_outputs_lie_between_untouched_bytes(hsp):
    args = make([150, 9], 5, 1, 512, True, 16, 8)
    buf = torch.full((2 * 4096 + 2 * 5 * 512,), 7.0, dtype=BF, device="cuda")
    out = buf[4096:4096 + 2 * 5 * 512].view(2, 5, 512)
    check(hsp, args, 0.07, 512, out=out)
    assert (buf[:4096] == 7).all() and (buf[-4096:] == 7).all()
    need = hsp.paged_attention_workspace_bytes(5, 1, 512, 512, True)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    assert torch.equal(hsp.paged_attention(*args, 0.07, workspace=ws[:need]), out)
    assert (ws[need:] == 0x5A).all()


def test_bad_pages_rows_and_lengths_are_reported(hsp):
    import hidden_state_projection_gb300 as m

    def expect(args, **kw):
        out = hsp.paged_attention(*args, 0.07, **kw)
        with pytest.raises(m.ProjError) as ei:
            hsp.check_device_error()
        assert ei.value.status_name == "PROJ_ERR_BAD_INDEX"
        hsp.check_device_error()                            # cleared
        return out

    q, k, v, table, lens = make([200, 100], 16, 1, 576, True, 64, 6)
    good = hsp.paged_attention(q, k, v, table, lens, 0.07)
    for bad in (-1, k.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        out = expect((q, k, v, t, lens))
        assert torch.equal(out[1], good[1])                 # the other sequence is as it was
    for n in (-3, table.shape[1] * 64 + 1):
        ln = lens.clone()
        ln[0] = n
        t = table.clone()
        t[0] = t[0, 0]
        expect((q, k, v, t, ln))
    expect((q, k, v, table, lens), rows=torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
    expect((q, k, v, table, lens), rows=torch.tensor([-1, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(hsp.paged_attention(q, k, v, table, lens, 0.07), good)
    hsp.check_device_error()


@pytest.mark.parametrize("latent", [True, False])
def test_bounded_waits_report_a_timeout(hsp, latent):
    """The test hook leaves the first tile of every CTA unloaded (the only one that every CTA has): the waits run out,
    and the next call is right again."""
    import hidden_state_projection_gb300 as m
    dk, dv = (576, 512) if latent else (128, 128)
    args = make([3000], 16, 1, dk, latent, 64, 12)
    want = hsp.paged_attention(*args, 0.07)
    hsp.set_options(pdl=True, wait_limit_us=20000, skip_stage=0)
    try:
        hsp.paged_attention(*args, 0.07)
        with pytest.raises(m.ProjError) as ei:
            hsp.check_device_error()
        assert ei.value.status_name == "PROJ_ERR_TIMEOUT"
    finally:
        hsp.set_options(pdl=True, wait_limit_us=0, skip_stage=None)
    assert torch.equal(hsp.paged_attention(*args, 0.07), want)
    hsp.check_device_error()


def test_no_sequences(hsp):
    q, k, v, table, lens = make([10], 4, 1, 576, True, 64, 1)
    n = hsp.launch_count()
    assert hsp.paged_attention(q[:0], k, v, table, lens, 0.07).shape == (0, 4, 512)
    assert hsp.launch_count() == n
