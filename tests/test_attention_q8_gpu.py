"""proj_paged_attention_q8 against softmax attention in 64 bits over the values that the codes and scales stand for.

Tolerances, derived before the first run.  With p_t the exact softmax weights, w_t = p_t vs_t, A = sum_t p_t |v_t|, and
s = scale * sum_i |q_i k_i| (the largest over t):
  * queries in two e4m3 pieces under the head's own power of two, 2^e <= max |q| / 224: exact but for what lies below
    2^-14 * 2^e, so 2^-21.8 max |q| each: a score is off by that times scale * sum_i |k_i|;
  * a score is an fp32 sum of dk products: dk * 2^-24 * s, and 2^-22 of its size for the scaling, the logarithm of the
    values' scale and the exponential; a weight and the sum l are off by that (relative) each, l by len * 2^-24 more;
  * a weight in two pieces, e4m3 (half a step 2^-4) and e5m2 (2^-3): 2^-7 of it while it is at least 2^-6; of a smaller
    one an eighth of 2^-10: 2^-13.  In these units the largest w of every 128-token tile is at least 2^-4, and that of the
    tile that set them 2^3, which the row's is not below: so 2^-9 of the tile's largest and 2^-16 of the row's, the smaller
    of the two.  fp16 in between: 2^-11.  The same in l, which the sum is divided by;
  * the fp32 sum over the tokens: len * 2^-24 * A; joining parts: a few 2^-24 * A more;
  * the result is rounded to bf16 once: 2^-8 |o|.
Rounding errors of many weights are as good as independent, and the bound above then far too wide.  So the 2-norm of all
errors is held too: with d_t the bound of a weight's error, the result's is sum_t d_t (vc_t - o / vs_t) / L at random signs,
whose square is at most sum_t d_t^2 (|vc_t| + |o| / vs_t)^2 on average, a third of that for errors spread evenly up to their
bounds; and 2^-8 |o| for the rounding, likewise.  The sum of these squares without the third is the bound.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
NAN8 = 0x7F


@pytest.fixture(scope="module")
def hsp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import hidden_state_projection_gb300 as m
    m.lib()
    m.set_options(pdl=True, wait_limit_us=0, skip_stage=None)
    return m


def make(lens, heads, kv_heads, dk, latent, page, seed, block=16, std=1.0, hnd=False, spare=2, spread=3):
    """A cache whose pages lie in no order, every code behind a sequence's last token NaN, scales there NaN too."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    block = min(block, page)
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    width = max(max(counts), 1) + 1
    table = torch.full((len(lens), width), 2 ** 30, dtype=torch.int32, device="cuda")   # never read past a row's pages
    shape = (pages, kv_heads, page, dk) if hnd else (pages, page, kv_heads, dk)

    def pool():
        t = torch.full(shape, NAN8, dtype=torch.uint8, device="cuda").view(F8)
        return (t.transpose(1, 2) if hnd else t), torch.full((pages, page // block, kv_heads), float("nan"), device="cuda")

    k, ks = pool()
    v, vs = (None, None) if latent else pool()
    at = 0
    for b, n in enumerate(lens):
        ids = perm[at:at + counts[b]]
        at += counts[b]
        table[b, :counts[b]] = ids
        for t, sc in ((k, ks), (v, vs)):
            if t is None or n == 0:
                continue
            nb = -(-n // block)
            e = torch.randint(-spread, spread + 1, (nb, kv_heads), generator=g, device="cuda").float()
            blk, tok = torch.arange(nb, device="cuda"), torch.arange(n, device="cuda")
            sc[ids.long()[blk * block // page], blk % (page // block)] = 2.0 ** (e - 6) * std
            rows = torch.randn(n, kv_heads, dk, generator=g, device="cuda") * 2.0 ** (6 - e)[tok // block][..., None]
            t.view(torch.uint8)[ids.long()[tok // page], tok % page] = rows.clamp(-448, 448).to(F8).view(torch.uint8)
    q = torch.randn(len(lens), heads, dk, generator=g, device="cuda").to(BF)
    return q, k, v, ks, vs, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def held(codes, scales, ids, n):
    """Codes [n, kv_heads, dim] and scales [n, kv_heads] of a sequence in 64 bits."""
    block = codes.shape[1] // scales.shape[1]
    c = codes.view(torch.uint8)[ids].view(F8).double().flatten(0, 1)[:n]
    return c, scales[ids].double().repeat_interleave(block, 1).flatten(0, 1)[:n]


def reference(q, k, v, ks, vs, table, lens, scale, dv, rows=None):
    """(out, lse, bound of out, bound of lse, the squares' bound) in 64 bits."""
    B, H, dk = q.shape
    page, kv = k.shape[1], k.shape[2]
    G = H // kv
    out = torch.zeros(B, H, dv, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    tol, ltol, square = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(out)
    for b in range(B):
        r = b if rows is None else rows[b]
        n = int(lens[r])
        if n == 0:
            continue
        ids = table[r, : -(-n // page)].long()
        kc, kscale = held(k, ks, ids, n)
        vc, vscale = (kc[..., :dv], kscale) if v is None else held(v, vs, ids, n)
        for h in range(kv):
            at = slice(h * G, (h + 1) * G)
            qq = q[b, at].double()
            kk, vv = kc[:, h] * kscale[:, h, None], vc[:, h] * vscale[:, h, None]
            x = qq @ kk.T * scale
            p = torch.softmax(x, -1)
            out[b, at] = p @ vv
            lse[b, at] = torch.logsumexp(x, -1)
            s = float((qq.abs() @ kk.abs().T).max()) * abs(scale)
            rel = dk * 2.0 ** -24 * s + 2.0 ** -22 * (1 + float(x.abs().max()))
            rel += float(qq.abs().max() * kk.abs().sum(-1).max()) * abs(scale) * 2.0 ** -21.8
            a = p @ vv.abs()
            pad = -n % 128
            w = torch.nn.functional.pad(p * vscale[:, h], (0, pad)).unflatten(-1, (-1, 128)).amax(-1)          # [G, tiles]
            w = torch.minimum(w * 2.0 ** -9, w.amax(-1, keepdim=True) * 2.0 ** -16)
            codes = torch.nn.functional.pad(vc[:, h].abs(), (0, 0, 0, pad)).unflatten(0, (-1, 128)).sum(1)     # [tiles, dv]
            inv = torch.nn.functional.pad(1 / vscale[:, h], (0, pad)).view(-1, 128).sum(-1)                    # [tiles]
            o = out[b, at].abs()
            tol[b, at] = (a + o) * (2.0 ** -7 + 2.0 ** -11) + w @ codes + o * (w @ inv)[:, None]
            tol[b, at] += a * (2 * rel + (2 * n + 64) * 2.0 ** -24) + o * 2.0 ** -8
            vs1 = vscale[:, h]
            d2 = ((p * vs1) * (2.0 ** -7 + 2.0 ** -11) + w.repeat_interleave(128, -1)[:, :n]) ** 2
            square[b, at] = d2 @ vc[:, h] ** 2 + 2 * o * ((d2 / vs1) @ vc[:, h].abs()) + o ** 2 * (d2 / vs1 ** 2).sum(-1, keepdim=True)
            square[b, at] += (2.0 ** -8 * o + a * 2 * rel) ** 2
            ltol[b, at] = rel + (n + 64) * 2.0 ** -24 + lse[b, at].abs() * 2.0 ** -22
    return out, lse, tol, ltol, square


def check(hsp, args, scale, dv, **kw):
    rows = kw.pop("rows", None)
    out, lse = hsp.paged_attention_q8(*args, scale, v_dim=dv, return_lse=True, rows=rows, **kw)
    hsp.check_device_error()
    ref, rlse, tol, ltol, square = reference(*args, scale, dv, None if rows is None else rows.tolist())
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), f"out off by {float((err - tol).max()):.3e}, {int((err > tol).sum())} of {err.numel()}"
    norm, most = float(torch.linalg.norm(err)), float(square.sum().sqrt())
    assert norm <= most, f"2-norm of the errors {norm:.3e}, {most:.3e} at most"
    empty = torch.isinf(rlse)
    assert torch.equal(torch.isneginf(lse), empty)
    lerr = (lse.double() - rlse).abs().masked_fill(empty, 0)
    assert (lerr <= ltol).all(), f"lse off by {float((lerr - ltol).max()):.3e}"
    return out, lse


# the smallest first: one tile, then tiles that end inside, pages that end inside a tile, several parts
LATENT = [([1], 16, 64), ([128], 16, 64), ([127], 1, 64), ([129], 7, 16), ([77], 16, 64), ([0], 16, 64),
          ([256, 0, 257, 1], 16, 32), ([300, 17, 1000], 20, 128), ([5, 700], 64, 64), ([130, 64], 128, 16),
          ([2000, 3, 0, 0, 999], 96, 256), ([20011], 16, 64), ([9000, 8000], 65, 1024)]


@pytest.mark.parametrize("dk", [576, 512])
@pytest.mark.parametrize("lens,heads,page", LATENT)
def test_latent(hsp, lens, heads, page, dk):
    check(hsp, make(lens, heads, 1, dk, True, page, 100 + len(lens) + heads), 192 ** -0.5, 512)


GROUPED = [([1], 1, 1, 64), ([128], 4, 4, 64), ([127, 0], 8, 2, 16), ([129], 3, 1, 16), ([257, 5, 640], 32, 8, 16),
           ([2, 1, 3], 40, 5, 32), ([777], 16, 1, 128), ([1000, 300], 64, 2, 64), ([513, 4000], 96, 2, 64),
           ([12345], 8, 8, 1024), ([700, 0, 0, 31], 130, 2, 32)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,heads,kv,page", GROUPED)
def test_grouped(hsp, lens, heads, kv, page, d):
    check(hsp, make(lens, heads, kv, d, False, page, 7 + heads), d ** -0.5, d)


@pytest.mark.parametrize("page,block", [(16, 1), (16, 16), (64, 4), (128, 128), (1024, 256)])
@pytest.mark.parametrize("latent", [True, False])
def test_blocks(hsp, latent, page, block):
    """A scale for every token up to one for many tiles, and scales that differ by 2^20."""
    dk, dv, kv = (576, 512, 1) if latent else (128, 128, 3)
    check(hsp, make([700, 33], 12, kv, dk, latent, page, 40 + block, block=block), 0.07, dv)
    args = make([500, 1300], 12, kv, dk, latent, page, 41 + block, block=block, spread=10, std=2.0 ** -9)
    check(hsp, args, 0.002, dv)


# Every shape of the copy ring (columns, head tiles), over sequences long enough for each CTA to go around it
# several times, next to short ones.
RAGGED = [64, 128, 127, 1, 1, 63, 7560, 0, 64, 0, 7122, 64, 0, 7560, 2569, 276, 7560, 0, 1, 2123, 129, 1, 65, 2814, 6038, 1954,
          1793, 0, 65, 0, 2096, 1, 6664, 7484, 1, 1930, 127, 4785, 4611]


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("d,kv,group", [(128, 3, 16), (128, 3, 17), (128, 3, 40), (64, 3, 5), (64, 3, 17), (64, 3, 64)])
def test_grouped_rings(hsp, d, kv, group, page):
    args = make(RAGGED, kv * group, kv, d, False, page, 616 + group)
    first = check(hsp, args, -0.1, d)
    for _ in range(20):                                     # other timings, the same bits
        out, lse = hsp.paged_attention_q8(*args, -0.1, v_dim=d, return_lse=True)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    hsp.check_device_error()


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("dk,heads", [(576, 16), (576, 32), (576, 64), (576, 100), (512, 16), (512, 32), (512, 64)])
def test_latent_rings(hsp, dk, heads, page):
    args = make(RAGGED, heads, 1, dk, True, page, 617 + heads)
    first = check(hsp, args, 0.06, 512)
    for _ in range(20):
        out, lse = hsp.paged_attention_q8(*args, 0.06, return_lse=True)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    hsp.check_device_error()


@pytest.mark.parametrize("latent", [True, False])
def test_many_sequences(hsp, latent):
    lens = [(37 * i) % 301 for i in range(391)]            # more sequences than threads, empty ones among them
    dk, dv, heads, kv = (576, 512, 16, 1) if latent else (128, 128, 8, 2)
    check(hsp, make(lens, heads, kv, dk, latent, 16, 3), dk ** -0.5, dv)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_a_part_for_every_sm(hsp, d, page):
    """From 152 sequences and kv heads on three CTAs share an SM: cut and whole ones, with shorter rings."""
    lens = [(331 * i) % 1500 for i in range(38)] + [4000, 0]
    check(hsp, make(lens, 20, 4, d, False, page, 9), d ** -0.5, d)


@pytest.mark.parametrize("latent", [True, False])
def test_many_short_sequences_are_not_cut(hsp, latent):
    """Tables of at most 256 tokens per row: no join."""
    lens = [(37 * i) % 241 for i in range(700)]
    dk, dv, heads, kv = (512, 512, 70, 1) if latent else (64, 64, 6, 3)
    args = make(lens, heads, kv, dk, latent, 16, 13)
    assert args[5].shape[1] * 16 == 256
    n = hsp.launch_count()
    check(hsp, args, dk ** -0.5, dv)
    assert hsp.launch_count() == n + 2


@pytest.mark.parametrize("latent", [True, False])
def test_a_padded_batch(hsp, latent):
    """A batch padded with empty sequences: zeros there, and the others as without them."""
    dk, dv, kv = (576, 512, 1) if latent else (128, 128, 2)
    q, k, v, ks, vs, table, lens = make([900, 0, 77] + [0] * 250 + [1500], 16, kv, dk, latent, 64, 23)
    out, lse = check(hsp, (q, k, v, ks, vs, table, lens), 0.07, dv)
    assert (out[lens == 0] == 0).all() and torch.isneginf(lse[lens == 0]).all()
    rows = torch.tensor([0, 2, 253], dtype=torch.int32, device="cuda")
    packed = hsp.paged_attention_q8(q[rows.long()], k, v, ks, vs, table, lens, 0.07, rows=rows)
    assert torch.equal(packed, out[rows.long()])


@pytest.mark.parametrize("latent", [True, False])
def test_a_cache_past_four_gigabytes(hsp, latent):
    """Pages whose offsets do not fit 32 bits; the new tokens of the next step land there and are read back."""
    dk, dv, kv, heads, page = (576, 512, 1, 16, 64) if latent else (128, 128, 4, 8, 64)
    lens = [200, 129]
    q, k, v, ks, vs, table, ln = make(lens, heads, kv, dk, latent, page, 17)
    pages = 2 ** 32 // (page * kv * dk) + 40
    at = pages - 1 - torch.arange(7, device="cuda") * 3
    used = sorted(set(table[table < 2 ** 30].tolist()))
    order = torch.tensor(used, device="cuda")

    def far(t):
        if t is None:
            return None
        big = torch.empty((pages,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda")
        big.view(torch.uint8 if t.dtype == F8 else t.dtype)[at] = t.view(torch.uint8 if t.dtype == F8 else t.dtype)[order][:7]
        return big

    assert len(used) == 7
    big = [far(t) for t in (k, v, ks, vs)]
    far_table = table.clone()
    for i, u in enumerate(used):
        far_table[table == u] = int(at[i])
    want = hsp.paged_attention_q8(q, k, v, ks, vs, table, ln, 0.07)
    assert torch.equal(hsp.paged_attention_q8(q, *big, far_table, ln, 0.07), want)
    kn = torch.randn(2, kv, dk, device="cuda").to(BF)
    for pool, tab in (([k, v, ks, vs], table), (big, far_table)):
        hsp.cache_append_q8(kn, None if latent else kn, *pool, tab, ln)
    a, b = hsp.cache_read_q8(k, v, ks, vs, table, ln), hsp.cache_read_q8(*big, far_table, ln)
    hsp.check_device_error()
    assert torch.equal(a[0], b[0]) and (latent or torch.equal(a[1], b[1]))
    assert ((a[0] - kn).abs() <= 2.0 ** -4 * kn.abs() + 2.0 ** -10 * 2.0 ** -3).all()   # (no scale above 2^-3: half of 2^-9 of it)


@pytest.mark.parametrize("latent", [True, False])
def test_heads_before_tokens_and_strided_inputs(hsp, latent):
    """Pages that hold head after head, queries and codes that are columns of wider tensors, scales in another order."""
    dk, dv, kv = (576, 512, 2) if latent else (128, 128, 2)
    q, k, v, ks, vs, table, lens = make([130, 70], 8, kv, dk, latent, 64, 5, hnd=True)
    wide = torch.randn(2, 9, dk + 24, device="cuda").to(BF)
    wide[:, :8, 16:16 + dk] = q
    kw = torch.zeros(k.shape[0], 64, kv, dk + 64, dtype=torch.uint8, device="cuda")
    kw[..., :dk] = k.view(torch.uint8)
    sw = torch.zeros(kv, k.shape[0], 9, device="cuda")
    sw[:, :, 3:7] = ks.permute(2, 0, 1)
    tw = torch.full((2, table.shape[1] + 3), -5, dtype=torch.int32, device="cuda")
    tw[:, :table.shape[1]] = table
    args = (wide[:, :8, 16:16 + dk], kw.view(F8)[..., :dk], v, sw[:, :, 3:7].permute(1, 2, 0), vs, tw[:, :table.shape[1]], lens)
    a, la = check(hsp, args, 0.07, dv)
    b, lb = check(hsp, (q, k, v, ks, vs, table, lens), 0.07, dv)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_rows_select_and_repeat(hsp):
    args = make([100, 0, 257, 64], 16, 1, 576, True, 64, 9)
    q = torch.randn(6, 16, 576, device="cuda").to(BF)
    rows = torch.tensor([3, 2, 2, 0, 1, 2], dtype=torch.int32, device="cuda")
    check(hsp, (q,) + args[1:], 192 ** -0.5, 512, rows=rows)


def shape_scores(args, weights, dk):
    """Keys of row 0 such that head 0's scores are the given numbers (log2, scale 1), nearly: one column carries them."""
    q, k, v, ks, vs, table, lens = args
    n, page, block = int(lens[0]), k.shape[1], k.shape[1] // ks.shape[1]
    q[0, :, 0] = 1.0
    tok = torch.arange(n, device="cuda")
    at, line = table[0].long()[tok // page], tok % page
    raw = k.view(torch.uint8)
    x = torch.as_tensor(weights, dtype=torch.float32, device="cuda") * math.log(2) / ks[at, line // block, 0]
    raw[at, line, 0, 0] = x.clamp(-448, 448).to(F8).view(torch.uint8)


@pytest.mark.parametrize("latent", [True, False])
@pytest.mark.parametrize("kind", ["grow", "fall", "first", "waves", "last"])
def test_weights_far_apart(hsp, latent, kind):
    """Scores that grow or fall along the sequence, a first or last token with nearly all the weight before or behind a
    long tail, tiles in turn far above and below each other."""
    dk, dv = (576, 512) if latent else (64, 64)
    n = 3000
    args = make([n, 40], 16, 1, dk, latent, 64, 21, std=2.0 ** -3, spread=0)
    t = torch.arange(n).float()
    shape_scores(args, {"grow": t / n * 50, "fall": 50 - t / n * 50, "first": torch.where(t == 0, 18.0, 0.0),
                        "last": torch.where(t == n - 1, 24.0, 0.0), "waves": 20 * torch.sin(t / 128)}[kind], dk)
    check(hsp, args, 1.0, dv)


@pytest.mark.parametrize("block", [1, 16])
def test_value_scales_far_apart(hsp, block):
    """Values that are large where the weights are small: the weight that counts is the product of both."""
    args = make([2000], 8, 1, 128, False, 16, 77, block=block, spread=0, std=2.0 ** -3)
    n = 2000
    tok = torch.arange(n, device="cuda")
    shape_scores(args, torch.where(torch.arange(n) % 400 < 200, 14.0, 0.0), 128)
    q, k, v, ks, vs, table, lens = args
    page = table[0].long()[tok // 16]
    big = (tok % 400) >= 200
    vs[page[big], (tok[big] % 16) // block, 0] = 2.0 ** 6
    check(hsp, args, 1.0, 128)


def test_one_token_takes_all_the_weight(hsp):
    q, k, v, ks, vs, table, lens = make([900], 16, 1, 128, False, 16, 2, std=2.0 ** -6, spread=0)
    at = 531
    p, line = int(table[0, at // 16]), at % 16
    ks[p, 0, 0] = 1.0
    k.view(torch.uint8)[p, :, 0] = 0                        # (its block: the others' scores are 0)
    k.view(torch.uint8)[p, line, 0] = (q[0, 3].float() * 4).to(F8).view(torch.uint8)
    out, _ = check(hsp, (q, k, v, ks, vs, table, lens), 1.0, 128)
    assert torch.equal(out[0, 3].float(), v[p, line, 0].float() * vs[p, 0, 0])


def test_heads_of_unlike_size(hsp):
    """Each head's queries have their own unit: a large head takes nothing from a small one."""
    args = list(make([300], 20, 1, 576, True, 64, 4, spread=0, std=2.0 ** -4))
    args[0] = (args[0].float() * (2.0 ** torch.linspace(-60, 3, 20, device="cuda"))[None, :, None]).to(BF)
    check(hsp, args, 0.3, 512)
    args[0] = args[0] * 2.0 ** -60
    check(hsp, args, 0.3, 512)                              # scores of nothing: the mean of the values
    args[0] = torch.zeros_like(args[0])
    check(hsp, args, 0.3, 512)


def test_infinite_and_nan_inputs_stay_where_they_are(hsp):
    """NaN or an infinity in one query head: the other heads are as before.  A NaN code of a token: its row is NaN."""
    args = list(make([200], 16, 1, 576, True, 64, 4))
    clean = hsp.paged_attention_q8(*args, 0.07)
    keep = [h for h in range(16) if h != 5]
    for bad in (float("nan"), float("inf")):
        args[0] = args[0].clone()
        args[0][0, 5, 7] = bad
        out = hsp.paged_attention_q8(*args, 0.07)
        assert torch.equal(out[0, keep], clean[0, keep]) and torch.isnan(out[0, 5]).all()
    args = list(make([200, 300], 16, 1, 128, False, 64, 4))
    clean = hsp.paged_attention_q8(*args, 0.07)
    args[2].view(torch.uint8)[args[5][0, 1].long(), 3, 0, 11] = NAN8
    out = hsp.paged_attention_q8(*args, 0.07)
    assert torch.isnan(out[0, :, 11]).all() and torch.equal(out[1], clean[1])
    assert torch.equal(out[0, :, :11], clean[0, :, :11]) and torch.equal(out[0, :, 12:], clean[0, :, 12:])
    hsp.check_device_error()


def test_scales_of_nothing(hsp):
    """Blocks whose scale is 0: their keys score 0 and their values count for nothing."""
    args = make([100], 4, 1, 64, False, 16, 5)
    q, k, v, ks, vs, table, lens = args
    ks[table[0, 2].long()], vs[table[0, 2].long()] = 0.0, 0.0
    out = hsp.paged_attention_q8(*args, 0.1)
    want = list(args)
    want[4] = vs.clone()
    want[4][table[0, 2].long()] = 2.0 ** -60
    ref, _, tol, _, _ = reference(*want, 0.1, 64)
    assert ((out.double() - ref).abs() <= tol).all()


def test_repeat_graph_and_side_stream_bitwise(hsp):
    lens = [4000, 65, 0, 2500, 1]
    args = make(lens, 16, 1, 576, True, 64, 31)
    first = hsp.paged_attention_q8(*args, 0.07, return_lse=True)
    again = hsp.paged_attention_q8(*args, 0.07, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = hsp.paged_attention_q8(*args, 0.07, return_lse=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    hsp.set_options(pdl=False)
    try:
        assert torch.equal(hsp.paged_attention_q8(*args, 0.07), first[0])
    finally:
        hsp.set_options(pdl=True)
    # captured: new queries, new lengths, the same addresses; two graphs live at once
    q, k, v, ks, vs, table, ln = args
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(hsp.paged_attention_q8(*args, 0.07, return_lse=True))
        graphs.append(g)
    for step, new in enumerate(([4000, 65, 0, 2500, 1], [3999, 1, 0, 64, 0])):
        q.copy_(torch.randn(q.shape, generator=torch.Generator("cuda").manual_seed(step), device="cuda"))
        ln.copy_(torch.tensor(new, dtype=torch.int32))
        want = hsp.paged_attention_q8(*args, 0.07, return_lse=True)
        for g, o in zip(graphs, outs):
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want))
    hsp.check_device_error()


def test_two_streams_at_once(hsp):
    a, b = make([3000, 40], 16, 1, 576, True, 64, 1), make([700] * 9, 8, 2, 128, False, 16, 2)
    wa, wb = hsp.paged_attention_q8(*a, 0.07), hsp.paged_attention_q8(*b, 0.09)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        with torch.cuda.stream(s1):
            x = hsp.paged_attention_q8(*a, 0.07)
        with torch.cuda.stream(s2):
            y = hsp.paged_attention_q8(*b, 0.09)
        got.append((x, y))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in got)


def test_outputs_and_workspace_lie_between_untouched_bytes(hsp):
    for heads, kv, dk, dv in ((5, 1, 512, 512), (70, 1, 576, 512), (12, 2, 128, 128), (3, 3, 64, 64)):
        args = make([1500, 9], heads, kv, dk, dv == 512, 16, 8)
        buf = torch.full((2 * 4096 + 2 * heads * dv,), 7.0, dtype=BF, device="cuda")
        out = buf[4096:4096 + 2 * heads * dv].view(2, heads, dv)
        check(hsp, args, 0.07, dv, out=out)
        assert (buf[:4096] == 7).all() and (buf[-4096:] == 7).all()
        need = hsp.paged_attention_q8_workspace_bytes(2, heads, kv, dk, dv, dv == 512)
        ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        assert torch.equal(hsp.paged_attention_q8(*args, 0.07, workspace=ws[:need]), out)
        assert (ws[need:] == 0x5A).all()


def test_bad_pages_rows_and_lengths_are_reported(hsp):
    import hidden_state_projection_gb300 as m

    def expect(args, **kw):
        out = hsp.paged_attention_q8(*args, 0.07, **kw)
        with pytest.raises(m.ProjError) as ei:
            hsp.check_device_error()
        assert ei.value.status_name == "PROJ_ERR_BAD_INDEX"
        hsp.check_device_error()                            # cleared
        return out

    q, k, v, ks, vs, table, lens = make([200, 100], 16, 1, 576, True, 64, 6)
    good = hsp.paged_attention_q8(q, k, v, ks, vs, table, lens, 0.07)
    for bad in (-1, k.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        out = expect((q, k, v, ks, vs, t, lens))
        assert torch.equal(out[1], good[1])                 # the other sequence is as it was
    for n in (-3, table.shape[1] * 64 + 1):
        ln = lens.clone()
        ln[0] = n
        t = table.clone()
        t[0] = t[0, 0]
        expect((q, k, v, ks, vs, t, ln))
    expect((q, k, v, ks, vs, table, lens), rows=torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
    expect((q, k, v, ks, vs, table, lens), rows=torch.tensor([-1, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(hsp.paged_attention_q8(q, k, v, ks, vs, table, lens, 0.07), good)
    hsp.check_device_error()


@pytest.mark.parametrize("latent", [True, False])
def test_bounded_waits_report_a_timeout(hsp, latent):
    """The test hook leaves the first tile of every CTA unloaded: the waits run out, and the next call is right again."""
    import hidden_state_projection_gb300 as m
    dk, dv = (576, 512) if latent else (128, 128)
    args = make([3000], 16, 1, dk, latent, 64, 12)
    want = hsp.paged_attention_q8(*args, 0.07)
    hsp.set_options(pdl=True, wait_limit_us=20000, skip_stage=0)
    try:
        hsp.paged_attention_q8(*args, 0.07)
        with pytest.raises(m.ProjError) as ei:
            hsp.check_device_error()
        assert ei.value.status_name == "PROJ_ERR_TIMEOUT"
    finally:
        hsp.set_options(pdl=True, wait_limit_us=0, skip_stage=None)
    assert torch.equal(hsp.paged_attention_q8(*args, 0.07), want)
    hsp.check_device_error()


def test_no_sequences(hsp):
    q, k, v, ks, vs, table, lens = make([10], 4, 1, 576, True, 64, 1)
    n = hsp.launch_count()
    assert hsp.paged_attention_q8(q[:0], k, v, ks, vs, table, lens, 0.07).shape == (0, 4, 512)
    assert hsp.launch_count() == n


def test_a_decode_run(hsp):
    """Prompts written in chunks, forked, grown token by token with the pages' calls on codes and scales in one pool of
    bytes, compacted, attended over: the values are those of the new rows within the codes' steps, and the attention is
    that over the values the cache gives back."""
    page, block, kv, d, heads, pages = 32, 16, 2, 128, 8, 64
    g = torch.Generator(device="cuda").manual_seed(8)
    size, nb = page * kv * d, page // block
    pool = torch.zeros(1, pages, 2 * (size + nb * kv * 4), dtype=torch.uint8, device="cuda")
    cut = [size, size, nb * kv * 4, nb * kv * 4]
    kb, vb, ksb, vsb = pool[0].split(cut, -1)
    k, v = kb.unflatten(1, (page, kv, d)).view(F8), vb.unflatten(1, (page, kv, d)).view(F8)
    ks, vs = ksb.view(torch.float32).unflatten(1, (nb, kv)), vsb.view(torch.float32).unflatten(1, (nb, kv))

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    table, lens, refs = torch.full((4, 8), -1, dtype=torch.int32, device="cuda"), ints([0] * 4), ints([0] * pages)
    index = (table, lens, refs)
    hist = {r: ([], []) for r in range(4)}

    def write(rows, pos):
        kn = (torch.randn(len(rows), kv, d, generator=g, device="cuda") * 2).to(BF)
        vn = (torch.randn(len(rows), kv, d, generator=g, device="cuda") * 0.3).to(BF)
        hsp.cache_append_q8(kn, vn, k, v, ks, vs, table, lens, rows=ints(rows), positions=ints(pos), ref_counts=refs)
        for i, r in enumerate(rows):
            assert len(hist[r][0]) == pos[i]
            hist[r][0].append(kn[i])
            hist[r][1].append(vn[i])

    def grow(rows, new):
        status = hsp.cache_resize(*index, ints(rows), ints(new), page, [pool])
        assert not status.any()

    grow([0, 2], [100, 41])
    write([0] * 70 + [2] * 41, list(range(70)) + list(range(41)))          # a chunk, then the rest
    write([0] * 30, list(range(70, 100)))
    assert not hsp.cache_fork(*index, ints([0]), ints([1]), page).any()
    hist[1] = (list(hist[0][0]), list(hist[0][1]))
    for step in range(20):                                                  # the children part on a page of their own
        rows = [0, 1, 2]
        now = lens.tolist()
        grow(rows, [now[r] + 1 for r in rows])
        write(rows, [now[r] for r in rows])
    assert int(hsp.cache_compact(*index, page, [pool])) == int((refs > 0).sum())
    hsp.check_device_error()
    for r in range(3):
        n = int(lens[r])
        kr, vr = hsp.cache_read_q8(k, v, ks, vs, table, lens, rows=ints([r] * n), positions=ints(list(range(n))))
        for got, want, sc in ((kr, hist[r][0], ks), (vr, hist[r][1], vs)):
            x = torch.stack(want).double()
            tok = torch.arange(n, device="cuda")
            s = sc[table[r].long()[tok // page], tok % page // block].double()[..., None]
            # a code is half a step off, 2^-4 of the value or 2^-10 of the scale; each time the scale grew (at most three
            # times here: values within 2^3 of each other) half of the smallest code of a lower scale more
            assert ((got.double() - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -9 * s).all()
    q = torch.randn(4, heads, d, generator=g, device="cuda").to(BF)
    check(hsp, (q, k, v, ks, vs, table, lens), d ** -0.5, d)
