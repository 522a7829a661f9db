"""The softmax's sum of proj_paged_attention_q8: every token counts in it with its probability, whatever the scale of its values.

The weight that is multiplied with the values, w_t = p_t vs_t, is held in two 8-bit pieces; the sum that the result is divided by
is that of the probabilities.  So the bounds of the two differ (derived before the first run; the rest as in
test_attention_q8_gpu.py, rel: what a score, and so a probability, is off by):
  * numerator: w_t is off by 2^-7 + 2^-11 (fp16 on the way) of itself while it is at least 2^-6 in units in which the largest w of every
    128-token tile is at least 2^-4 and the row's at least 2^3, and by 2^-13 of such a unit below: 2^-9 of the tile's largest and
    2^-16 of the row's, the smaller of the two.  A reference point stops 30 below its highest: 2^-43 of the row's largest more;
  * sum: p_t is off by 2^-7 + 2^-11 of itself at most (nothing but rel where the unrounded one is summed): there is no 1 / vs in it.
    A token whose w_t is below 2^-120 of the row's largest may be missing;
  * a score is held in log2 units with the values' scale: rel has 2^-22 of log2 vs too.
The 2-norm of all errors, at random signs: sum_t (dw_t |vc_t| + |o| dp_t)^2, and the rounding to bf16 likewise.
"""
import math

import pytest
import torch

from test_attention_q8_gpu import BF, F8, held, hsp, make  # noqa: F401  (hsp: the fixture)

pytestmark = pytest.mark.gpu
R = 2.0 ** -7 + 2.0 ** -11


def reference(q, k, v, ks, vs, table, lens, scale, dv):
    """(out, lse, bound of out, bound of lse, the squares' bound, sum p |v|) in 64 bits."""
    B, H, dk = q.shape
    page, kv = k.shape[1], k.shape[2]
    G = H // kv
    out = torch.zeros(B, H, dv, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    tol, square, size, ltol = torch.zeros_like(out), torch.zeros_like(out), torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            continue
        ids = table[b, : -(-n // page)].long()
        kc, kscale = held(k, ks, ids, n)
        vc, vscale = (kc[..., :dv], kscale) if v is None else held(v, vs, ids, n)
        for h in range(kv):
            at = slice(h * G, (h + 1) * G)
            qq, kk = q[b, at].double(), kc[:, h] * kscale[:, h, None]
            c, s = vc[:, h], vscale[:, h]
            x = qq @ kk.T * scale
            p = torch.softmax(x, -1)
            out[b, at] = o = p @ (c * s[:, None])
            size[b, at] = a = p @ (c * s[:, None]).abs()
            lse[b, at] = torch.logsumexp(x, -1)
            rel = dk * 2.0 ** -24 * float((qq.abs() @ kk.abs().T).max()) * abs(scale)
            rel += float(qq.abs().max() * kk.abs().sum(-1).max()) * abs(scale) * 2.0 ** -21.8
            rel += 2.0 ** -22 * (1 + 1.5 * float(x.abs().max()) + float(s.log2().abs().max()))
            w = p * s
            tile = torch.nn.functional.pad(w, (0, -n % 128)).unflatten(-1, (-1, 128)).amax(-1)
            row = w.amax(-1, keepdim=True)
            low = torch.minimum(tile * 2.0 ** -9, row * 2.0 ** -16) + row * 2.0 ** -43
            dp = R * p + p * (w < row * 2.0 ** -120)
            dw = R * w + low.repeat_interleave(128, -1)[:, :n]
            slack = 2 * rel + (2 * n + 64) * 2.0 ** -24
            tol[b, at] = dw @ c.abs() + (dp.sum(-1, keepdim=True) + 2.0 ** -8) * o.abs() + (a + o.abs()) * slack
            square[b, at] = dw ** 2 @ c ** 2 + 2 * o.abs() * ((dw * dp) @ c.abs()) + o ** 2 * (dp ** 2).sum(-1, keepdim=True)
            square[b, at] += ((2.0 ** -8 + slack) * o.abs() + slack * a) ** 2
            ltol[b, at] = rel + (n + 64) * 2.0 ** -24 + lse[b, at].abs() * 2.0 ** -22
    return out, lse, tol, ltol, square, size


def check(m, args, scale, dv):
    out, lse = m.paged_attention_q8(*args, scale, v_dim=dv, return_lse=True)
    m.check_device_error()
    ref, rlse, tol, ltol, square, size = reference(*args, scale, dv)
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), f"out off by {float((err - tol).max()):.3e}, {int((err > tol).sum())} of {err.numel()}"
    for h in range(out.shape[1]):                           # (a head with large values hides no other)
        norm, most = float(torch.linalg.norm(err[:, h])), float(square[:, h].sum().sqrt())
        assert norm <= most, f"2-norm of head {h}'s errors {norm:.3e}, {most:.3e} at most"
        assert most <= 2.0 ** -5 * float(torch.linalg.norm(size[:, h])), "the bound would hide a token"
    lerr = (lse.double() - rlse).abs().nan_to_num(0.0)      # (two infinities: no sequence)
    assert (lerr <= ltol).all(), f"lse off by {float((lerr - ltol).max()):.3e}"
    return out, lse


def places(args, tok, block):
    table, page = args[5], args[1].shape[1]
    return table[0].long()[tok // page], tok % page, tok % page // block


def set_scores(args, tok, bits, block):
    """Keys of row 0's tokens `tok` such that every head's scores (scale 1) are `bits` log2 units above those of other tokens, nearly:
    column 0, which is 0 elsewhere, and queries of 64 there."""
    q, k, _, ks = args[:4]
    q[:, :, 0] = 64.0
    page, line, blk = places(args, torch.arange(int(args[6][0]), device="cuda"), block)
    k.view(torch.uint8)[page, line, :, 0] = 0
    page, line, blk = places(args, tok, block)
    x = torch.as_tensor(bits, device="cuda", dtype=torch.float32).expand(len(tok))[:, None] * math.log(2) / 64 / ks[page, blk]
    assert float(x.abs().max()) <= 448
    k.view(torch.uint8)[page, line, :, 0] = x.to(F8).view(torch.uint8)


def set_values(args, tok, block, exponent, zero=False):
    """Value scales 2^exponent of row 0's tokens `tok` (whole blocks), their codes 0 where zero."""
    k, v, ks, vs = args[1:5]
    codes, scales = (k, ks) if v is None else (v, vs)
    page, line, blk = places(args, tok, block)
    scales[page, blk] = 2.0 ** torch.as_tensor(exponent, device="cuda").float().expand(len(tok))[:, None]
    if zero:
        codes.view(torch.uint8)[page, line] = 0


KINDS = [(True, 576, 512, 16, 1), (True, 512, 512, 70, 1), (False, 64, 64, 8, 4), (False, 128, 128, 36, 2), (False, 128, 128, 60, 1)]


@pytest.mark.parametrize("latent,dk,dv,heads,kv", KINDS)
@pytest.mark.parametrize("first", [True, False])
def test_two_tokens_one_without_values(hsp, latent, dk, dv, heads, kv, first):
    """Equal scores, one token's values zero, as the append writes them: half of the other's values."""
    k = torch.zeros(4, 16, kv, dk, dtype=torch.uint8, device="cuda").view(F8)
    v = None if latent else torch.zeros(4, 16, kv, dv, dtype=torch.uint8, device="cuda").view(F8)
    ks = torch.zeros(4, 16, kv, device="cuda")
    vs = None if latent else torch.zeros_like(ks)
    table, lens = torch.tensor([[2, 1]], dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda")
    new = torch.randn(2, kv, dk, device="cuda").to(BF)
    new[0 if first else 1] = 0
    pos = torch.arange(2, dtype=torch.int32, device="cuda")
    hsp.cache_append_q8(new, None if latent else new, k, v, ks, vs, table, lens, rows=torch.zeros_like(pos), positions=pos)
    q = torch.zeros(1, heads, dk, device="cuda").to(BF)
    out, _ = check(hsp, (q, k, v, ks, vs, table, lens), 1.0, dv)
    x = hsp.cache_read_q8(k, v, ks, vs, table, lens, rows=torch.zeros_like(pos), positions=pos)[0 if latent else 1]
    want = x[1 if first else 0, :, :dv].float().repeat_interleave(heads // kv, 0) / 2
    assert ((out[0].float() - want).abs() <= 2.0 ** -7 * want.abs()).all()


@pytest.mark.parametrize("latent,dk,dv,heads,kv", KINDS)
@pytest.mark.parametrize("n", [128, 300, 5000])
@pytest.mark.parametrize("where", ["first", "middle", "last", "tile", "in turn"])
@pytest.mark.parametrize("block", [1, 16])
def test_zero_values_with_half_the_weight(hsp, latent, dk, dv, heads, kv, n, where, block):
    """Tokens of zero values among others: a quarter or half of all, and a block of 16 with about as much weight as the rest."""
    args = make([n, 33], heads, kv, dk, latent, 16, 50 + n, block=block, std=2.0 ** -4)
    t = torch.arange(n, device="cuda")
    half = n // 2 // 16 * 16
    chosen = {"first": t < half, "middle": (t >= half // 32 * 16) & (t < half // 32 * 16 + half), "last": t >= n // 16 * 16 - half,
              "tile": t // 128 % 2 == 0 if n > 128 else t < 64, "in turn": t // 16 % 2 == 1}[where]
    if n == 5000 and where != "tile":                       # a whole part of such tokens, more than one where they are all in one place
        assert int(chosen.sum()) > 2000
    set_values(args, t[chosen], block, -60, zero=True)      # (of a latent cache the keys too: scores of 0)
    check(hsp, args, 0.05, dv)
    if latent:
        return
    args = make([n, 33], heads, kv, dk, latent, 16, 51 + n, block=block, std=2.0 ** -3, spread=0)
    one = t[chosen][-16:] // 16 * 16 + torch.arange(16, device="cuda")
    one = one[one < n]
    set_scores(args, one, max(1.0, math.log2(n / 16)), block)
    set_values(args, one, block, -60, zero=True)
    check(hsp, args, 1.0, dv)


@pytest.mark.parametrize("d,heads,kv", [(64, 8, 4), (128, 36, 2), (128, 60, 1)])
@pytest.mark.parametrize("n", [100, 3000])
@pytest.mark.parametrize("bits", [6, 12, 16, 20, 24, 30, 50])
def test_the_heaviest_token_has_small_values(hsp, d, heads, kv, n, bits):
    """Nine tenths of the weight on a token whose values are 2^bits smaller than the others'."""
    for at in (0, n // 2, n - 1):
        args = make([n], heads, kv, d, False, 16, 80 + bits, block=1, std=2.0 ** -3, spread=0)
        one = torch.tensor([at], device="cuda")
        set_scores(args, one, math.log2(9 * n), 1)
        set_values(args, one, 1, -9 - bits)
        check(hsp, args, 1.0, d)


@pytest.mark.parametrize("d,heads,kv", [(64, 8, 4), (128, 36, 2), (128, 60, 1)])
@pytest.mark.parametrize("n", [200, 4000])
@pytest.mark.parametrize("spread", [5, 10, 25, 48, 60])
def test_value_scales_of_the_whole_range(hsp, d, heads, kv, n, spread):
    args = make([n], heads, kv, d, False, 16, 90 + spread, block=1, std=2.0 ** -3, spread=0)
    t = torch.arange(n, device="cuda")
    e = torch.randint(-spread, spread + 1, (n,), generator=torch.Generator("cuda").manual_seed(spread), device="cuda")
    set_values(args, t, 1, e)
    check(hsp, args, 0.3, d)


@pytest.mark.parametrize("d,heads,kv", [(64, 8, 4), (128, 60, 1)])
@pytest.mark.parametrize("n", [200, 4000])
@pytest.mark.parametrize("below", [0, 3, 6, 8])
def test_one_scale_at_the_top_all_others_at_the_bottom(hsp, d, heads, kv, n, below):
    """Values of nothing beside values of 2^52: weights 2^-112 of the largest, nearly, with probabilities of 2^-8 and more of its."""
    for at in (0, n // 2, n - 1):
        args = make([n], heads, kv, d, False, 16, 70 + below, block=1, std=2.0 ** -5, spread=0)
        set_values(args, torch.arange(n, device="cuda"), 1, -60)
        one = torch.tensor([at], device="cuda")
        set_scores(args, one, below, 1)
        set_values(args, one, 1, 52 - below)
        check(hsp, args, 1.0, d)


@pytest.mark.parametrize("n", [300, 4000])
def test_out_agrees_with_lse(hsp, n):
    """Values of one under scales from 2^-8 to 2^6, every third block zero: out is the probability of the tokens that have values."""
    args = make([n, n], 8, 2, 128, False, 16, 33, block=4, std=2.0 ** -4)
    q, k, v, ks, vs, table, lens = args
    q[1] = q[0]
    t = torch.arange(n, device="cuda")
    page, line = table[0].long()[t // 16], t % 16
    e = (t // 4 * 7 % 15 - 8).float()
    v.view(torch.uint8)[page, line] = (2.0 ** -e).to(F8).view(torch.uint8)[:, None, None]
    vs[page, line // 4] = (2.0 ** e)[:, None]
    zero = t // 4 % 3 == 1
    set_values(args, t[zero], 4, -60, zero=True)
    # row 1: the tokens with values alone
    keep = t[~zero]
    lens[1] = len(keep)
    to = torch.arange(len(keep), device="cuda")
    p1, l1 = table[1].long()[to // 16], to % 16
    for pool, scales in ((k, ks), (v, vs)):
        pool.view(torch.uint8)[p1, l1] = pool.view(torch.uint8)[page[keep], line[keep]]
    assert bool((zero.view(-1, 4).all(1) | ~zero.view(-1, 4).any(1)).all())   # (whole blocks move)
    for scales in (ks, vs):
        scales[p1, l1 // 4] = scales[page[keep], line[keep] // 4]
    out, lse = check(hsp, args, 0.1, 128)
    want = torch.exp(lse[0] - lse[1]).reciprocal()
    # p in two pieces in the numerator, and in the sum: 2 (2^-7 + 2^-11), bf16 2^-8
    assert ((out[0].float() - want[:, None]).abs() <= (2 * R + 2.0 ** -8) * want[:, None]).all()
    assert ((out[1].float() - 1).abs() <= 2 * R + 2.0 ** -8).all()


@pytest.mark.parametrize("latent,dk,dv,heads,kv", KINDS)
@pytest.mark.parametrize("kind", ["grow", "fall", "first", "waves", "last", "steps"])
def test_scores_far_apart(hsp, latent, dk, dv, heads, kv, kind):
    """Reference points that follow the tiles up and down: scores that grow or fall by 50 log2 units along the sequence, a first or last
    token with nearly all the weight, tiles in turn far above and below each other."""
    n = 3000
    args = make([n, 40], heads, kv, dk, latent, 64, 21, std=2.0 ** -3, spread=0)
    t = torch.arange(n, device="cuda").float()
    bits = {"grow": t / n * 50, "fall": 50 - t / n * 50, "first": (t == 0) * 18.0, "last": (t == n - 1) * 24.0,
            "waves": 20 * torch.sin(t / 128), "steps": (t // 128 * 37 % 61)}[kind]
    set_scores(args, t.long(), bits, 16)
    check(hsp, args, 1.0, dv)
