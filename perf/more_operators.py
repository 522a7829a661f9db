"""The operators of the paged cache held in 8 bits: their cases, their plain forms and their definition.

The cache holds e4m3 codes and one fp32 scale for each block of `block` tokens of a page and each key head: a value
is code * scale.  cache_append_q8 quantises the new tokens as it writes them (after the rotary turn of their keys),
cache_read_q8 gives tokens back in bf16, paged_attention_q8 is the attention of one new token per sequence.

A written block's scale is the smallest power of two with amax / scale <= 448 over its new tokens (from 2^-60 to
2^60), and not below the scale of the tokens that the block holds in front of them; where it grows, those tokens'
codes are rounded to the new scale.

Shapes: a latent cache has one key head of 576 columns (512 latent + 64 rotary: the kv_a projection) or of 512 (the
wkv projection), whose first 512 columns are the values too; a grouped cache has its own key and value heads of 64 or
128 columns.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn


# ---- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # one user, a short prompt, a tensor-parallel share of the heads: the latency of a call
        dict(name="attn_latent_short", op="attn", batch=1, heads=16, kv_heads=1, dk=576, dv=512, latent=True,
             max_len=77, page=64, block=16, ragged=False),
        # a serving batch of ragged lengths, all the heads of a latent-attention layer on one GPU
        dict(name="attn_latent_batch", op="attn", batch=48, heads=128, kv_heads=1, dk=576, dv=512, latent=True,
             max_len=6001, page=64, block=64, ragged=True),
        # one sequence of a long document, half the heads: the split over the cache's length
        dict(name="attn_latent_long", op="attn", batch=1, heads=64, kv_heads=1, dk=512, dv=512, latent=True,
             max_len=131071, page=64, block=32, ragged=False),
        # grouped heads with small pages, ragged, a sequence without tokens among them
        dict(name="attn_grouped_batch", op="attn", batch=61, heads=32, kv_heads=8, dk=128, dv=128, latent=False,
             max_len=4099, page=16, block=16, ragged=True),
        # narrow heads, an odd group, a scale of its own for every token
        dict(name="attn_narrow_batch", op="attn", batch=13, heads=28, kv_heads=4, dk=64, dv=64, latent=False,
             max_len=2333, page=32, block=1, ragged=True),
        # the new tokens of a decode step: eight latent rows and their queries
        dict(name="append_latent_step", op="append", tokens=8, heads=16, kv_heads=1, dk=576, dv=512, latent=True,
             page=64, block=64, rot=64, interleaved=True),
        # a chunk of a prompt, grouped heads, rotary over the whole head
        dict(name="append_grouped_chunk", op="append", tokens=2047, heads=32, kv_heads=8, dk=128, dv=128, latent=False,
             page=16, block=16, rot=128, interleaved=False),
        # a chunk of latent rows, blocks of half a page
        dict(name="append_latent_chunk", op="append", tokens=1501, heads=16, kv_heads=1, dk=576, dv=512, latent=True,
             page=64, block=32, rot=64, interleaved=True),
        # a few tokens handed to a kernel that wants bf16
        dict(name="read_few", op="read", tokens=77, kv_heads=1, dk=576, dv=512, latent=True, page=64, block=16),
        # a long shared prefix, latent
        dict(name="read_latent_prefix", op="read", tokens=16001, kv_heads=1, dk=576, dv=512, latent=True, page=64, block=64),
        # the prefixes of a batch, grouped heads
        dict(name="read_grouped_prefix", op="read", tokens=40009, kv_heads=8, dk=128, dv=128, latent=False, page=16, block=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "read"])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (1, 4, 16, 32, 64, 128) if b <= page])
    c = dict(op=op, page=page, block=block)
    if op == "attn":
        if rng.random() < 0.6:
            heads, kv, dk, dv, latent = rng.choice([1, 7, 8, 16, 20, 32, 64, 96, 128]), 1, rng.choice([576, 512]), 512, True
        else:
            dk = rng.choice([64, 128])
            kv = rng.choice([1, 2, 5, 8])
            heads, dv, latent = kv * rng.choice([1, 3, 4, 8, 16]), dk, False
        batch = _log(rng, 1, 64)
        most = 131071 if batch == 1 else max(64, min(65537, 380000 // (batch * (1 if latent else max(1, kv // 2)))))
        if latent:
            most = min(most, max(64, 131071 * 128 // (heads * batch)))
        return dict(c, batch=batch, heads=heads, kv_heads=kv, dk=dk, dv=dv, latent=latent, max_len=_log(rng, 1, most),
                    ragged=rng.random() < 0.7)
    latent = rng.random() < 0.5
    if latent:
        dk, dv, kv = rng.choice([576, 512]), 512, 1
    else:
        dk = rng.choice([64, 128])
        dv, kv = dk, rng.choice([1, 2, 5, 8])
    c.update(kv_heads=kv, dk=dk, dv=dv, latent=latent)
    if op == "read":
        return dict(c, tokens=_log(rng, 1, 40009))
    return dict(c, tokens=_log(rng, 1, 2047), heads=rng.choice([1, 8, 16, 20, 64]) if latent else kv * rng.choice([1, 4]),
                rot=64 if latent else rng.choice([32, dk]), interleaved=rng.random() < 0.5)


def _lens(case):
    """The lengths of a case's sequences: the case's alone, so that its work is known without a seed."""
    n, most = case["batch"], case["max_len"]
    if not case["ragged"]:
        return [most] * n
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    got = [max(1, min(most, int(most * r.uniform(0.02, 1.0)))) for _ in range(n)]
    got[0] = most
    if n > 2:
        got[n // 2] = 0
    return got


# ---- inputs -----------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _table(g, counts, width, num_pages):
    """A block table whose rows hold counts[i] pages each, all different, in no order; -1 elsewhere."""
    ids = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    c = torch.tensor(counts, dtype=torch.int64, device=DEV)
    first = torch.cumsum(c, 0) - c
    j = torch.arange(width, device=DEV)
    at = (first[:, None] + j[None, :]).clamp(max=num_pages - 1)
    return torch.where(j[None, :] < c[:, None], ids[at], torch.full_like(ids[at], -1)).contiguous()


def _pages(g, pages, case, dim):
    """Codes and scales of a cache that holds something: values of about one, blocks of unlike scales."""
    scales = 2.0 ** torch.randint(-7, -4, (pages, case["page"] // case["block"], case["kv_heads"]), generator=g, device=DEV).float()
    x = torch.randn(pages, case["page"], case["kv_heads"], dim, generator=g, device=DEV)
    x /= scales.repeat_interleave(case["block"], 1)[..., None]
    return x.clamp_(-448, 448).to(F8), scales


def prepare(case, seed):
    g = _gen(seed)
    op, page = case["op"], case["page"]
    s = dict(case=case)
    if op == "attn":
        lens = _lens(case)
        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + 3
        s["table"] = _table(g, counts, max(counts) + 1, pages)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = _normal(g, case["batch"], case["heads"], case["dk"])
        s["scale"] = (192 if case["latent"] else case["dk"]) ** -0.5
    else:
        # sequences of up to 512 tokens of the call each, at far positions of their rows
        n = case["tokens"]
        seqs = max(1, -(-n // 512)) if n > 64 else n
        per = -(-n // seqs)
        start = torch.randint(0, 3000, (seqs,), generator=g, device=DEV)
        token = torch.arange(n, device=DEV)
        s["rows"] = (token // per).to(torch.int32)
        s["pos"] = (start[token // per] + token % per).to(torch.int32)
        width = -(-(3000 + per) // page)
        pages = seqs * width + 5
        s["table"] = _table(g, [width] * seqs, width, pages)
        s["lens"] = (start + per).to(torch.int32)
    s["k"], s["ks"] = _pages(g, pages, case, case["dk"])
    s["v"], s["vs"] = (None, None) if case["latent"] else _pages(g, pages, case, case["dv"])
    if op == "read":
        s["k_out"] = torch.zeros(case["tokens"], case["kv_heads"], case["dk"], dtype=torch.bfloat16, device=DEV)
        s["v_out"] = None if case["latent"] else torch.zeros_like(s["k_out"])
    if op == "append":
        # tokens of unlike size, so that blocks grow
        size = torch.exp(torch.randn(n, 1, 1, generator=g, device=DEV) * 0.7)
        s["k_new"] = (torch.randn(n, case["kv_heads"], case["dk"], generator=g, device=DEV) * size).to(torch.bfloat16)
        s["v_new"] = None if case["latent"] else (torch.randn(n, case["kv_heads"], case["dv"], generator=g, device=DEV) * size).to(torch.bfloat16)
        s["q"] = _normal(g, n, case["heads"], case["dk"])
        s["q_out"] = torch.empty_like(s["q"])
        half = case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        ang = torch.arange(4096, dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32).contiguous()
    return s


# ---- one pass ---------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import hidden_state_projection_gb300 as proj
    if op == "attn":
        if own:
            out, lse = proj.paged_attention_q8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"], s["scale"],
                                               v_dim=case["dv"], return_lse=True)
        else:
            out, lse = _attention(s, case["dv"])
        return {"out": out, "lse": lse}
    if op == "read":
        if own:
            k, v = proj.cache_read_q8(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"], rows=s["rows"],
                                      positions=s["pos"], k_out=s["k_out"], v_out=s["v_out"])
        else:
            at, off = _places(s)
            k = _values(s["k"], s["ks"], at, off).to(torch.bfloat16)
            v = None if s["v"] is None else _values(s["v"], s["vs"], at, off).to(torch.bfloat16)
        return {"k": k, "v": v}
    if own:
        proj.cache_append_q8(s["k_new"], s["v_new"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"], rows=s["rows"],
                             positions=s["pos"], cos_sin=s["cos_sin"], interleaved=case["interleaved"], q=s["q"],
                             q_out=s["q_out"])
    else:
        _append(s)
    return {"q": s["q_out"], "k": s["k"], "k_scales": s["ks"], "v": s["v"], "v_scales": s["vs"]}


def _values(codes, scales, page, line):
    """What the cache holds at lines `line` of pages `page`, in 32 bits."""
    block = codes.shape[1] // scales.shape[1]
    c = codes.view(torch.uint8)[page, line].view(F8).float()
    return c * scales[page, line // block][..., None]


def _places(s):
    page = s["k"].shape[1]
    at = s["table"][s["rows"].long(), (s["pos"] // page).long()].long()
    return at, (s["pos"] % page).long()


def _attention(s, dv):
    q, k, v, table, lens = s["q"], s["k"], s["v"], s["table"], s["lens"]
    B, H, dk = q.shape
    page, kv = k.shape[1], k.shape[2]
    most = table.shape[1] * page
    t = torch.arange(most, device=q.device)
    at = table.long().clamp(min=0)[:, t // page]                             # [B, T]
    seen = t[None, :] < lens[:, None]
    qf = q.float().view(B, kv, H // kv, dk)
    kf = _values(k, s["ks"], at, (t % page)[None, :].expand(B, -1)).permute(0, 2, 1, 3)      # [B, kv, T, dk]
    vf = kf[..., :dv] if v is None else _values(v, s["vs"], at, (t % page)[None, :].expand(B, -1)).permute(0, 2, 1, 3)
    sc = torch.matmul(qf, kf.transpose(2, 3)) * s["scale"]                   # [B, kv, G, T]
    sc = sc.masked_fill(~seen[:, None, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m.clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    vf = vf.masked_fill(~seen[:, None, :, None], 0.0)
    o = torch.matmul(p, vf) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total)).view(B, H)
    return o.reshape(B, H, dv).to(q.dtype), lse


def _turn(x, cs, rot, interleaved):
    """The last rot columns of x [n, heads, dim] turned by the angles whose cosines and sines cs [n, rot] holds."""
    a, y = x[..., : x.shape[-1] - rot], x[..., x.shape[-1] - rot:]
    half = rot // 2
    c, sn = cs[:, None, :half], cs[:, None, half:]
    if interleaved:
        u, w = y[..., 0::2], y[..., 1::2]
        y = torch.stack([u * c - w * sn, u * sn + w * c], -1).flatten(-2)
    else:
        u, w = y[..., :half], y[..., half:]
        y = torch.cat([u * c - w * sn, u * sn + w * c], -1)
    return torch.cat([a, y], -1)


def _two_to(e):
    """2^e in 64 bits, from its bits (a device's pow may be off by its last one)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x rounded to the nearest e4m3 value (ties to the even code), at most 448; x in 64 bits, where no value near a
    border changes sides."""
    _, e = torch.frexp(x)                                                    # |x| in [2^(e-1), 2^e)
    step = _two_to((e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _quantise(x, codes, scales, page, line):
    """The rows x [n, heads, dim] (64 bits) into lines `line` of pages `page`."""
    per = codes.shape[1] // scales.shape[1]
    raw = codes.view(torch.uint8)
    blk = line // per
    ids, group = torch.unique(page * scales.shape[1] + blk, return_inverse=True)     # the blocks that are written
    p, b = ids // scales.shape[1], ids % scales.shape[1]
    n, (tokens, heads, _) = ids.shape[0], x.shape
    m, e = torch.frexp(x.abs().amax(-1).clamp(min=2.0 ** -60) / 448)         # a token's and head's exponent
    need = _two_to((e - (m == 0.5).int()).clamp(-60, 60))
    new = torch.zeros(n, heads, dtype=torch.float64, device=x.device)
    new.scatter_reduce_(0, group[:, None].expand(-1, heads), need, "amax")
    first = torch.full((n,), per, dtype=torch.int64, device=x.device)
    first.scatter_reduce_(0, group, line % per, "amin")
    old = scales[p, b].double()
    now = torch.where((first > 0)[:, None], torch.maximum(old, new), new)
    # the tokens in front of the first new one
    lines = (b * per)[:, None] + torch.arange(per, device=x.device)[None, :]
    kept = raw[p[:, None], lines].view(F8).double()
    moved = _e4m3(kept * (old / now)[:, None, :, None])
    front = torch.arange(per, device=x.device)[None, :] < first[:, None]
    raw[p[:, None], lines] = torch.where(front[..., None, None], moved, kept).to(torch.float32).to(F8).view(torch.uint8)
    raw[page, line] = _e4m3(x / now[group][..., None]).to(torch.float32).to(F8).view(torch.uint8)
    scales[p, b] = now.float()


def _append(s):
    case = s["case"]
    at, off = _places(s)
    cs = s["cos_sin"][s["pos"].long()]
    _quantise(_turn(s["k_new"].double(), cs.double(), case["rot"], case["interleaved"]), s["k"], s["ks"], at, off)
    if s["v"] is not None:
        _quantise(s["v_new"].double(), s["v"], s["vs"], at, off)
    s["q_out"].copy_(_turn(s["q"].float(), cs, case["rot"], case["interleaved"]).to(torch.bfloat16))


# ---- what a pass cannot do without ------------------------------------------------------------------

def work(case):
    op = case["op"]
    row = case["kv_heads"] * (case["dk"] + (0 if case["latent"] else case["dv"]))        # elements of a token
    sides = 1 if case["latent"] else 2
    if op == "attn":
        lens = _lens(case)
        tok = sum(lens)
        scales = 4 * sides * case["kv_heads"] * sum(-(-n // case["block"]) for n in lens)
        io = case["batch"] * case["heads"] * ((case["dk"] + case["dv"]) * 2 + 4)
        return {"bytes": tok * row + scales + io + 4 * sum(-(-n // case["page"]) for n in lens) + 4 * len(lens),
                "flops": 2.0 * tok * case["heads"] * (case["dk"] + case["dv"])}
    n = case["tokens"]
    scales = 4 * sides * case["kv_heads"] * -(-n // case["block"])
    if op == "read":
        return {"bytes": 3 * n * row + scales + 8 * n, "flops": n * row}
    return {"bytes": 3 * n * row + 2 * scales + 2 * n * case["heads"] * case["dk"] * 2 + n * (case["rot"] * 4 + 12),
            "flops": 3.0 * n * (case["heads"] + case["kv_heads"]) * case["rot"] + 2.0 * n * row}


# ---- the definition, in 64 bits ---------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    page, block = case["page"], case["block"]
    if case["op"] == "attn":
        out = torch.zeros(case["batch"], case["heads"], case["dv"], dtype=torch.float64, device=DEV)
        lse = torch.full((case["batch"], case["heads"]), -math.inf, dtype=torch.float64, device=DEV)
        group = case["heads"] // case["kv_heads"]

        def held(codes, scales, ids, n, h):
            x = codes[..., h, :].view(torch.uint8)[ids].view(F8).double()                 # [pages, page, dim]
            y = x.unflatten(1, (page // block, block)) * scales[ids, :, h].double()[:, :, None, None]
            return y.flatten(0, 2)[:n]

        for b, n in enumerate(s["lens"].tolist()):
            if n == 0:
                continue
            ids = s["table"][b, : -(-n // page)].long()
            for h in range(case["kv_heads"]):
                at = slice(h * group, (h + 1) * group)
                keys = held(s["k"], s["ks"], ids, n, h)
                vals = keys[:, : case["dv"]] if s["v"] is None else held(s["v"], s["vs"], ids, n, h)
                x = s["q"][b, at].double() @ keys.T * float(s["scale"])
                lse[b, at] = torch.logsumexp(x, -1)
                out[b, at] = torch.softmax(x, -1) @ vals
        return {"out": out, "lse": lse}
    rows, pos = s["rows"].cpu().numpy(), s["pos"].cpu().numpy()
    at, off = s["table"].cpu().numpy()[rows, pos // page], pos % page

    def numbers(t):
        return None if t is None else t.float().cpu().numpy().astype(np.float64)

    k, ks, v, vs = (numbers(s[x]) for x in ("k", "ks", "v", "vs"))
    if case["op"] == "read":
        return {"k": k[at, off] * ks[at, off // block][..., None],
                "v": None if v is None else v[at, off] * vs[at, off // block][..., None]}
    rot = case["rot"]
    cs = s["cos_sin"].cpu().numpy().astype(np.float64)[pos]
    c, sn = cs[:, None, : rot // 2], cs[:, None, rot // 2:]

    def turned(x):
        y = x.copy()
        i, a = np.arange(rot // 2), x.shape[-1] - rot
        one, two = (a + 2 * i, a + 2 * i + 1) if case["interleaved"] else (a + i, a + rot // 2 + i)
        y[..., one] = x[..., one] * c - x[..., two] * sn
        y[..., two] = x[..., two] * c + x[..., one] * sn
        return y

    # the 127 values that a code without its sign stands for
    grid = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])[:127]

    def nearest(x):
        y = np.abs(x)
        hi = np.searchsorted(grid, y).clip(1, 126)
        low, up = y - grid[hi - 1], grid[hi] - y
        i = np.where((low < up) | ((low == up) & (hi % 2 == 1)), hi - 1, hi)
        return np.copysign(grid[i], x)

    def write(x, codes, scales):
        blocks = {}
        for i in range(len(x)):
            blocks.setdefault((at[i], off[i] // block), []).append(i)
        for (p, b), tokens in blocks.items():
            first = int(off[tokens].min())
            for h in range(x.shape[1]):
                amax, new = np.abs(x[tokens, h]).max(), -60
                while new < 60 and amax > 448 * 2.0 ** new:
                    new += 1
                new = 2.0 ** new
                if first > b * block and scales[p, b, h] >= new:
                    new = scales[p, b, h]
                lines = slice(b * block, first)
                codes[p, lines, h] = nearest(codes[p, lines, h] * scales[p, b, h] / new)
                codes[p, off[tokens], h] = nearest(x[tokens, h] / new)
                scales[p, b, h] = new

    write(turned(numbers(s["k_new"])), k, ks)
    if v is not None:
        write(numbers(s["v_new"]), v, vs)
    return {"q": turned(numbers(s["q"])), "k": k, "k_scales": ks, "v": v, "v_scales": vs}
