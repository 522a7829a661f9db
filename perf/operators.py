"""The operators of the paged key-value cache: their cases, their plain forms and their definition.

A decode step projects the hidden states (fused_gemm), grows the sequences (cache_resize), writes the
new keys and values into their pages (cache_append) and attends over them (paged_attention); beam search
and prefix sharing fork sequences (cache_fork), and a server that shrinks or tidies its cache moves pages
(cache_compact, cache_copy_pages).

Shapes: a latent cache has one key head of 576 columns (512 latent + 64 rotary: the kv_a projection) or of
512 (the wkv projection), whose first 512 columns are the values too; a grouped cache has its own key and
value heads of 64 or 128 columns.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # one user, a short prompt, a tensor-parallel share of the heads: the latency of a call
        dict(name="attn_latent_short", op="attn", batch=1, heads=16, kv_heads=1, dk=576, dv=512, latent=True,
             max_len=77, page=64, ragged=False),
        # a serving batch of ragged lengths, all the heads of a latent-attention layer on one GPU
        dict(name="attn_latent_batch", op="attn", batch=48, heads=128, kv_heads=1, dk=576, dv=512, latent=True,
             max_len=6001, page=64, ragged=True),
        # one sequence of a long document, half the heads: the split over the cache's length
        dict(name="attn_latent_long", op="attn", batch=1, heads=64, kv_heads=1, dk=512, dv=512, latent=True,
             max_len=131071, page=64, ragged=False),
        # grouped heads with small pages, ragged, a sequence without tokens among them
        dict(name="attn_grouped_batch", op="attn", batch=61, heads=32, kv_heads=8, dk=128, dv=128, latent=False,
             max_len=4099, page=16, ragged=True),
        # the new tokens of a decode step: eight latent rows and their queries
        dict(name="append_latent_step", op="append", tokens=8, heads=16, kv_heads=1, dk=576, dv=512, latent=True,
             page=64, rot=64, interleaved=True),
        # a chunk of a prompt, grouped heads, rotary over the whole head
        dict(name="append_grouped_chunk", op="append", tokens=2047, heads=32, kv_heads=8, dk=128, dv=128, latent=False,
             page=16, rot=128, interleaved=False),
        # a beam-search step of one request: the old beams go, the new ones share and grow by a token
        dict(name="beam_small", op="beam", parents=3, children=8, max_len=500, page=16, row_bytes=1152, layers=2,
             pages=512),
        # the same for a batch of requests over long prompts and several layers
        dict(name="beam_large", op="beam", parents=64, children=512, max_len=16383, page=64, row_bytes=1152, layers=4,
             pages=12000),
        # a small cache tidied: what the bookkeeping costs
        dict(name="compact_small", op="compact", rows=9, max_len=300, page=16, row_bytes=1152, layers=1, pages=400),
        # a server's cache after many requests ended: a quarter of the live pages move
        dict(name="compact_large", op="compact", rows=96, max_len=6001, page=64, row_bytes=1152, layers=2, pages=8000),
        # a few pages copied (a prefix handed to another request)
        dict(name="copy_few", op="copy", pairs=3, page=16, row_bytes=1152, layers=1, pages=64),
        # a swap-in of many pages
        dict(name="copy_many", op="copy", pairs=1500, page=64, row_bytes=1152, layers=4, pages=4001),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "beam", "compact", "copy"])
    page = rng.choice([16, 32, 64, 128])
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
        return dict(op=op, batch=batch, heads=heads, kv_heads=kv, dk=dk, dv=dv, latent=latent,
                    max_len=_log(rng, 1, most), page=page, ragged=rng.random() < 0.7)
    if op == "append":
        latent = rng.random() < 0.5
        if latent:
            dk, dv, kv, rot, heads = 576, 512, 1, 64, rng.choice([1, 8, 16, 20, 64, 128])
        else:
            dk = rng.choice([64, 128])
            kv = rng.choice([1, 2, 5, 8])
            dv, rot, heads = dk, rng.choice([32, dk]), kv * rng.choice([1, 4])
        return dict(op=op, tokens=_log(rng, 1, 2047), heads=heads, kv_heads=kv, dk=dk, dv=dv, latent=latent,
                    page=page, rot=rot, interleaved=rng.random() < 0.5)
    row_bytes = rng.choice([1152, 1024, 2048])
    layers = rng.choice([1, 2, 3])
    if op == "beam":
        parents = _log(rng, 1, 32)
        max_len = _log(rng, 20, 8000)
        children = _log(rng, 1, 256)
        pages = parents * -(-max_len // page) + children * 2 + rng.randrange(1, 200)
        return dict(op=op, parents=parents, children=children, max_len=max_len, page=page, row_bytes=row_bytes,
                    layers=layers, pages=pages)
    if op == "compact":
        rows = _log(rng, 1, 64)
        max_len = _log(rng, 20, 4000)
        pages = int(rows * -(-max_len // page) * rng.uniform(1.05, 2.0)) + rng.randrange(1, 50)
        return dict(op=op, rows=rows, max_len=max_len, page=page, row_bytes=row_bytes, layers=layers, pages=pages)
    pairs = _log(rng, 1, 1000)
    return dict(op=op, pairs=pairs, page=page, row_bytes=row_bytes, layers=layers, pages=2 * pairs + rng.randrange(1, 100))


def _lens(case, n, at_least=1):
    """The lengths of a case's n sequences: the case's alone, so that its work is known without a seed."""
    most = case["max_len"]
    if not case.get("ragged", True):
        return [most] * n
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    got = [max(at_least, min(most, int(most * r.uniform(0.02, 1.0)))) for _ in range(n)]
    got[0] = most
    if case["op"] == "attn" and n > 2:
        got[n // 2] = 0
    return got


# ---- inputs -----------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _table(g, counts, width, num_pages):
    """A block table whose rows hold counts[i] pages each, all different, in no order; -1 elsewhere."""
    ids = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    c = torch.tensor(counts, dtype=torch.int64, device=DEV)
    first = torch.cumsum(c, 0) - c
    j = torch.arange(width, device=DEV)
    at = (first[:, None] + j[None, :]).clamp(max=num_pages - 1)
    return torch.where(j[None, :] < c[:, None], ids[at], torch.full_like(ids[at], -1)).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, page = case["op"], case["page"]
    s = dict(case=case)
    if op == "attn":
        lens = _lens(case, case["batch"])
        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + 3
        s["table"] = _table(g, counts, max(counts) + 1, pages)
        s["lens"] = _ints(lens)
        s["q"] = _normal(g, case["batch"], case["heads"], case["dk"])
        s["k"] = _normal(g, pages, page, case["kv_heads"], case["dk"])
        s["v"] = None if case["latent"] else _normal(g, pages, page, case["kv_heads"], case["dv"])
        s["scale"] = (192 if case["latent"] else case["dk"]) ** -0.5
        return s
    if op == "append":
        # sequences of up to 512 new tokens each, at far positions of their rows
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
        s["k"] = _normal(g, pages, page, case["kv_heads"], case["dk"])
        s["v"] = None if case["latent"] else _normal(g, pages, page, case["kv_heads"], case["dv"])
        s["k_new"] = _normal(g, n, case["kv_heads"], case["dk"])
        s["v_new"] = None if case["latent"] else _normal(g, n, case["kv_heads"], case["dv"])
        s["q"] = _normal(g, n, case["heads"], case["dk"])
        s["q_out"] = torch.empty_like(s["q"])
        half = case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        ang = torch.arange(4096, dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32).contiguous()
        return s
    pages, layers = case["pages"], case["layers"]
    s["pool"] = _normal(g, layers, pages, page, case["row_bytes"] // 2)
    if op == "copy":
        ids = torch.randperm(pages, generator=g, device=DEV)[: 2 * case["pairs"]].to(torch.int32).cpu()
        s["src"], s["dst"] = ids[: case["pairs"]].contiguous(), ids[case["pairs"]:].contiguous()
        return s
    if op == "beam":
        P, C = case["parents"], case["children"]
        lens = _lens(case, P)
        counts = [-(-n // page) for n in lens]
        width = max(counts) + 1
        s["table"] = torch.cat([_table(g, counts, width, pages),
                                torch.full((C, width), -1, dtype=torch.int32, device=DEV)])
        s["lens"] = _ints(lens + [0] * C)
        s["parents"] = torch.randint(0, P, (C,), generator=g, device=DEV).to(torch.int32)
        s["children"] = (P + torch.randperm(C, generator=g, device=DEV)).to(torch.int32)
        s["zero"] = torch.zeros(C, dtype=torch.int32, device=DEV)
        s["next"] = s["lens"][s["parents"].long()] + 1
    else:
        R = case["rows"]
        counts = [-(-n // page) for n in _lens(case, R)]
        s["table0"] = _table(g, counts, max(counts) + 1, pages)
        s["table"] = s["table0"].clone()
        s["lens"] = _ints(_lens(case, R))
        s["live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    used = s["table"][s["table"] >= 0].long()
    s["refs"] = torch.bincount(used, minlength=pages).to(torch.int32)
    s["refs0"] = s["refs"].clone()
    return s


# ---- one pass ---------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import hidden_state_projection_gb300 as proj
    if op == "attn":
        if own:
            out, lse = proj.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"],
                                            v_dim=case["dv"], return_lse=True)
        else:
            out, lse = _attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"], case["dv"])
        return {"out": out, "lse": lse}
    if op == "append":
        if own:
            proj.cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], rows=s["rows"],
                              positions=s["pos"], cos_sin=s["cos_sin"], interleaved=case["interleaved"], q=s["q"],
                              q_out=s["q_out"])
        else:
            _append(s, case["rot"], case["interleaved"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if op == "copy":
        if own:
            proj.cache_copy_pages([s["pool"]], s["src"], s["dst"])
        else:
            s["pool"][:, s["dst"].to(DEV).long()] = s["pool"][:, s["src"].to(DEV).long()]
        return {"pool": s["pool"].view(torch.int16)}
    if op == "beam":
        # the beams of the last step go, the new ones share their parents' pages, and each grows by one
        # token, which gives it a last page of its own
        a = (s["table"], s["lens"], s["refs"])
        resize, fork = (proj.cache_resize, proj.cache_fork) if own else (_resize, _fork)
        gone = resize(*a, s["children"], s["zero"], case["page"], [s["pool"]])
        shared = fork(*a, s["parents"], s["children"], case["page"])
        grown = resize(*a, s["children"], s["next"], case["page"], [s["pool"]])
        return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "pool": s["pool"].view(torch.int16),
                "gone": gone, "shared": shared, "grown": grown}
    # compaction: the bookkeeping as it was before, since a tidy cache has nothing to move (the pages that
    # moved are still in their old places too)
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    (proj.cache_compact if own else _compact)(s["table"], s["lens"], s["refs"], case["page"], [s["pool"]], live=s["live"])
    return {"table": s["table"], "refs": s["refs"], "pool": s["pool"].view(torch.int16), "live": s["live"]}


def _attention(q, k, v, table, lens, scale, dv):
    B, H, dk = q.shape
    page, kv = k.shape[1], k.shape[2]
    most = table.shape[1] * page
    t = torch.arange(most, device=q.device)
    ids = table.long().clamp(min=0)
    seen = t[None, :] < lens[:, None]                                        # [B, T]
    qf = q.float().view(B, kv, H // kv, dk)
    kf = k[ids].float().view(B, most, kv, dk).permute(0, 2, 1, 3)            # [B, kv, T, dk]
    vf = kf[..., :dv] if v is None else v[ids].float().view(B, most, kv, dv).permute(0, 2, 1, 3)
    sc = torch.matmul(qf, kf.transpose(2, 3)) * scale                        # [B, kv, G, T]
    sc = sc.masked_fill(~seen[:, None, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m.clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    vf = vf.masked_fill(~seen[:, None, :, None], 0.0)
    o = torch.matmul(p, vf) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total)).view(B, H)
    return o.reshape(B, H, dv).to(q.dtype), lse


def _turn(x, cs, interleaved):
    """x [n, heads, rot] turned by the angles whose cosines and sines cs [n, rot] holds."""
    half = x.shape[-1] // 2
    c, s = cs[:, None, :half], cs[:, None, half:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _append(s, rot, interleaved):
    cs = s["cos_sin"][s["pos"].long()]
    page = s["k"].shape[1]
    at = s["table"][s["rows"].long(), (s["pos"] // page).long()].long()
    off = (s["pos"] % page).long()
    kn, q = s["k_new"].float(), s["q"].float()
    kn = torch.cat([kn[..., :-rot], _turn(kn[..., -rot:], cs, interleaved)], -1) if rot < kn.shape[-1] else _turn(kn, cs, interleaved)
    qn = torch.cat([q[..., :-rot], _turn(q[..., -rot:], cs, interleaved)], -1) if rot < q.shape[-1] else _turn(q, cs, interleaved)
    s["k"][at, off] = kn.to(torch.bfloat16)
    if s["v"] is not None:
        s["v"][at, off] = s["v_new"]
    s["q_out"].copy_(qn.to(torch.bfloat16))


def _resize(table, lens, refs, rows, new_lens, page, pools):
    """Rows grow into the lowest free pages, in the order of the call, or give their last pages back; a row that
    grows and whose last page is part full and shared gets a copy of that page first."""
    r = rows.long()
    old, new = lens[r].long(), new_lens.long()
    have, want = (old + page - 1) // page, (new + page - 1) // page
    last = table[r, (have - 1).clamp(min=0)].long()
    part = (new > old) & (old % page != 0)
    cow = part & (refs[last.clamp(min=0)] > 1)
    need = (want - have).clamp(min=0) + cow
    upto = torch.cumsum(need, 0)
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)            # the free pages first, in order
    ok = (need == 0) | (upto <= (refs == 0).sum())
    first = upto - need
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    grows = ok[:, None] & (j >= have[:, None]) & (j < want[:, None])
    cows = (ok & cow)[:, None] & (j == have[:, None] - 1)
    gives = ok[:, None] & (j >= want[:, None]) & (j < have[:, None])
    now = table[r].long()
    at = torch.where(cows, first[:, None], first[:, None] + cow[:, None] + j - have[:, None])
    taken = free[at.clamp(0, free.shape[0] - 1)]
    d = torch.zeros(refs.shape[0] + 1, dtype=torch.int32, device=refs.device)
    none = torch.full_like(now, refs.shape[0])
    one = torch.ones(now.numel(), dtype=torch.int32, device=refs.device)
    d.index_add_(0, torch.where(grows | cows, taken, none).flatten(), one)
    d.index_add_(0, torch.where(gives | cows, now, none).flatten(), -one)
    refs += d[:-1]
    table[r] = torch.where(grows | cows, taken, torch.where(gives, torch.full_like(now, -1), now)).to(torch.int32)
    lens[r] = torch.where(ok, new, old).to(torch.int32)
    moved = (ok & cow).nonzero().flatten()
    to = free[first[moved]]
    for pool in pools:
        pool[:, to] = pool[:, last[moved]]
    return torch.where(ok, 0, 1).to(torch.int32)


def _fork(table, lens, refs, parents, children, page):
    p, c = parents.long(), children.long()
    n = lens[p]
    used = torch.arange(table.shape[1], device=table.device)[None, :] < ((n + page - 1) // page)[:, None]
    rows = torch.where(used, table[p], torch.full_like(table[p], -1))
    table[c] = torch.where(used, rows, table[c])
    lens[c] = n
    d = torch.zeros(refs.shape[0] + 1, dtype=torch.int32, device=refs.device)
    at = torch.where(used, rows.long(), torch.full_like(rows.long(), refs.shape[0]))
    d.index_add_(0, at.flatten(), torch.ones(at.numel(), dtype=torch.int32, device=refs.device))
    refs += d[:-1]
    return torch.zeros_like(parents)


def _compact(table, lens, refs, page, pools, live):
    """The k-th live page at or past the number of live pages moves to the k-th free page before it."""
    alive = refs > 0
    n = alive.sum()
    ids = torch.arange(refs.shape[0], device=refs.device)
    holes = (~alive & (ids < n)).nonzero().flatten()
    tails = (alive & (ids >= n)).nonzero().flatten()
    for pool in pools:
        pool[:, holes] = pool[:, tails]
    to = ids.clone()
    to[tails] = holes
    used = torch.arange(table.shape[1], device=table.device)[None, :] < ((lens + page - 1) // page)[:, None]
    table.copy_(torch.where(used, to[table.long().clamp(min=0)].to(torch.int32), table))
    refs[holes] = refs[tails]
    refs[tails] = 0
    live.copy_(n.to(torch.int32).view(1))


# ---- what a pass cannot do without ------------------------------------------------------------------

def work(case):
    op, page = case["op"], case["page"]
    if op == "attn":
        lens = _lens(case, case["batch"])
        tok = sum(lens)
        row = case["kv_heads"] * (case["dk"] + (0 if case["latent"] else case["dv"])) * 2
        io = case["batch"] * case["heads"] * ((case["dk"] + case["dv"]) * 2 + 4)
        return {"bytes": tok * row + io + 4 * sum(-(-n // page) for n in lens) + 4 * len(lens),
                "flops": 2.0 * tok * case["heads"] * (case["dk"] + case["dv"])}
    if op == "append":
        n = case["tokens"]
        row = case["kv_heads"] * (case["dk"] + (0 if case["latent"] else case["dv"])) * 2
        return {"bytes": 2 * n * row + 2 * n * case["heads"] * case["dk"] * 2 + n * (case["rot"] * 4 + 12),
                "flops": 3.0 * n * (case["heads"] + case["kv_heads"]) * case["rot"]}
    one = case["page"] * case["row_bytes"] * case["layers"]
    if op == "copy":
        return {"bytes": 2 * case["pairs"] * one + 8 * case["pairs"], "flops": 0}
    if op == "beam":
        lens = _lens(case, case["parents"])
        part = sum(n % page != 0 for n in lens) / len(lens)
        pages = case["children"] * sum(-(-n // page) for n in lens) / len(lens)
        return {"bytes": 2 * case["children"] * part * one + 4 * (5 * pages + case["pages"]), "flops": 0}
    # compaction: a page moves if it lies past the number of live pages; live pages lie anywhere
    counts = sum(-(-n // page) for n in _lens(case, case["rows"]))
    moved = counts * (1 - counts / case["pages"])
    return {"bytes": 2 * moved * one + 4 * (2 * counts + 2 * case["pages"]), "flops": 0}


# ---- the definition, in 64 bits ---------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op not in ("attn", "append"):
        return None                     # whole numbers and copies: nothing is computed
    s = prepare(case, seed)
    if op == "attn":
        out = torch.zeros(case["batch"], case["heads"], case["dv"], dtype=torch.float64, device=DEV)
        lse = torch.full((case["batch"], case["heads"]), -math.inf, dtype=torch.float64, device=DEV)
        group = case["heads"] // case["kv_heads"]
        for b, n in enumerate(s["lens"].tolist()):
            if n == 0:
                continue
            ids = s["table"][b, : -(-n // case["page"])].long()
            keys = s["k"][ids].flatten(0, 1)[:n]
            vals = keys[..., : case["dv"]] if s["v"] is None else s["v"][ids].flatten(0, 1)[:n]
            for h in range(case["kv_heads"]):
                at = slice(h * group, (h + 1) * group)
                x = s["q"][b, at].double() @ keys[:, h].double().T * float(s["scale"])
                lse[b, at] = torch.logsumexp(x, -1)
                out[b, at] = torch.softmax(x, -1) @ vals[:, h].double()
        return {"out": out, "lse": lse}
    n, rot = case["tokens"], case["rot"]
    rows, pos = s["rows"].cpu().numpy(), s["pos"].cpu().numpy()
    table = s["table"].cpu().numpy()
    cs = s["cos_sin"].cpu().numpy().astype(np.float64)[pos]
    c, sn = cs[:, None, : rot // 2], cs[:, None, rot // 2:]

    def turned(x):
        y = x.astype(np.float64)
        a = x.shape[-1] - rot
        i = np.arange(rot // 2)
        one, two = (a + 2 * i, a + 2 * i + 1) if case["interleaved"] else (a + i, a + rot // 2 + i)
        u, w = y[..., one].copy(), y[..., two].copy()
        y[..., one] = u * c - w * sn
        y[..., two] = w * c + u * sn
        return y

    k = s["k"].float().cpu().numpy().astype(np.float64)
    at, off = table[rows, pos // case["page"]], pos % case["page"]
    k[at, off] = turned(s["k_new"].float().cpu().numpy())
    v = None
    if s["v"] is not None:
        v = s["v"].float().cpu().numpy().astype(np.float64)
        v[at, off] = s["v_new"].float().cpu().numpy()
    return {"q": turned(s["q"].float().cpu().numpy()), "k": k, "v": v}
