"""cache_append into pages that hold heads before tokens or lie in wider tensors, and with queries and turned queries
that are parts of wider tensors.  The bounds of a turned value are those of test_cache_gpu.turned."""
import pytest
import torch

from test_cache_gpu import BF, hsp, turned  # noqa: F401  (hsp: the module's fixture)

pytestmark = pytest.mark.gpu


def pages_of(kind, pages, page, heads, dim, g):
    """(buffer, its [pages, page, heads, dim] view)"""
    if kind == "heads first":
        buf = torch.randn(pages, heads, page, dim, generator=g, device="cuda").to(BF)
        return buf, buf.transpose(1, 2)
    if kind == "columns of a wider tensor":
        buf = torch.randn(pages, page, heads, dim + 24, generator=g, device="cuda").to(BF)
        return buf, buf[..., 16:16 + dim]
    buf = torch.randn(page, pages, 2, heads, dim, generator=g, device="cuda").to(BF)   # a token of all pages, keys beside values
    return buf, buf[:, :, 1].transpose(0, 1)


@pytest.mark.parametrize("kind", ["heads first", "columns of a wider tensor", "tokens first"])
@pytest.mark.parametrize("n,heads,kv,dk,latent,rot,inter", [(7, 5, 1, 576, True, 64, True), (33, 16, 8, 128, False, 128, False),
                                                            (300, 3, 3, 64, False, 32, True), (1, 128, 1, 512, True, 48, False)])
def test_layouts(hsp, kind, n, heads, kv, dk, latent, rot, inter):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(n + heads)
    page, width, seqs = 16, 8, 5
    pages = seqs * width + 2
    table = torch.randperm(pages, generator=g, device="cuda")[:seqs * width].view(seqs, width).to(torch.int32)
    which = torch.randperm(seqs * width * page, generator=g, device="cuda")[:n]
    rows, pos = (which // (width * page)).to(torch.int32), (which % (width * page)).to(torch.int32)
    lens = torch.full((seqs,), width * page, dtype=torch.int32, device="cuda")
    kb, k = pages_of(kind, pages, page, kv, dk, g)
    vb, v = (None, None) if latent else pages_of(kind, pages, page, kv, dk, g)
    kn = torch.randn(n, kv, dk, generator=g, device="cuda").to(BF)
    vn = None if latent else torch.randn(n, kv, dk, generator=g, device="cuda").to(BF)
    ang = torch.rand(width * page, rot // 2, generator=g, device="cuda") * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).contiguous()
    qw = torch.randn(heads, n, dk + 40, generator=g, device="cuda").to(BF)              # heads first, columns of a wider tensor
    q = qw[..., 8:8 + dk].transpose(0, 1)
    ow = torch.full((n, heads + 2, dk + 8), 3.0, dtype=BF, device="cuda")
    q_out = ow[:, 1:heads + 1, :dk]
    want_k, want_v, q0 = kb.clone(), None if latent else vb.clone(), qw.clone()
    got = hsp.cache_append(kn, vn, k, v, table, lens, rows=rows, positions=pos, cos_sin=cs, interleaved=inter, q=q, q_out=q_out)
    hsp.check_device_error()
    assert got is q_out and torch.equal(qw, q0)
    at, off = table[rows.long(), (pos // page).long()].long(), (pos % page).long()
    y, t = turned(kn, cs[pos.long()], rot, inter)
    assert ((k[at, off].double() - y).abs() <= t).all()
    # nothing else has changed: the buffer as it was, with the new rows in their places
    view = {"heads first": lambda b: b.transpose(1, 2), "columns of a wider tensor": lambda b: b[..., 16:16 + dk],
            "tokens first": lambda b: b[:, :, 1].transpose(0, 1)}[kind]
    view(want_k)[at, off] = k[at, off]
    assert torch.equal(kb, want_k)
    if not latent:
        view(want_v)[at, off] = vn
        assert torch.equal(vb, want_v)
    y, t = turned(q, cs[pos.long()], rot, inter)
    assert ((q_out.double() - y).abs() <= t).all()
    turned_q = q_out.clone()
    ow[:, 1:heads + 1, :dk] = 3.0
    assert (ow == 3.0).all()
    # in place, with the queries' own strides
    assert hsp.cache_append(kn, vn, k, v, table, lens, rows=rows, positions=pos, cos_sin=cs, interleaved=inter, q=q, q_out=q) is q
    assert torch.equal(q, turned_q)
    q0[..., 8:8 + dk] = qw[..., 8:8 + dk]
    assert torch.equal(qw, q0)
    hsp.check_device_error()


@pytest.mark.parametrize("heads,kv,dk,rot,inter", [(8, 2, 128, 64, False), (4, 4, 64, 32, True), (6, 1, 128, 32, False)])
def test_models_that_turn_the_first_columns(hsp, heads, kv, dk, rot, inter):  # noqa: F811
    """Weights whose rows are rolled by `rot` within each head put the columns to turn last; the attention is that of
    the model as it is written, which turns the first columns."""
    g = torch.Generator(device="cuda").manual_seed(heads)
    K, n, page = 256, 70, 16
    wq, wk, wv = ((torch.randn(h, dk, K, generator=g, device="cuda") * K ** -0.5).to(BF) for h in (heads, kv, kv))
    x = torch.randn(n, K, generator=g, device="cuda").to(BF)
    ang = torch.rand(n, rot // 2, generator=g, device="cuda") * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).contiguous()
    laid_out = torch.cat([w.roll(-rot, 1).reshape(-1, K) for w in (wq, wk)] + [wv.reshape(-1, K)])
    k, v = (torch.zeros(8, page, kv, dk, dtype=BF, device="cuda") for _ in range(2))
    table = torch.tensor([[5, 2, 7, 0, 4]], dtype=torch.int32, device="cuda")
    out = []
    for t in range(n):                                      # decode, token by token
        lens = torch.tensor([t + 1], dtype=torch.int32, device="cuda")
        q, kn, vn = hsp.fused_gemm(x[t:t + 1], laid_out, [heads * dk, kv * dk, kv * dk])
        q = hsp.cache_append(kn, vn, k, v, table, lens, cos_sin=cs, interleaved=inter, q=q.view(1, heads, dk))
        out.append(hsp.paged_attention(q, k, v, table, lens, dk ** -0.5))
    hsp.check_device_error()
    # the model in 64 bits, its projections rounded as the library's are

    def project(w):
        return torch.stack([hsp.fused_gemm(x[t:t + 1], w.reshape(-1, K), [w.shape[0] * dk])[0][0] for t in range(n)]).view(n, -1, dk)

    def first(y):
        half, c, s = rot // 2, ang.double().cos()[:, None], ang.double().sin()[:, None]
        y = y.double().clone()
        one, two = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, half), slice(half, rot))
        a, b = y[..., one].clone(), y[..., two].clone()
        y[..., one], y[..., two] = a * c - b * s, b * c + a * s
        return y

    qq, kk, vv = first(project(wq)), first(project(wk)), project(wv).double()
    for t in range(n):
        for h in range(heads):
            keys, vals = kk[:t + 1, h * kv // heads], vv[:t + 1, h * kv // heads]
            sc = keys @ qq[t, h] * dk ** -0.5
            p = torch.softmax(sc, 0)
            # turned queries and keys are rounded once more: scores off by 2^-7 of their terms' sum, weights by e^that
            off = 2.0 ** -7 * float((keys.abs() @ qq[t, h].abs()).max()) * dk ** -0.5 + 2.0 ** -7
            tol = (p @ vals.abs()) * (torch.tensor(2 * off).exp() - 1 + 2.0 ** -7).cuda() + 2.0 ** -8 * (p @ vals).abs()
            assert ((out[t][0, h].double() - p @ vals).abs() <= tol).all(), (t, h)
