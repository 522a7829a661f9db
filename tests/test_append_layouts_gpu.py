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
