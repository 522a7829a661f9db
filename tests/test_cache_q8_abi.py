"""What the calls of the cache in 8 bits refuse before anything is enqueued (no GPU needed)."""
import struct

import pytest
import torch

A = 0x7F0000000000


@pytest.fixture(scope="module")
def hsp():
    from hidden_state_projection_gb300 import build
    build.build()
    import hidden_state_projection_gb300 as m
    m.lib()
    return m


def index(table=A, stride=8, lens=A, refs=A, rows=4, width=8, pages=32, page=64):
    return struct.pack("PqPPiiii", table, stride, lens, refs, rows, width, pages, page)


def kv(k=A, v=0, ks=A, vs=0, heads=1, dk=576, dv=512, block=16, kst=(36864, 576, 576), vst=(0, 0, 0), kss=(4, 1, 1), vss=(0, 0, 0)):
    return struct.pack("PPPPiiii12q", k, v, ks, vs, heads, dk, dv, block, *kst, *vst, *kss, *vss)


GROUPED = dict(v=A, vs=A, heads=2, dk=128, dv=128, kst=(16384, 256, 128), vst=(16384, 256, 128), kss=(8, 2, 1), vss=(8, 2, 1))
BAD = [(dict(kvp=kv(k=0)), 0), (dict(kvp=kv(ks=0)), 0), (dict(kvp=kv(v=A)), 0), (dict(kvp=kv(vs=A)), 0), (dict(ix=index(table=0)), 0),
       (dict(ix=index(lens=0)), 0), (dict(ix=index(rows=-1)), 0), (dict(ix=index(stride=7)), 0), (dict(rows=A + 1), 2),
       (dict(kvp=kv(block=0)), 1), (dict(kvp=kv(block=-4)), 1), (dict(kvp=kv(block=128)), 1), (dict(kvp=kv(block=24)), 1),
       (dict(kvp=kv(kst=(-36864, 576, 576))), 1), (dict(kvp=kv(kst=(1 << 40, 576, 576))), 1), (dict(kvp=kv(kss=(-4, 1, 1))), 1),
       (dict(kvp=kv(kss=(4, 1 << 39, 1))), 1), (dict(ix=index(page=48)), 1), (dict(ix=index(pages=0)), 1),
       (dict(kvp=kv(k=A + 8)), 2), (dict(kvp=kv(ks=A + 2)), 2), (dict(kvp=kv(kst=(36864, 584, 576))), 2)]


def refused(hsp, call, cases):
    S = hsp.STATUS
    bad, n = (S["PROJ_ERR_INVALID_ARG"], S["PROJ_ERR_UNSUPPORTED_SHAPE"], S["PROJ_ERR_MISALIGNED"]), hsp.launch_count()
    for kw, want in cases:
        assert call(**kw) == bad[want], kw
        assert hsp.lib().proj_last_error_string()
    assert hsp.launch_count() == n


def test_attention_refusals(hsp):
    def call(q=A, qs=(9216, 576), kvp=None, ix=None, rows=None, batch=2, heads=16, scale=0.1, out=A, lse=None, ws=A, n=1 << 40):
        return hsp.lib().proj_paged_attention_q8(q, *qs, kvp or kv(), ix or index(), rows, batch, heads, scale, out, lse, ws, n, None)

    refused(hsp, call, BAD + [
        (dict(q=None), 0), (dict(out=None), 0), (dict(batch=-1), 0), (dict(heads=0), 0), (dict(scale=float("nan")), 0),
        (dict(scale=3e38), 0), (dict(batch=5), 0), (dict(kvp=kv(dk=640)), 1), (dict(kvp=kv(dv=576)), 1), (dict(kvp=kv(heads=3)), 1),
        (dict(kvp=kv(dk=128, dv=128)), 1), (dict(heads=70000), 1), (dict(kvp=kv(**{**GROUPED, "dv": 64})), 1),
        (dict(kvp=kv(kst=(36864, 0, 576))), 1), (dict(kvp=kv(kst=(0, 576, 576))), 1), (dict(ix=index(width=1 << 25, stride=1 << 25)), 1),
        (dict(qs=(0, 576)), 1), (dict(q=A + 8), 2), (dict(out=A + 8), 2), (dict(qs=(9216, 577)), 2), (dict(lse=A + 2), 2)])
    assert call(batch=0) == 0 and call(batch=0, kvp=kv(**GROUPED)) == 0
    for ws in (dict(ws=None), dict(n=1000), dict(ws=A + 8)):
        assert call(**ws) != 0


def test_append_refusals(hsp):
    def call(kn=A, ks=576, vn=0, vs=0, kvp=None, ix=None, rows=None, pos=A, tokens=2, rot=None, q=0, qs=(9216, 576), qo=0, qos=(9216, 576),
             heads=16):
        return hsp.lib().proj_cache_append_q8(kn, ks, vn, vs, kvp or kv(), ix or index(), rows, pos, tokens, rot, q, *qs, qo, *qos, heads, None)

    def rotary(cs=A, max_pos=512, dim=64):
        return struct.pack("Piiii", cs, max_pos, dim, 1, 0)

    refused(hsp, call, BAD + [
        (dict(kn=0), 0), (dict(tokens=-1), 0), (dict(tokens=5), 0), (dict(vn=A), 0), (dict(kvp=kv(**GROUPED)), 0), (dict(q=A, qo=A), 0),
        (dict(q=A, rot=rotary()), 0), (dict(q=A, qo=A, rot=rotary(), heads=0), 0), (dict(rot=rotary(cs=0)), 0), (dict(rot=rotary(max_pos=0)), 0),
        (dict(q=A, qo=A, rot=rotary(), qos=(9216 * 2, 576)), 0), (dict(rot=rotary(dim=24)), 1), (dict(rot=rotary(dim=640)), 1),
        (dict(kvp=kv(dk=8)), 1), (dict(kvp=kv(dk=568)), 1), (dict(kvp=kv(heads=0)), 1), (dict(q=A, qo=A, rot=rotary(), heads=65536), 1),
        (dict(kvp=kv(kst=(36864, 560, 576))), 1), (dict(kvp=kv(kss=(3, 1, 1))), 1), (dict(kvp=kv(**{**GROUPED, "vss": (8, 1, 1)}), vn=A), 1),
        (dict(q=A, qo=A + 1024, rot=rotary(), qos=(9216, 512)), 1), (dict(kn=A + 8), 2), (dict(ks=577), 2), (dict(pos=A + 2), 2),
        (dict(rot=rotary(cs=A + 4)), 2), (dict(q=A + 2, qo=A, rot=rotary()), 2)])
    assert call(tokens=0) == 0 and call(tokens=0, kvp=kv(**GROUPED), vn=A) == 0


def test_read_refusals(hsp):
    def call(kvp=None, ix=None, rows=None, pos=A, tokens=2, ko=A, ks=576, vo=0, vs=0):
        return hsp.lib().proj_cache_read_q8(kvp or kv(), ix or index(), rows, pos, tokens, ko, ks, vo, vs, None)

    refused(hsp, call, BAD + [
        (dict(ko=0), 0), (dict(tokens=-1), 0), (dict(tokens=5), 0), (dict(vo=A), 0), (dict(kvp=kv(**GROUPED)), 0), (dict(kvp=kv(dk=24)), 1),
        (dict(kvp=kv(heads=-2)), 1), (dict(kvp=kv(heads=1 << 16, dk=512)), 1), (dict(ks=568), 1), (dict(ko=A + 8), 2), (dict(ks=580), 2),
        (dict(pos=A + 3), 2)])
    assert call(tokens=0) == 0


def test_workspace_bytes(hsp):
    for heads, kvh, dk, dv, latent in ((16, 1, 576, 512, True), (128, 1, 512, 512, True), (32, 8, 128, 128, False), (28, 4, 64, 64, False)):
        a, b = (hsp.paged_attention_q8_workspace_bytes(n, heads, kvh, dk, dv, latent) for n in (1, 9))
        assert b >= a + 8 * heads * 2 * dk and hsp.paged_attention_q8_workspace_bytes(0, heads, kvh, dk, dv, latent) <= a
    for args in ((1, 16, 1, 640, 512, True), (1, 0, 1, 576, 512, True), (1, 7, 2, 64, 64, False), (1, 8, 2, 96, 96, False),
                 (1, 1 << 40, 1, 576, 512, True), (-1, 16, 1, 576, 512, True)):
        with pytest.raises(hsp.ProjError):
            hsp.paged_attention_q8_workspace_bytes(*args)


def test_workspace_of_a_larger_batch_serves_a_smaller_one(hsp):
    for heads, kv, dk, dv, latent in ((16, 1, 576, 512, True), (128, 1, 512, 512, True), (32, 8, 128, 128, False), (28, 4, 64, 64, False), (80, 2, 64, 64, False)):
        sizes = [hsp.paged_attention_q8_workspace_bytes(b, heads, kv, dk, dv, latent) for b in (0, 1, 2, 18, 19, 20, 37, 38, 39, 151, 152, 153, 4000)]
        assert sizes == sorted(sizes) and sizes[-1] > sizes[0]


def test_python_refusals(hsp):
    k, ks = torch.zeros(4, 16, 1, 576, dtype=torch.float8_e4m3fn), torch.ones(4, 1, 1)
    table, lens, q = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    for call in (lambda: hsp.paged_attention_q8(q, k, None, ks, None, table, lens, 0.1),
                 lambda: hsp.cache_append_q8(q[:, 0], None, k, None, ks, None, table, lens),
                 lambda: hsp.cache_read_q8(k, None, ks, None, table, lens),
                 lambda: hsp.cache_read_q8(k, None, 3, None, table, lens)):
        with pytest.raises(hsp.ProjError) as e:
            call()
        assert e.value.status == hsp.STATUS["PROJ_ERR_INVALID_ARG"]
