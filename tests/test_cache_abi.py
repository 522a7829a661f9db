"""What the paged cache's calls refuse before anything is enqueued (no GPU needed), and the sizes they ask for."""
import ctypes
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


def kv(k=A, v=0, heads=1, dk=576, dv=512, ks=(36864, 576, 576), vs=(0, 0, 0)):
    return struct.pack("PPiiiiqqqqqq", k, v, heads, dk, dv, 0, *ks, *vs)


def pool(base=A, layer=1 << 20, page=4096, size=4096, layers=2):
    return struct.pack("Pqqqii", base, layer, page, size, layers, 0)


def attend(hsp, q=A, qs=(9216, 576), kvp=None, ix=None, rows=None, batch=2, heads=16, scale=0.1, out=A, lse=None, ws=A,
           ws_bytes=1 << 40):
    return hsp.lib().proj_paged_attention(q, *qs, kvp or kv(), ix or index(), rows, batch, heads, scale, out, lse, ws,
                                          ws_bytes, None)


def test_attention_refusals(hsp):
    S, n = hsp.STATUS, hsp.launch_count()
    bad = S["PROJ_ERR_INVALID_ARG"], S["PROJ_ERR_UNSUPPORTED_SHAPE"], S["PROJ_ERR_MISALIGNED"]
    for kw, want in [(dict(q=None), 0), (dict(out=None), 0), (dict(batch=-1), 0), (dict(heads=0), 0), (dict(scale=float("nan")), 0),
                     (dict(scale=float("inf")), 0), (dict(scale=3e38), 0), (dict(batch=5), 0), (dict(kvp=kv(k=0)), 0), (dict(ix=index(table=0)), 0),
                     (dict(ix=index(lens=0)), 0), (dict(ix=index(rows=-1)), 0), (dict(ix=index(stride=7)), 0),
                     (dict(kvp=kv(dk=575)), 1), (dict(kvp=kv(dk=640)), 1), (dict(kvp=kv(dv=576)), 1), (dict(kvp=kv(dk=128, dv=128)), 1),
                     (dict(kvp=kv(v=A, vs=(36864, 576, 576))), 1), (dict(kvp=kv(heads=3)), 1), (dict(heads=70000), 1),
                     (dict(ix=index(page=48)), 1), (dict(ix=index(page=8)), 1), (dict(ix=index(page=2048)), 1),
                     (dict(ix=index(rows=0)), 1), (dict(ix=index(width=0)), 1), (dict(ix=index(pages=0)), 1),
                     (dict(ix=index(width=1 << 25, stride=1 << 25)), 1), (dict(kvp=kv(ks=(36864, 0, 576))), 1),
                     (dict(kvp=kv(ks=(0, 576, 576))), 1), (dict(kvp=kv(ks=(1 << 40, 576, 576))), 1),
                     (dict(kvp=kv(ks=(-36864, 576, 576))), 1),
                     (dict(q=A + 8), 2), (dict(out=A + 8), 2), (dict(qs=(9216, 577)), 2), (dict(qs=(9217, 576)), 2),
                     (dict(lse=A + 2), 2), (dict(rows=A + 1), 2), (dict(kvp=kv(k=A + 8)), 2), (dict(kvp=kv(ks=(36864, 580, 576))), 2),
                     (dict(ix=index(table=A + 2)), 2)]:
        assert attend(hsp, **kw) == bad[want], kw
        assert hsp.lib().proj_last_error_string()
    for ws in (dict(ws=None), dict(ws_bytes=1000), dict(ws=A + 8)):   # a table row of 512 tokens: sequences may be cut
        assert attend(hsp, **ws) in (*bad, S["PROJ_ERR_DEVICE"], S["PROJ_ERR_CUDA"])
    for qs in ((0, 576), (9216, 0), (-9216, 576), (9216, 1 << 39)):
        assert attend(hsp, qs=qs) == bad[1], qs
    assert attend(hsp, batch=0) == S["PROJ_OK"]
    assert hsp.launch_count() == n


def test_attention_workspace(hsp):
    for heads, kvh, dk, dv, lat in [(16, 1, 576, 512, 1), (128, 1, 512, 512, 1), (32, 8, 128, 128, 0), (1, 1, 64, 64, 0),
                                    (1000, 2, 128, 128, 0)]:
        assert hsp.paged_attention_workspace_bytes(heads, kvh, dk, dv, bool(lat)) > 0
    for heads, kvh, dk, dv, lat in [(16, 3, 576, 512, 1), (0, 1, 576, 512, 1), (16, 1, 576, 576, 1), (16, 1, 96, 96, 0),
                                    (16, 1, 576, 512, 0)]:
        with pytest.raises(hsp.ProjError):
            hsp.paged_attention_workspace_bytes(heads, kvh, dk, dv, bool(lat))


def test_append_refusals(hsp):
    S, n = hsp.STATUS, hsp.launch_count()

    def rot(table=A, most=100, dim=64, inter=1):
        return struct.pack("Piiii", table, most, dim, inter, 0)

    def call(k=A, ks=576, v=None, vs=0, kvp=None, ix=None, rows=None, pos=None, tokens=2, r=rot(), q=None, qs=(9216, 576),
             qo=None, os=(9216, 576), heads=16):
        return hsp.lib().proj_cache_append(k, ks, v, vs, kvp or kv(), ix or index(), rows, pos, tokens, r, q, *qs, qo, *os,
                                           heads, None)

    for kw, want in [(dict(k=None), "INVALID_ARG"), (dict(tokens=-1), "INVALID_ARG"), (dict(tokens=5), "INVALID_ARG"),
                     (dict(v=A), "INVALID_ARG"), (dict(kvp=kv(v=A)), "INVALID_ARG"), (dict(q=A), "INVALID_ARG"),
                     (dict(q=A, qo=A, r=None), "INVALID_ARG"), (dict(q=A, qo=A, heads=0), "INVALID_ARG"),
                     (dict(r=rot(table=0)), "INVALID_ARG"), (dict(r=rot(most=0)), "INVALID_ARG"),
                     (dict(r=rot(dim=8)), "UNSUPPORTED_SHAPE"), (dict(r=rot(dim=72)), "UNSUPPORTED_SHAPE"),
                     (dict(r=rot(dim=592)), "UNSUPPORTED_SHAPE"), (dict(kvp=kv(dk=12)), "UNSUPPORTED_SHAPE"),
                     (dict(kvp=kv(heads=0)), "UNSUPPORTED_SHAPE"), (dict(r=rot(table=A + 4)), "MISALIGNED"),
                     (dict(k=A + 2), "MISALIGNED"), (dict(ks=577), "MISALIGNED"), (dict(q=A, qo=A + 8), "MISALIGNED"),
                     (dict(q=A, qo=A, qs=(9216, 4)), "MISALIGNED"), (dict(pos=A + 2), "MISALIGNED"),
                     (dict(ix=index(page=20)), "UNSUPPORTED_SHAPE"), (dict(q=A, qo=A, heads=65536), "UNSUPPORTED_SHAPE"),
                     (dict(kvp=kv(heads=65536, dk=512)), "UNSUPPORTED_SHAPE")]:
        assert call(**kw) == S["PROJ_ERR_" + want], (kw, hsp.lib().proj_last_error_string())
    assert call(tokens=0) == S["PROJ_OK"]
    for strides in ((0, 576, 576), (36864, 0, 576)):               # places that would be written twice
        assert call(kvp=kv(ks=strides)) == S["PROJ_ERR_UNSUPPORTED_SHAPE"], strides
    assert call(kvp=kv(v=A, dk=64, dv=64, heads=2, ks=(8192, 128, 64), vs=(8192, 128, 0)), v=A, r=None) == S["PROJ_ERR_UNSUPPORTED_SHAPE"]
    assert hsp.launch_count() == n


def test_page_call_refusals(hsp):
    S, n, lib = hsp.STATUS, hsp.launch_count(), hsp.lib()

    def resize(ix=None, rows=A, new=A, cnt=3, pools=pool(), np=1, st=A, ws=A, wb=1 << 30):
        return lib.proj_cache_resize(ix or index(), rows, new, cnt, pools, np, st, ws, wb, None)

    def fork(ix=None, p=A, c=A, cnt=3, st=A):
        return lib.proj_cache_fork(ix or index(), p, c, cnt, st, None)

    def compact(ix=None, pools=pool(), np=1, live=A, ws=A, wb=1 << 30):
        return lib.proj_cache_compact(ix or index(), pools, np, live, ws, wb, None)

    bad = S["PROJ_ERR_INVALID_ARG"]
    for st in [resize(rows=None), resize(new=None), resize(st=None), resize(cnt=-1), resize(ws=None), resize(wb=100),
               resize(pools=None), resize(np=0), resize(np=5), resize(ix=index(refs=0)), resize(pools=pool(base=0)),
               resize(pools=pool(layers=0)), resize(pools=pool(size=0)), resize(pools=pool(page=2048)),
               fork(p=None), fork(c=None), fork(st=None), fork(cnt=-2), fork(ix=index(refs=0)),
               compact(live=None), compact(ws=None), compact(wb=64), compact(pools=None)]:
        assert st == bad, hsp.lib().proj_last_error_string()
    for st in [resize(rows=A + 2), resize(ws=A + 4), resize(pools=pool(base=A + 8)), resize(pools=pool(page=4104)),
               resize(pools=pool(layer=8)), fork(p=A + 1), compact(live=A + 2), compact(ws=A + 8)]:
        assert st == S["PROJ_ERR_MISALIGNED"]
    assert resize(cnt=0) == fork(cnt=0) == S["PROJ_OK"]
    assert hsp.launch_count() == n
    table = torch.zeros(4, 8, dtype=torch.int32)
    assert hsp.cache_workspace_bytes(table, 32, 0) < hsp.cache_workspace_bytes(table, 32, 1000)


def test_copy_refusals(hsp):
    S, n, lib = hsp.STATUS, hsp.launch_count(), hsp.lib()

    def copy(src, dst, cnt=None, pages=16, pools=pool()):
        a, b = (ctypes.c_int32 * max(1, len(src)))(*src), (ctypes.c_int32 * max(1, len(dst)))(*dst)
        return lib.proj_cache_copy_pages(pools, 1, pages, a, b, len(src) if cnt is None else cnt, None)

    bad = S["PROJ_ERR_INVALID_ARG"]
    assert copy([0], [16]) == copy([-1], [2]) == copy([16], [2]) == copy([0], [-1]) == bad
    assert copy([0, 1], [2, 2]) == bad and "twice" in lib.proj_last_error_string().decode()
    assert copy([0, 1], [2, 0]) == bad and "a source and a destination" in lib.proj_last_error_string().decode()
    assert copy([3], [3]) == bad
    assert copy([0], [1], cnt=-1) == bad
    assert copy([0] * 2049, list(range(1, 2050)), pages=5000) == S["PROJ_ERR_UNSUPPORTED_SHAPE"]
    src, dst = [0] * 2048, list(range(1, 2049))
    dst[2047] = 1
    assert copy(src, dst, pages=5000) == bad                       # the last destination again, in a full table
    dst[2047] = 0
    assert copy(src, dst, pages=5000) == bad
    assert copy([], []) == S["PROJ_OK"]
    assert hsp.launch_count() == n


def test_a_flag_that_has_no_truth_value(hsp):
    q, k = torch.zeros(1, 16, 576, dtype=torch.bfloat16), torch.zeros(4, 64, 1, 576, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="ambiguous"):
        hsp.paged_attention(q, k, None, table, lens, 0.1, return_lse=torch.zeros(2))


def test_python_checks(hsp):
    """Tensors that are not on the GPU, or not what the call documents."""
    q, k = torch.zeros(1, 16, 576, dtype=torch.bfloat16), torch.zeros(4, 64, 1, 576, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    refs = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: hsp.paged_attention(q, k, None, table, lens, 0.1),
                 lambda: hsp.cache_append(k[0, :1, 0], None, k, None, table, lens),
                 lambda: hsp.cache_resize(table, lens, refs, lens, lens, 64, [k[None]]),
                 lambda: hsp.cache_fork(table, lens, refs, lens, lens, 64),
                 lambda: hsp.cache_compact(table, lens, refs, 64, [k[None]]),
                 lambda: hsp.cache_copy_pages([k[None]], [0], [1])):
        with pytest.raises(hsp.ProjError) as ei:
            call()
        assert ei.value.status_name == "PROJ_ERR_INVALID_ARG"
