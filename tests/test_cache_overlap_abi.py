"""What the paged cache's calls write must not overlap itself: strides for which two threads would store to one place
are refused before anything is enqueued (no GPU needed)."""
import struct

import pytest

from test_cache_abi import A, hsp, index, kv, pool  # noqa: F401  (hsp: the module's fixture)


def append(hsp, kvp, ix=None, v=None, tokens=2, q=None, qo=None, qs=(9216, 576), os=(9216, 576), heads=16):  # noqa: F811
    rot = struct.pack("Piiii", A, 100, 16, 1, 0)
    dk = struct.unpack_from("PPiiii", kvp)[3]
    return hsp.lib().proj_cache_append(A, dk * 8, v, dk * 8, kvp, ix or index(), None, None, tokens, rot if q else None, q, *qs, qo,
                                       *os, heads, None)


# (kv heads, k_dim, (page, token, head) strides) over 32 pages of 64 tokens
APART = [(1, 576, (36864, 576, 0)), (1, 576, (36864, 576, 8)), (1, 576, (576, 576 * 32, 576)), (2, 128, (16384, 256, 128)),
         (2, 128, (16384, 128, 8192)), (2, 128, (1 << 20, 384, 128)), (2, 128, (256, 8192, 128))]
OVERLAP = [(1, 576, (36864, 568, 576)), (1, 576, (36856, 576, 576)), (1, 576, (576, 576, 576)), (2, 128, (16384, 8, 128)),
           (2, 128, (16384, 256, 64)), (2, 128, (16384, 128, 128)), (2, 128, (8192, 128, 8192)), (2, 128, (16384, 248, 128)),
           (2, 128, (16376, 128, 8192))]


@pytest.mark.parametrize("heads,dk,ks", APART)
def test_caches_that_lie_apart(hsp, heads, dk, ks):  # noqa: F811
    if heads == 1:
        assert append(hsp, kv(dk=dk, ks=ks), tokens=0) == hsp.STATUS["PROJ_OK"]
    else:
        good = (1 << 20, 384, 128)
        for a, b in ((ks, good), (good, ks)):
            assert append(hsp, kv(v=A, heads=heads, dk=dk, dv=dk, ks=a, vs=b), v=A, tokens=0) == hsp.STATUS["PROJ_OK"]


@pytest.mark.parametrize("heads,dk,ks", OVERLAP)
def test_caches_that_overlap(hsp, heads, dk, ks):  # noqa: F811
    want = hsp.STATUS["PROJ_ERR_UNSUPPORTED_SHAPE"]
    if heads == 1:
        assert append(hsp, kv(dk=dk, ks=ks), tokens=0) == want
    else:
        good = (1 << 20, 384, 128)
        for a, b in ((ks, good), (good, ks)):
            assert append(hsp, kv(v=A, heads=heads, dk=dk, dv=dk, ks=a, vs=b), v=A, tokens=0) == want
    assert b"overlap" in hsp.lib().proj_last_error_string()


def test_one_page_steps_anywhere(hsp):  # noqa: F811
    assert append(hsp, kv(ks=(8, 576, 0)), ix=index(pages=1), tokens=0) == hsp.STATUS["PROJ_OK"]


@pytest.mark.parametrize("strides", [(0, 576), (9216, 0), (9208, 576), (9216, 568), (576, 576), (-9216, 576), (9216, -576), (1152, 1152)])
def test_turned_queries_that_overlap(hsp, strides):  # noqa: F811
    n = hsp.launch_count()
    assert append(hsp, kv(), q=A, qo=A + (1 << 20), os=strides) == hsp.STATUS["PROJ_ERR_UNSUPPORTED_SHAPE"]
    assert b"q_out" in hsp.lib().proj_last_error_string()
    assert hsp.launch_count() == n


def test_queries_turned_in_place_keep_their_strides(hsp):  # noqa: F811
    n = hsp.launch_count()
    for qs, os in (((9216, 576), (18432, 576)), ((9216, 576), (576, 1152)), ((9216, 0), (9216, 576))):
        assert append(hsp, kv(), q=A, qo=A, qs=qs, os=os) == hsp.STATUS["PROJ_ERR_INVALID_ARG"]
    assert hsp.launch_count() == n


def test_layers_of_a_pool(hsp):  # noqa: F811
    lib, S = hsp.lib(), hsp.STATUS

    def calls(p, pages=32):
        ix = index(pages=pages)
        return (lib.proj_cache_resize(ix, A, A, 0, p, 1, A, A, 1 << 30, None),
                lib.proj_cache_copy_pages(p, 1, pages, None, None, 0, None),
                lib.proj_cache_compact(ix, p, 1, None, A, 1 << 30, None))

    good = (S["PROJ_OK"], S["PROJ_OK"], S["PROJ_ERR_INVALID_ARG"])       # (compact: live is NULL)
    for p in (pool(), pool(layer=4096 * 32), pool(layer=4096, page=8192), pool(layer=0, layers=1), pool(layer=4096, page=8192 + 16)):
        assert calls(p) == good
        assert b"live" in lib.proj_last_error_string()
    assert calls(pool(layer=4096, page=4096), pages=1) == good
    bad = S["PROJ_ERR_INVALID_ARG"]
    for p in (pool(layer=0), pool(layer=16), pool(layer=4080), pool(layer=4096), pool(layer=4096 * 31), pool(layer=4096, page=8176),
              pool(layer=4096, page=8192, layers=3)):
        assert calls(p) == (bad, bad, bad)
        assert b"overlap" in lib.proj_last_error_string()
    assert calls(pool(layer=0), pages=1) == (bad, bad, bad)
