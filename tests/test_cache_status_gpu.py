"""A refused call says the same with and without a given workspace, on the current stream and on another."""
import pytest
import torch

from test_cache_gpu import BF, hsp  # noqa: F401  (hsp: the module's fixture)

pytestmark = pytest.mark.gpu


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def refusal(hsp, call):  # noqa: F811
    n = hsp.launch_count()
    with pytest.raises(hsp.ProjError) as ei:
        call()
    assert hsp.launch_count() == n
    return ei.value.status_name, str(ei.value)


# (queries, keys, values, table); a table of 64 pages can be cut and takes a workspace, one of 4 does not
ATTENTION = {"no heads": ((2, 0, 576), (8, 16, 1, 576), None, "INVALID_ARG"),
             "heads that do not divide": ((2, 16, 576), (8, 16, 3, 576), None, "UNSUPPORTED_SHAPE"),
             "columns": ((2, 16, 96), (8, 16, 1, 96), (8, 16, 1, 96), "UNSUPPORTED_SHAPE"),
             "page size": ((2, 16, 576), (8, 24, 1, 576), None, "UNSUPPORTED_SHAPE"),
             "no pages": ((2, 16, 576), (0, 16, 1, 576), None, "UNSUPPORTED_SHAPE"),
             "rows of the table on top of each other": ((2, 16, 576), (8, 16, 1, 576), None, "INVALID_ARG"),
             "queries of two dimensions": ((2, 576), (8, 16, 1, 576), None, "INVALID_ARG"),
             "keys of three dimensions": ((2, 16, 576), (8, 16, 576), None, "INVALID_ARG"),
             "values of three dimensions": ((2, 16, 64), (8, 16, 1, 64), (8, 16, 64), "INVALID_ARG"),
             "more sequences than rows": ((3, 16, 576), (8, 16, 1, 576), None, "INVALID_ARG")}


@pytest.mark.parametrize("width", [4, 64])
@pytest.mark.parametrize("what", list(ATTENTION))
def test_attention(hsp, what, width):  # noqa: F811
    qs, ks, vs, want = ATTENTION[what]
    q, k = torch.zeros(qs, dtype=BF, device="cuda"), torch.zeros(ks, dtype=BF, device="cuda")
    v = None if vs is None else torch.zeros(vs, dtype=BF, device="cuda")
    table, lens = ints(2, width), ints(2)
    if "on top" in what:
        table = table[:1].expand(2, width)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    got = {refusal(hsp, lambda: hsp.paged_attention(q, k, v, table, lens, 0.1, workspace=w, stream=s)) for w in (None, ws) for s in (None, side)}
    assert {x for x, _ in got} == {"PROJ_ERR_" + want}, got
    assert len(got) == 1, got


PAGES = {"rows of the table on top of each other": dict(expand=True, want="INVALID_ARG"), "page size": dict(page=24, want="UNSUPPORTED_SHAPE"),
         "no rows": dict(rows=0, want="UNSUPPORTED_SHAPE"), "rows of two dimensions": dict(shape=(3, 1), want="INVALID_ARG"),
         "counts of two dimensions": dict(refs=(4, 2), want="INVALID_ARG"), "pools of other pages": dict(pages=9, want="INVALID_ARG")}


@pytest.mark.parametrize("what", list(PAGES))
def test_page_calls(hsp, what):  # noqa: F811
    c = dict(expand=False, page=16, rows=4, shape=(3,), refs=(8,), pages=8)
    c.update(PAGES[what])
    table, lens, refs, req = ints(c["rows"], 8), ints(c["rows"]), ints(*c["refs"]), ints(*c["shape"])
    if c["expand"]:
        table = table[:1].expand(c["rows"], 8)
    pool = torch.zeros(1, c["pages"], 16, 8, dtype=BF, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    a = (table, lens, refs)
    for name, call in (("resize", lambda w, s: hsp.cache_resize(*a, req, req, c["page"], [pool], workspace=w, stream=s)),
                       ("fork", lambda w, s: hsp.cache_fork(*a, req, req, c["page"], stream=s)),
                       ("compact", lambda w, s: hsp.cache_compact(*a, c["page"], [pool], workspace=w, stream=s))):
        if (name == "compact" and what == "rows of two dimensions") or (name == "fork" and what == "pools of other pages"):
            continue
        got = {refusal(hsp, lambda: call(w, s)) for w in (None, ws) for s in (None, side)}
        assert {x for x, _ in got} == {"PROJ_ERR_" + c["want"]}, (name, got)
        assert len(got) == 1, (name, got)


def test_what_is_wrong_with_a_workspace(hsp):  # noqa: F811
    """Too short, misaligned, not dense: refused; the NULL of a C caller too."""
    from test_attention_gpu import make
    args = make([600], 16, 1, 576, True, 64, 1)
    need = hsp.paged_attention_workspace_bytes(16, 1, 576, 512, True)
    ws = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
    for w, want in ((ws[:need - 1], "INVALID_ARG"), (ws[8:], "MISALIGNED"), (ws[::2], "INVALID_ARG"), (ws[:0], "INVALID_ARG")):
        assert refusal(hsp, lambda: hsp.paged_attention(*args, 0.1, workspace=w))[0] == "PROJ_ERR_" + want
    hsp.paged_attention(*args, 0.1, workspace=ws[16:16 + need])
    q, k, _, table, lens = args
    import struct
    kv = struct.pack("PPiiiiqqqqqq", k.data_ptr(), 0, 1, 576, 512, 0, *k.stride()[:3], 0, 0, 0)
    index = struct.pack("PqPPiiii", table.data_ptr(), table.stride(0), lens.data_ptr(), 0, 1, table.shape[1], k.shape[0], 64)
    out = torch.empty(1, 16, 512, dtype=BF, device="cuda")
    n = hsp.launch_count()
    for p, size, want in ((None, need, "INVALID_ARG"), (ws.data_ptr() + 4, need, "MISALIGNED"), (ws.data_ptr(), need - 1, "INVALID_ARG")):
        assert hsp.lib().proj_paged_attention(q.data_ptr(), *q.stride()[:2], kv, index, None, 1, 16, 0.1, out.data_ptr(), None, p, size,
                                              None) == hsp.STATUS["PROJ_ERR_" + want]
    assert hsp.launch_count() == n
    hsp.check_device_error()


def test_sizes_that_do_not_fit_32_bits(hsp):  # noqa: F811
    """Sizes far outside their range are refused, not cut to 32 bits; a negative v_dim is none of the defaults."""
    q, k = torch.zeros(1, 16, 576, dtype=BF, device="cuda"), torch.zeros(4, 16, 1, 576, dtype=BF, device="cuda")
    table, lens, refs, pool = ints(1, 4), ints(1), ints(4), torch.zeros(1, 4, 16, 8, dtype=BF, device="cuda")
    for big in (2 ** 32, -2 ** 32, 2 ** 40, -2 ** 40):
        want = "PROJ_ERR_UNSUPPORTED_SHAPE"
        for stream in (None, torch.cuda.Stream()):
            assert refusal(hsp, lambda: hsp.paged_attention(q, k, None, table, lens, 0.1, v_dim=512 + big, stream=stream))[0] == want
        assert refusal(hsp, lambda: hsp.cache_resize(table, lens, refs, lens, lens, 16 + big, [pool]))[0] == want
        assert refusal(hsp, lambda: hsp.cache_fork(table, lens, refs, lens, lens, 16 + big))[0] == want
        assert refusal(hsp, lambda: hsp.cache_compact(table, lens, refs, 16 + big, [pool]))[0] == want
    for v_dim in (-1, -2, 0, 576):
        assert refusal(hsp, lambda: hsp.paged_attention(q, k, None, table, lens, 0.1, v_dim=v_dim))[0] == "PROJ_ERR_UNSUPPORTED_SHAPE"
    g = torch.zeros(4, 16, 1, 64, dtype=BF, device="cuda")
    for v_dim in (-1, 63, 64 + 2 ** 32):
        assert refusal(hsp, lambda: hsp.paged_attention(q[..., :64], g, g, table, lens, 0.1, v_dim=v_dim))[0] == "PROJ_ERR_INVALID_ARG"
    assert not hsp.paged_attention(q, k, None, table, lens, 0.1, v_dim=512).any()
    hsp.check_device_error()


def test_no_memory_for_an_output_is_torchs_own_error(hsp):  # noqa: F811
    """The output of so many (expanded) queries does not fit any GPU: the error that a server catches to make room."""
    q, k = torch.zeros(1, 1, 576, dtype=BF, device="cuda").expand(2 ** 22, 256, 576), torch.zeros(4, 16, 1, 576, dtype=BF, device="cuda")
    n = hsp.launch_count()
    with pytest.raises(torch.OutOfMemoryError):
        hsp.paged_attention(q, k, None, ints(1, 4), ints(1), 0.1)
    assert hsp.launch_count() == n
