"""Programmatic-dependent-launch ordering of the paged cache's kernels: a consumer that never waits on its grid
dependency reads final values, as behind the projections (test_pdl_order_gpu.py, which has the positive control of
the method).  In a CUDA graph, every replay: the outputs as they were before -> the call -> a consumer (PDL launch,
no griddepcontrol.wait) that counts the words that differ from the expected ones."""
import pytest
import torch

from test_pdl_order_gpu import PER_GRAPH, REPLAYS, consumer, hsp  # noqa: F401  (the fixtures)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def words(t):
    return t.contiguous().view(-1).view(torch.int32)


def stress(hsp, consumer, state, call, replays=REPLAYS):  # noqa: F811
    """`state`: one int32 buffer that holds everything that `call` changes; its present contents are put back
    before every call."""
    start = state.clone()
    call()
    torch.cuda.synchronize()
    hsp.check_device_error()
    want = state.clone()
    assert not torch.equal(want, start)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        stream = torch.cuda.current_stream().cuda_stream
        for _ in range(PER_GRAPH):
            state.copy_(start)
            call()
            assert consumer.pdl_consumer_launch(state.data_ptr(), want.data_ptr(), state.numel(), 0, counter.data_ptr(), stream) == 0
    for _ in range(replays // PER_GRAPH):
        g.replay()
    torch.cuda.synchronize()
    hsp.check_device_error()
    assert torch.equal(state, want)
    assert int(counter.item()) == 0


def parts(sizes):
    """One int32 buffer of -1 and its views: (dtype, shape) each, 16-byte aligned."""
    views, at, spans = [], 0, []
    for dtype, shape in sizes:
        n = 1
        for d in shape:
            n *= d
        w = -(-n * torch.empty(0, dtype=dtype).element_size() // 16) * 4
        spans.append((at, w, n, dtype, shape))
        at += w
    buf = torch.full((at,), -1, dtype=torch.int32, device="cuda")
    for o, w, n, dtype, shape in spans:
        views.append(buf[o:o + w].view(dtype)[:n].view(shape))
    return buf, views


# one launch; cut and joined; many grouped sequences, some joined and some whole
@pytest.mark.parametrize("lens,heads,kv,dk,dv", [([77, 200, 0], 16, 1, 576, 512), ([9000], 64, 1, 512, 512),
                                                 ([1000, 30, 0, 2500, 64], 8, 2, 128, 128)])
def test_attention(hsp, consumer, lens, heads, kv, dk, dv):  # noqa: F811
    from test_attention_gpu import make
    q, k, v, table, ln = make(lens, heads, kv, dk, dv == 512, 64, 3)
    buf, (out, lse) = parts([(BF, (len(lens), heads, dv)), (torch.float32, (len(lens), heads))])
    stress(hsp, consumer, buf, lambda: hsp.paged_attention(q, k, v, table, ln, 0.07, out=out, lse=lse, return_lse=True))


@pytest.mark.parametrize("tokens", [3, 600])
def test_append(hsp, consumer, tokens):  # noqa: F811
    page, width = 64, 2
    buf, (k, v, q_out) = parts([(BF, (2 * width * 5 + 1, page, 2, 128)), (BF, (2 * width * 5 + 1, page, 2, 128)), (BF, (tokens, 4, 128))])
    table = torch.randperm(10 * width, device="cuda").to(torch.int32).view(10, width).contiguous()
    lens = torch.full((10,), page * width, dtype=torch.int32, device="cuda")
    at = torch.randperm(10 * page * width, device="cuda")[:tokens].to(torch.int32)
    kn, vn, q = (torch.randn(tokens, h, 128, device="cuda").to(BF) for h in (2, 2, 4))
    cs = torch.randn(page * width, 64, device="cuda")
    stress(hsp, consumer, buf, lambda: hsp.cache_append(kn, vn, k, v, table, lens, rows=at // (page * width), positions=at % (page * width),
                                                        cos_sin=cs, q=q, q_out=q_out))


# a request for one launch, and one that takes two (more pages than one launch serves)
@pytest.mark.parametrize("pages", [300, 4400])
@pytest.mark.parametrize("op", ["resize", "fork", "compact"])
def test_pages(hsp, consumer, op, pages):  # noqa: F811
    rows, width, page = 40, 8, 16
    buf, (table, lens, refs, pool, status) = parts([(torch.int32, (rows, width)), (torch.int32, (rows,)), (torch.int32, (pages,)),
                                                    (torch.int16, (2, pages, page, 8)), (torch.int32, (20,))])
    lens.zero_()
    refs.zero_()
    pool.copy_(torch.randint(-9, 9, pool.shape, device="cuda"))

    def ints(v):
        return torch.tensor(list(v), dtype=torch.int32, device="cuda")

    a = (table, lens, refs)
    hsp.cache_resize(*a, ints(range(20)), ints([37 + i for i in range(20)]), page, [pool])
    hsp.cache_fork(*a, ints(range(10)), ints(range(20, 30)), page)
    hsp.cache_resize(*a, ints(range(0, 20, 4)), ints([0] * 5), page, [pool])
    who, new = ints(range(10, 30)), ints([60 + i for i in range(20)])
    parent, child = ints(range(10, 20)), ints(range(30, 40))
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(hsp.cache_workspace_bytes(table, pages, 20), dtype=torch.uint8, device="cuda")
    stress(hsp, consumer, buf, {"resize": lambda: hsp.cache_resize(*a, who, new, page, [pool], status=status, workspace=ws),
                                "fork": lambda: hsp.cache_fork(*a, parent, child, page, status=status[:10]),
                                "compact": lambda: hsp.cache_compact(*a, page, [pool], live=live, workspace=ws)}[op],
           replays=REPLAYS // 4)


def test_copy(hsp, consumer):  # noqa: F811
    buf, (pool,) = parts([(torch.int16, (1, 300, 16, 16))])
    pool.copy_(torch.randint(-9, 9, pool.shape, device="cuda"))
    src, dst = list(range(0, 100)), list(range(100, 200))
    stress(hsp, consumer, buf, lambda: hsp.cache_copy_pages([pool], src, dst))
