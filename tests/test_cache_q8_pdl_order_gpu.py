"""Programmatic-dependent-launch ordering of the kernels of the 8-bit cache, on both sides.  Behind them: a consumer
that never waits on its grid dependency reads final values (as test_cache_pdl_order_gpu.py has it).  In front: the
kernels read inputs that were written right before the call, at addresses where they read other values the call before;
the attention among them, which starts while the kernel that splits its queries runs."""
import pytest
import torch

from test_cache_pdl_order_gpu import parts, stress
from test_pdl_order_gpu import PER_GRAPH, REPLAYS, consumer, hsp  # noqa: F401  (the fixtures)

pytestmark = pytest.mark.gpu
BF, F8, I32, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.float32

# not cut; cut and joined, with 64 heads; many grouped sequences, some joined and some whole
ATTENTION = [([77, 200, 0], 16, 1, 576, 512), ([9000], 64, 1, 512, 512), ([1000, 30, 0, 2500, 64], 8, 2, 128, 128)]


@pytest.mark.parametrize("lens,heads,kv,dk,dv", ATTENTION)
def test_attention(hsp, consumer, lens, heads, kv, dk, dv):  # noqa: F811
    from test_attention_q8_gpu import make
    args = make(lens, heads, kv, dk, dv == 512, 64, 3)
    buf, (out, lse) = parts([(BF, (len(lens), heads, dv)), (F32, (len(lens), heads))])
    stress(hsp, consumer, buf, lambda: hsp.paged_attention_q8(*args, 0.07, out=out, lse=lse, return_lse=True))


# rows of 128 and 256 columns in runs; one latent head whose blocks several CTAs share
@pytest.mark.parametrize("tokens,kv,dk,dv,heads", [(3, 2, 128, 128, 4), (600, 2, 128, 128, 4), (600, 2, 128, 128, 0), (520, 1, 576, None, 0),
                                                   (520, 1, 576, None, 6)])
def test_append(hsp, consumer, tokens, kv, dk, dv, heads):  # noqa: F811
    page, width, block = 64, 2, 32
    pages = 2 * width * 5 + 1
    g = torch.Generator(device="cuda").manual_seed(tokens)
    sides = [(F8, (pages, page, kv, dk)), (F32, (pages, page // block, kv))] + ([(F8, (pages, page, kv, dv)), (F32, (pages, page // block, kv))] if dv else [])
    buf, views = parts(sides + ([(BF, (tokens, heads, dk))] if heads else []))
    k, ks = views[:2]
    v, vs = views[2:4] if dv else (None, None)
    for t in (k, v):
        if t is not None:
            t.view(torch.uint8).copy_(torch.randint(0, 100, t.shape, generator=g, device="cuda"))
    for t in (ks, vs):
        if t is not None:
            t.fill_(2.0 ** -12)
    table = torch.randperm(10 * width, generator=g, device="cuda").to(I32).view(10, width).contiguous()
    lens = torch.full((10,), page * width, dtype=I32, device="cuda")
    at = (torch.arange(tokens, device="cuda") * (10 * page * width) // tokens).to(I32)      # blocks with tokens in front and between
    kn, vn = (torch.randn(tokens, kv, d, generator=g, device="cuda").to(BF) if d else None for d in (dk, dv))
    q = torch.randn(tokens, heads, dk, generator=g, device="cuda").to(BF) if heads else None
    cs = torch.randn(page * width, 64, generator=g, device="cuda")
    stress(hsp, consumer, buf, lambda: hsp.cache_append_q8(kn, vn, k, v, ks, vs, table, lens, rows=at // (page * width), positions=at % (page * width),
                                                           cos_sin=cs, q=q, q_out=views[-1] if heads else None))


@pytest.mark.parametrize("tokens", [3, 600])
def test_read(hsp, consumer, tokens):  # noqa: F811
    from test_attention_q8_gpu import make
    lens = [tokens, 5]
    _, k, v, ks, vs, table, ln = make(lens, 4, 2, 128, False, 64, 5)
    buf, (ko, vo) = parts([(BF, (tokens, 2, 128)), (BF, (tokens, 2, 128))])
    rows, pos = torch.zeros(tokens, dtype=I32, device="cuda"), torch.arange(tokens, dtype=I32, device="cuda")
    stress(hsp, consumer, buf, lambda: hsp.cache_read_q8(k, v, ks, vs, table, ln, rows=rows, positions=pos, k_out=ko, v_out=vo))


def alternate(hsp, consumer, inputs, contents, outputs, call):  # noqa: F811
    """In a graph, in turn for every contents: they are written to the inputs, the call, and a consumer of its outputs."""
    want = []
    for c in contents:
        inputs.copy_(c)
        call()
        torch.cuda.synchronize()
        hsp.check_device_error()
        want.append(outputs.clone())
    assert not torch.equal(want[0], want[1])
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        stream = torch.cuda.current_stream().cuda_stream
        for _ in range(PER_GRAPH // 2):
            for c, w in zip(contents, want):
                inputs.copy_(c)
                call()
                assert consumer.pdl_consumer_launch(outputs.data_ptr(), w.data_ptr(), outputs.numel(), 0, counter.data_ptr(), stream) == 0
    for _ in range(REPLAYS // PER_GRAPH):
        g.replay()
    torch.cuda.synchronize()
    hsp.check_device_error()
    assert int(counter.item()) == 0


@pytest.mark.parametrize("lens,heads,kv,dk,dv", ATTENTION)
def test_inputs_of_the_attention(hsp, consumer, lens, heads, kv, dk, dv):  # noqa: F811
    from test_attention_q8_gpu import make
    sets = [[t for t in make(n, heads, kv, dk, dv == 512, 64, seed) if t is not None] for seed, n in ((3, lens), (4, lens[::-1]))]
    inputs, views = parts([(t.dtype, t.shape) for t in sets[0]])
    contents = []
    for s in sets:
        for to, t in zip(views, s):
            to.view(torch.uint8).copy_(t.view(torch.uint8)) if t.dtype == F8 else to.copy_(t)
        contents.append(inputs.clone())
    q, k, ks = views[0], views[1], views[2 if dv == 512 else 3]
    v, vs = (None, None) if dv == 512 else (views[2], views[4])
    table, ln = views[-2:]
    outputs, (out, lse) = parts([(BF, (len(lens), heads, dv)), (F32, (len(lens), heads))])
    alternate(hsp, consumer, inputs, contents, outputs, lambda: hsp.paged_attention_q8(q, k, v, ks, vs, table, ln, 0.07, out=out, lse=lse, return_lse=True))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("tokens", [3, 300])
def test_inputs_of_the_append(hsp, consumer, tokens, interleaved):  # noqa: F811
    page, kv, d, heads, rot = 64, 2, 128, 6, 64
    pages = -(-tokens // page) + 1
    inputs, (kn, vn, q, cs, rows, pos, table, ln) = parts([(BF, (tokens, kv, d)), (BF, (tokens, kv, d)), (BF, (tokens, heads, d)), (F32, (tokens, rot)),
                                                           (I32, (tokens,)), (I32, (tokens,)), (I32, (2, pages)), (I32, (2,))])
    contents = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (kn, vn, q, cs):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        rows.fill_(seed - 1)
        pos.copy_(torch.arange(tokens) if seed == 1 else torch.arange(tokens - 1, -1, -1))
        table.copy_(torch.randperm(2 * pages, generator=g, device="cuda").view(2, pages))
        ln.fill_(tokens)
        contents.append(inputs.clone())
    outputs, (k, v, ks, vs, q_out) = parts([(F8, (2 * pages, page, kv, d)), (F8, (2 * pages, page, kv, d)), (F32, (2 * pages, page // 16, kv)),
                                            (F32, (2 * pages, page // 16, kv)), (BF, (tokens, heads, d))])
    start = outputs.clone()

    def call():
        outputs.copy_(start)
        hsp.cache_append_q8(kn, vn, k, v, ks, vs, table, ln, rows=rows, positions=pos, cos_sin=cs, interleaved=interleaved, q=q, q_out=q_out)

    alternate(hsp, consumer, inputs, contents, outputs, call)
