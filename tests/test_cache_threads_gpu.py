"""The paged cache's Python calls from several host threads at once (they release the interpreter lock), each with a
cache and a stream of its own: every step has the bits of the same run made alone."""
import threading

import pytest
import torch

from test_cache_gpu import BF, hsp  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu
STEPS = 40


def run(hsp, kind, seed, errors=None):  # noqa: F811
    """A decode run of its own; returns what it computed."""
    latent, heads, kv, dk, page = kind
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, width, pages = 6, 40, 200
    k = torch.zeros(1, pages, page, kv, dk, dtype=BF, device="cuda")
    v = None if latent else torch.zeros_like(k)
    pools = [k] if latent else [k, v]
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    a = (table, lens, refs)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    r, fork, zero = ints([0, 2, 4]), (ints([0, 2]), ints([1, 3])), ints([0, 0])
    start = ints([page * 3 + 1, 5, 300 + seed % 7])
    hsp.cache_resize(*a, r, start, page, pools)
    k.copy_(torch.randn(k.shape, generator=g, device="cuda"))
    got = []
    for step in range(STEPS):
        new = lens[r.long()] + 1
        hsp.cache_resize(*a, r, new, page, pools)
        kn = torch.randn(3, kv, dk, generator=g, device="cuda").to(BF)
        q = torch.randn(3, heads, dk, generator=g, device="cuda").to(BF)
        hsp.cache_append(kn, None if latent else kn, k[0], None if latent else v[0], table, lens, rows=r, positions=new - 1)
        got += hsp.paged_attention(q, k[0], None if latent else v[0], table, lens, 0.07, rows=r, return_lse=True)
        if step % 10 == 4:
            got.append(hsp.cache_fork(*a, *fork, page))
        if step % 10 == 7:
            got.append(hsp.cache_resize(*a, fork[1], zero, page, pools))
            got.append(hsp.cache_compact(*a, page, pools))
        if step % 10 == 8:
            hsp.cache_copy_pages(pools, [0], [pages - 1])
        if errors is not None and step % 3 == 0:              # a refused call of this thread: its own text
            try:
                hsp.cache_copy_pages(pools, [seed], [seed])
                errors.append("not refused")
            except hsp.ProjError as e:
                if f"page {seed} is a source and a destination" not in str(e):
                    errors.append(str(e))
    return got + [table, lens, refs, *pools]


KINDS = [(True, 16, 1, 576, 64), (False, 8, 2, 128, 16), (True, 64, 1, 512, 32), (False, 40, 2, 64, 64)]


def test_threads(hsp):  # noqa: F811
    want = [run(hsp, kind, 10 + i) for i, kind in enumerate(KINDS)]
    torch.cuda.synchronize()
    hsp.check_device_error()
    got, errors, barrier = [None] * len(KINDS), [], threading.Barrier(len(KINDS))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            barrier.wait()
            with torch.cuda.stream(stream):
                for _ in range(4):
                    got[i] = run(hsp, KINDS[i], 10 + i, errors)
                    stream.synchronize()
        except Exception as e:  # noqa: BLE001 -- reported below
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(KINDS))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    hsp.check_device_error()
    assert not errors, errors[:5]
    for i in range(len(KINDS)):
        assert all(torch.equal(x, y) for x, y in zip(got[i], want[i])), KINDS[i]
