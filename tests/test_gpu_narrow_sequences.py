"""GPU tests of calls on a narrow (8-bit) cache that follow one another on the stream with nothing
between them, and of its decode steps beside the fp16 cache's."""
import pytest
import torch

import query_aware_kv_gb300 as q
import span_reference as R
from test_gpu_narrow import assert_cache, empty, ok, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunk", [1, 7, 16, 40])
def test_chunks_back_to_back(chunk):
    """Chunks written with nothing between them on the stream: each begins at the length that the
    one before it left, and over the open page that it left."""
    hkv, P, n = 6, 16, 640 // chunk
    cache = empty(3, hkv, hkv, P, 642 // P + 1, seed=chunk)
    ws = q.narrow_workspace(cache)
    k, v = tokens(3, n * chunk, hkv, seed=51)
    parts = [(k[:, i * chunk:(i + 1) * chunk].contiguous().cuda(),
              v[:, i * chunk:(i + 1) * chunk].contiguous().cuda()) for i in range(n)]
    torch.cuda.synchronize()
    for kc, vc in parts:
        q.narrow_prefill(cache, kc, vc, ws)
    ok(ws)
    ref = R.NarrowReference(3, hkv, P)
    ref.write(k, v)
    assert_cache(cache, ref)


def test_a_table_that_changes_between_chunks():
    """A chunk sees the entries that a copy just before it on the stream has written: those of the
    pages that it fills, and of the page that it leaves open."""
    hkv, P, n = 2, 16, 37
    cache = empty(1, hkv, hkv, P, 24, seed=6)
    ws = q.narrow_workspace(cache)
    mapped = cache.block_table.clone()
    cache.block_table.fill_(-1)
    k, v = tokens(1, 8 * n, hkv, seed=52)
    parts = [(k[:, i * n:(i + 1) * n].contiguous().cuda(), v[:, i * n:(i + 1) * n].contiguous().cuda())
             for i in range(8)]
    torch.cuda.synchronize()
    for i, (kc, vc) in enumerate(parts):
        upto = ((i + 1) * n + P - 1) // P
        cache.block_table[:, :upto].copy_(mapped[:, :upto])
        q.narrow_prefill(cache, kc, vc, ws)
    ok(ws)
    ref = R.NarrowReference(1, hkv, P)
    ref.write(k, v)
    assert_cache(cache, ref)


def test_calls_on_two_streams_at_once():
    """Prompt chunks, decode over split rows and narrow steps on two streams, each stream with its
    own caches and workspaces: the same bits as one after the other."""
    def state(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        mp = 130
        pools = [torch.randn((2 * mp, 4, 16, 128), device="cuda", generator=g).half() for _ in range(2)]
        bt = torch.randperm(2 * mp, device="cuda", generator=g).view(2, mp).int()
        lens = torch.tensor([2050, 1234], dtype=torch.int32, device="cuda")
        paged = q.PagedCache.allocate_meta(*pools, bt, lens, 8)
        narrow = q.NarrowCache.allocate(2 * mp, 4, 16, bt, torch.zeros(2, dtype=torch.int32, device="cuda"), 8)
        kv = torch.randn((2, 2, 700, 4, 128), device="cuda", generator=g).half()
        return dict(paged=paged, narrow=narrow, wws=q.window_workspace(paged, 400), nws=q.narrow_workspace(narrow, 12),
                    kv=kv, qn=torch.randn((2, 400, 8, 128), device="cuda", generator=g).half(),
                    q1=torch.randn((8, 2, 8, 128), device="cuda", generator=g).half(),
                    new=torch.randn((8, 2, 2, 4, 128), device="cuda", generator=g).half())

    def work(s):
        got = []
        q.narrow_prefill(s["narrow"], s["kv"][0], s["kv"][1], s["nws"])
        for i in range(8):
            n = (400, 7, 33, 250)[i % 4]
            got += q.window_prefill(s["paged"], s["qn"][:, :n].contiguous(), 4, 1500, s["wws"])
            got += q.window_decode(s["paged"], s["q1"][i], 4, 1900, s["wws"])
            got += q.narrow_decode_step(s["narrow"], s["q1"][i], s["new"][i, 0], s["new"][i, 1], 12, s["nws"])
        return got

    want = [work(state(seed)) for seed in (1, 2)]
    torch.cuda.synchronize()
    states = [state(seed) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    got = []
    for s, stream in zip(states, streams):
        with torch.cuda.stream(stream):
            got.append(work(s))
    torch.cuda.synchronize()
    for s, a, b in zip(states, got, want):
        ok(s["nws"])
        ok(s["wws"])
        for x, y in zip(a, b):
            assert torch.equal(x, y)
