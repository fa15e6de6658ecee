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
