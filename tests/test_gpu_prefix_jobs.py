"""Shared-prefix attention: what a job of the queue may and may not depend on."""
import pytest
import torch

import query_aware_kv_gb300 as q
import span_reference as R
from test_gpu_prefix import BIG, INF, make, queries
from test_gpu_window import logical, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(0)


def growing(cache, groups, by=4.0):
    """Keys of a sequence's own tokens that grow with their position: the maxima move after a job's
    first tile too."""
    P, b = cache.page_size, 0
    for count, prefix in groups:
        for _ in range(count):
            own = cache.block_table[b, prefix // P:].long()
            up = 0.5 + by * torch.arange(len(own), device="cuda") / len(own)
            cache.k_pool[own] = (cache.k_pool[own].float() * up[:, None, None, None]).half()
            b += 1
    return cache


@pytest.mark.parametrize("geom,n", [((32, 8, 16), None), ((8, 8, 32), None), ((16, 8, 16), 3)], ids=str)
def test_the_same_bits_every_time_with_default_splits(geom, n):
    """Tails of several tiles behind several prefixes, more jobs than CTAs, which take them in any
    order: no bit of a result depends on what a CTA did before."""
    G = geom[0] // geom[1]
    cache, groups = make([(2048, [2048 + 700 + 17 * i for i in range(128 // G)]),
                          (1600, [1600 + 400 + 9 * i for i in range(20)])], *geom)
    growing(cache, groups)
    shape = (cache.batch, geom[0], 128) if n is None else (cache.batch, n, geom[0], 128)
    # (the rows of either group move their maxima at other tiles)
    qq = torch.randn(shape, device="cuda") * torch.linspace(0.2, 6, cache.batch, device="cuda").view(-1, *[1] * (len(shape) - 1))
    qq = qq.half()
    ws = q.prefix_workspace(cache, groups, None, n or 1)
    plan = q.PrefixPlan(cache, groups, ws, n_tokens=n)
    first = [t.clone() for t in plan.decode(qq)]
    for _ in range(40):
        out, lse = plan.decode(qq)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    ok(ws)


@pytest.mark.parametrize("geom", [(32, 8, 16), (8, 8, 32)], ids=str)
def test_a_sequence_does_not_depend_on_the_batch_beside_it(geom):
    """Large queries of a prefix's rows stay in shared memory behind a tail's few rows: the tails of
    the sequences beside that group are the same bits whatever they are."""
    G = geom[0] // geom[1]
    cache, groups = make([(2048, [2100] * (128 // G)), (0, [1100 + 50 * i for i in range(24)])], *geom)
    growing(cache, groups, 2.0)
    alone = slice(128 // G, None)
    qq = queries(cache)
    plan = q.PrefixPlan(cache, groups, q.prefix_workspace(cache, groups))
    want = [t[alone].clone() for t in plan.decode(qq)]
    for scale in (0.0, 8.0, 60.0):
        other = qq.clone()
        other[:128 // G] = torch.randn_like(other[:128 // G]) * scale
        for _ in range(8):
            out, lse = plan.decode(other)
            assert torch.equal(out[alone], want[0]) and torch.equal(lse[alone], want[1]), scale


def close_to_64_bits(cache, qq, out, lse, rows, skip=()):
    """The sequences `rows`; dims `skip` are not looked at."""
    n, hq = qq.shape[1:3]
    G = hq // cache.num_kv_heads
    dims = [d for d in range(128) if d not in skip]
    for b in rows:
        L = int(cache.seq_lens[b])
        allowed = R.window_mask(L, n, 0, BIG, "cuda")
        for h in range(hq):
            k, v = logical(cache, b, h // G, "k_pool"), logical(cache, b, h // G, "v_pool")
            ref = R.attend(qq[b, :, h], k, torch.where(torch.isinf(v), 0.0, v), allowed)
            ref = (ref[0][:, dims], ref[1], ref[2][:, dims], ref[3])
            R.assert_close(out[b, :, h][:, dims], lse[b, :, h], ref, True, f"{b} {h}")


def test_a_short_limit_is_no_limit_on_the_product_that_other_warps_hold_up():
    """All rows of a job are taken again by the warps of one half, while the other half's are at the
    next job, whose maxima move at its second tile: their wait for the product of its first tile is a
    wait for the warps that are late.  (A sequence's 16 tokens of 8 heads are a job's 128 rows, and
    there are two jobs a CTA.)"""
    tokens, n = 8192, 16
    cache, groups = make([(tokens, [tokens + 40] * 304)], 8, 1, 32)
    for page in range(tokens // 32):  # (scores of the second tile: 14 in 2^x where the first had 1)
        cache.k_pool[int(cache.block_table[0, page])] *= 0.25 if page < 4 else 4.0
    at = int(cache.block_table[0, 3])
    cache.v_pool[at, :, 5, 9] = INF
    qq = torch.randn((304, n, 8, 128), device="cuda").half()
    long = q.opts(pages_per_split=16384)
    ws = q.prefix_workspace(cache, groups, long, n)
    want, want_lse = q.prefix_decode(cache, qq, groups, ws, long)
    ok(ws)
    short = q.opts(pages_per_split=16384, wait_limit_ns=300_000)
    for _ in range(3):
        out, lse = q.prefix_decode(cache, qq, groups, ws, short)
        ok(ws)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert bool((want[..., 9] == INF).all())
    close_to_64_bits(cache, qq, want, want_lse, (0, 151, 303), skip=(9,))


def test_the_longest_job_may_be_taken_again():
    """Rows of 512K tokens in one job each, two jobs a CTA.  An infinite value of the first sequences
    makes their 32 rows be taken again, a token at a time and for longer than a second: what waits for
    them waits as long as they move on."""
    B, n, P, pages = 304, 4, 32, 16384
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((pages + 4, 1, P, 128), generator=g, device="cuda", dtype=torch.float16) for _ in "kv")
    bt = torch.arange(pages, device="cuda", dtype=torch.int32).repeat(B, 1)
    for b in range(4):  # (a page of their own; the others hold the same ones without being a group)
        bt[b, 7] = pages + b
    lens = torch.full((B,), pages * P, dtype=torch.int32, device="cuda")
    cache = q.PagedCache.allocate_meta(k, v, bt, lens, 8)
    v[pages:, :, 5, 9] = INF
    qq = torch.randn((B, n, 8, 128), device="cuda", generator=g, dtype=torch.float16)
    groups = [(B, 0)]
    o = q.opts(pages_per_split=pages)
    ws = q.prefix_workspace(cache, groups, o, n)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    out, lse = q.prefix_decode(cache, qq, groups, ws, o)
    end.record()
    ok(ws)
    assert start.elapsed_time(end) > 1000  # (or the test shows nothing)
    assert bool((out[:4, ..., 9] == INF).all()) and bool(torch.isfinite(out[4:]).all())
    close_to_64_bits(cache, qq, out, lse, (0, 4), skip=(9,))


@pytest.mark.parametrize("batch,hkv,tokens", [(4, 8, 20000), (24, 1, 700), (11, 2, 30000), (15, 4, 9000), (28, 1, 3000)])
def test_unshared_rows_are_split_as_a_window_decodes_are(batch, hkv, tokens):
    """Nothing shared: long rows, and any number of rows whose CTAs fit the GPU at once, take the split
    that the span decode chooses for a window over everything, and so its bits."""
    g = torch.Generator(device="cuda").manual_seed(batch)
    lens = [tokens - (3 * tokens * b) // (4 * batch) for b in range(batch)]
    mp = -(-tokens // 16) + 1
    k, v = (torch.randn((batch * mp, hkv, 16, 128), generator=g, device="cuda", dtype=torch.float16) for _ in "kv")
    bt = torch.randperm(batch * mp, generator=g, device="cuda").view(batch, mp).int()
    cache = q.PagedCache.allocate_meta(k, v, bt, torch.tensor(lens, dtype=torch.int32).cuda(), 4 * hkv)
    qq = torch.randn((batch, 4 * hkv, 128), generator=g, device="cuda", dtype=torch.float16)
    groups = [(batch, 0)]
    ws, wws = q.prefix_workspace(cache, groups), q.window_workspace(cache)
    out, lse = q.prefix_decode(cache, qq, groups, ws)
    want, want_lse = q.window_decode(cache, qq, 0, BIG, wws)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    ok(ws), ok(wws)
