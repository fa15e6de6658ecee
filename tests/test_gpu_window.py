"""GPU parity of windowed attention with sink tokens (quest_window_decode and
quest_window_prefill) against the plain 64-bit form, through the C ABI."""
import pytest
import torch

import query_aware_kv_gb300 as q
import span_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(0)
BIG = 2 ** 31 - 1


def make(lens, hq, hkv, P, extra_pages=1, seed=0, junk=float("nan")):
    """A paged cache with these lengths; every slot that holds no token is junk."""
    g = torch.Generator().manual_seed(seed)
    B, mp = len(lens), max(-(-max(lens) // P), 1) + extra_pages
    nph = B * mp + 2
    k = torch.randn((nph, hkv, P, 128), generator=g).half()
    v = torch.randn((nph, hkv, P, 128), generator=g).half()
    bt = torch.randperm(nph, generator=g)[:B * mp].view(B, mp).int()
    free = torch.ones((nph, P), dtype=torch.bool)
    for b, L in enumerate(lens):
        for p in range(-(-L // P)):
            free[bt[b, p], :min(P, L - p * P)] = False
    k.masked_fill_(free[:, None, :, None], junk)
    v.masked_fill_(free[:, None, :, None], junk)
    return q.PagedCache.allocate_meta(k.cuda(), v.cuda(), bt.cuda(),
                                      torch.tensor(lens, dtype=torch.int32).cuda(), hq)


def logical(cache, b, g, name):
    L, P = int(cache.seq_lens[b]), cache.page_size
    pool = getattr(cache, name)
    phys = cache.block_table[b, :-(-L // P)].long().clamp(min=0)
    return pool[phys, g].reshape(-1, 128)[:L]


def check(cache, qq, out, lse, sink, window, prompt):
    """qq, out [B, n, Hq, 128], lse [B, n, Hq]."""
    B, n, hq, _ = qq.shape
    G = hq // cache.num_kv_heads
    for b in range(B):
        L = int(cache.seq_lens[b])
        allowed = R.window_mask(L, n, sink, window, qq.device)
        for g in range(cache.num_kv_heads):
            k, v = logical(cache, b, g, "k_pool"), logical(cache, b, g, "v_pool")
            for h in range(g * G, g * G + G):
                R.assert_close(out[b, :, h], lse[b, :, h], R.attend(qq[b, :, h], k, v, allowed), prompt,
                               f"sequence {b} head {h} (L {L}, sink {sink}, window {window})")


def ok(ws):
    rc, detail = q.read_status(ws)
    assert rc == 0, (rc, detail)


GEOMS = [(4, 4, 16), (8, 1, 32), (8, 2, 16), (6, 3, 32)]
WINDOWS = [(0, 1), (4, 7), (0, 64), (1, 100), (40, 33), (17, 1000), (300, 5), (4, BIG), (BIG, 1)]


@pytest.mark.parametrize("geom", GEOMS, ids=str)
@pytest.mark.parametrize("sink,window", WINDOWS)
def test_decode(geom, sink, window):
    hq, hkv, P = geom
    lens = [0, 1, P - 1, P, P + 1, 333, 1025]
    cache = make(lens, hq, hkv, P, seed=window % 97)
    ws = q.window_workspace(cache)
    qq = torch.randn((len(lens), hq, 128), device="cuda").half()
    out, lse = q.window_decode(cache, qq, sink, window, ws)
    ok(ws)
    check(cache, qq[:, None], out[:, None], lse[:, None], sink, window, False)


@pytest.mark.parametrize("n", [1, 2, 5, 31, 64, 130, 257, 400])
@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_prompt(geom, n):
    """Chunks behind a context, sequences shorter than the chunk (empty rows), windows that
    end inside pages, sinks that meet the window."""
    hq, hkv, P = geom
    lens = [0, 1, P, 77, 300, 645]
    cache = make(lens, hq, hkv, P, seed=n)
    ws = q.window_workspace(cache, n)
    qq = torch.randn((len(lens), n, hq, 128), device="cuda").half()
    for sink, window in WINDOWS:
        out, lse = q.window_prefill(cache, qq, sink, window, ws)
        ok(ws)
        check(cache, qq, out, lse, sink, window, True)


def test_prompt_equals_decode_token_by_token():
    """A chunk's last row is what window_decode gives for the last token."""
    cache = make([500, 900], 8, 2, 16, seed=5)
    ws = q.window_workspace(cache, 70)
    qq = torch.randn((2, 70, 8, 128), device="cuda").half()
    po, pl = q.window_prefill(cache, qq, 4, 120, ws)
    do, dl = q.window_decode(cache, qq[:, -1].contiguous(), 4, 120, ws)
    ok(ws)
    torch.testing.assert_close(po[:, -1], do, atol=2e-3, rtol=2e-3)
    torch.testing.assert_close(pl[:, -1], dl, atol=1e-4, rtol=1e-5)


def test_a_window_as_long_as_the_sequence_is_dense_attention():
    cache = make([777, 40], 8, 4, 16, seed=6)
    ws = q.window_workspace(cache)
    dws = q.workspace(cache, 1)
    qq = torch.randn((2, 8, 128), device="cuda").half()
    out, lse = q.window_decode(cache, qq, 0, 777, ws)
    ref, ref_lse = q.dense_decode(cache, qq, dws)
    torch.testing.assert_close(out, ref, atol=1e-3, rtol=1e-3)
    torch.testing.assert_close(lse, ref_lse, atol=1e-4, rtol=1e-5)


@pytest.mark.parametrize("pps", [1, 3, 100])
@pytest.mark.parametrize("n", [1, 3, 200])
def test_splits(pps, n):
    """The long axis split over work items, more of them than a short row has pages."""
    lens = [5, 700, 2000]
    cache = make(lens, 8, 2, 16, seed=8)
    o = q.opts(pages_per_split=pps)
    ws = q.window_workspace(cache, n, o)
    qq = torch.randn((3, n, 8, 128), device="cuda").half()
    for sink, window in [(4, 1500), (0, 20), (100, 100)]:
        out, lse = q.window_prefill(cache, qq, sink, window, ws, o)
        ok(ws)
        check(cache, qq, out, lse, sink, window, True)


def test_pages_behind_the_window_may_be_unmapped():
    P, sink, window, L, n = 16, 20, 100, 1000, 40
    cache = make([L], 4, 4, P, seed=9)
    first = (L - n - window + 1) // P
    keep = logical(cache, 0, 0, "k_pool").clone()
    ws = q.window_workspace(cache, n)
    qq = torch.randn((1, n, 4, 128), device="cuda").half()
    want, want_lse = q.window_prefill(cache, qq, sink, window, ws)
    want, want_lse = want.clone(), want_lse.clone()
    cache.block_table[0, -(-sink // P):first] = -1
    cache.block_table[0, -(-L // P):] = -1
    out, lse = q.window_prefill(cache, qq, sink, window, ws)
    ok(ws)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    one, _ = q.window_decode(cache, qq[:, -1].contiguous(), sink, window, ws)
    ok(ws)
    torch.testing.assert_close(one, want[:, -1], atol=2e-3, rtol=2e-3)
    assert keep.shape[0] == L


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")], ids=str)
def test_hidden_tokens_do_not_reach_a_result(value):
    """Keys and values that no query of the call sees, in pages that are read: between the
    sinks and the window."""
    P, sink, window, L = 32, 5, 70, 500
    for n in (1, 9):
        cache = make([L], 8, 2, P, seed=10)
        lo = L - n - window + 1
        for t in list(range(sink, P)) + list(range(lo // P * P, lo)):
            phys = int(cache.block_table[0, t // P])
            cache.k_pool[phys, :, t % P] = value
            cache.v_pool[phys, :, t % P] = value
        ws = q.window_workspace(cache, n)
        qq = torch.randn((1, n, 8, 128), device="cuda").half()
        out, lse = q.window_prefill(cache, qq, sink, window, ws)
        ok(ws)
        check(cache, qq, out, lse, sink, window, True)


@pytest.mark.parametrize("n", [40, 300])
@pytest.mark.parametrize("pps", [0, 3])
def test_odd_values_reach_only_the_rows_that_see_them(n, pps):
    """A NaN and an infinity among the values: rows before them, and rows whose window has
    passed them, are as if they were 0; the others are not finite there."""
    sink, window, L = 3, 70, 700
    cache = make([L], 8, 2, 16, seed=14)
    o = q.opts(pages_per_split=pps)
    ws = q.window_workspace(cache, n, o)
    qq = torch.randn((1, n, 8, 128), device="cuda").half()
    clean = cache.v_pool.clone()
    at = [(L - n + 9, 5, float("nan")), (L - 25, 77, float("inf"))]
    for t, d, value in at:
        cache.v_pool[int(cache.block_table[0, t // 16]), :, t % 16, d] = value
    out, lse = q.window_prefill(cache, qq, sink, window, ws, o)
    ok(ws)
    cache.v_pool.copy_(clean)
    for t, d, _ in at:
        cache.v_pool[int(cache.block_table[0, t // 16]), :, t % 16, d] = 0
    allowed = R.window_mask(L, n, sink, window, "cuda")
    for g in range(2):
        k, v = logical(cache, 0, g, "k_pool"), logical(cache, 0, g, "v_pool")
        for h in range(g * 4, g * 4 + 4):
            got = out[0, :, h].clone()
            ref = R.attend(qq[0, :, h], k, v, allowed)
            for t, d, _ in at:
                sees = allowed[:, t]
                assert not torch.isfinite(got[sees, d]).any()
                assert torch.isfinite(got[~sees, d]).all()
                got[sees, d] = ref[0][sees, d].half()
            R.assert_close(got, lse[0, :, h], ref, True)


def test_odd_values_in_a_share_that_a_row_does_not_see():
    """The K / V axis split: rows that see nothing of a split's tokens, NaN among which other
    rows see, are as if the NaN were 0."""
    n, window, L = 250, 40, 900
    cache = make([L], 2, 2, 16, seed=15)
    o = q.opts(pages_per_split=8)  # 128 tokens a split
    ws = q.window_workspace(cache, n, o)
    qq = torch.randn((1, n, 2, 128), device="cuda").half()
    slot = (int(cache.block_table[0, (L - 1) // 16]), slice(None), (L - 1) % 16)
    clean = cache.v_pool[slot].clone()
    cache.v_pool[slot] = float("nan")
    out, lse = q.window_prefill(cache, qq, 0, window, ws, o)
    ok(ws)
    assert torch.isnan(out[0, -1]).all()
    cache.v_pool[slot] = clean
    want, want_lse = q.window_prefill(cache, qq, 0, window, ws, o)
    ok(ws)
    assert torch.equal(lse, want_lse)
    out[0, -1] = want[0, -1]
    check(cache, qq, out, lse, 0, window, True)


def test_large_scores_and_values():
    """Scores far from 0 (both signs) and a maximum that comes last: the running maximum
    moves, small weights vanish."""
    cache = make([600], 4, 4, 16, seed=11, junk=0.0)
    ramp = torch.linspace(0.1, 6, cache.k_pool.shape[0], device="cuda").half()
    cache.k_pool.mul_(ramp[:, None, None, None])
    cache.v_pool.mul_(100)
    for n in (1, 150):
        ws = q.window_workspace(cache, n)
        qq = (torch.randn((1, n, 4, 128), device="cuda") * 4).half()
        out, lse = q.window_prefill(cache, qq, 4, 333, ws)
        ok(ws)
        check(cache, qq, out, lse, 4, 333, True)


def test_long_prompt_in_chunks():
    """A whole prompt, written and attended chunk by chunk, equals one call."""
    hq, hkv, P, n = 8, 4, 16, 1200
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((2, n, hkv, 128), device="cuda", generator=g).half() for _ in range(2))
    qq = torch.randn((2, n, hq, 128), device="cuda", generator=g).half()

    def run(chunks):
        cache = make([0, 0], hq, hkv, P, extra_pages=n // P + 1)
        pws, ws = q.workspace(cache, 1), q.window_workspace(cache, n)
        outs, at = [], 0
        for m in chunks:
            q.prefill(cache, k[:, at:at + m].contiguous(), v[:, at:at + m].contiguous(), pws)
            outs.append(q.window_prefill(cache, qq[:, at:at + m].contiguous(), 4, 256, ws))
            at += m
        ok(ws)
        return cache, torch.cat([o for o, _ in outs], 1), torch.cat([z for _, z in outs], 1)

    cache, one, one_lse = run([n])
    check(cache, qq, one, one_lse, 4, 256, True)
    cache, many, many_lse = run([1, 500, 16, 3, 680])
    check(cache, qq, many, many_lse, 4, 256, True)


def test_streams_graphs_and_reuse():
    """On a side stream, replayed from a graph with new inputs in place, and twice on one
    workspace."""
    cache = make([900, 300], 8, 2, 16, seed=12)
    ws = q.window_workspace(cache, 33)
    q1 = torch.randn((2, 8, 128), device="cuda").half()
    qn = torch.randn((2, 33, 8, 128), device="cuda").half()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        plan = q.WindowPlan(cache, 4, 200, ws)
        out = torch.empty_like(qn)
        lse = torch.empty(qn.shape[:3], device="cuda")
        for _ in range(2):
            plan.decode(q1)
            q.window_prefill(cache, qn, 4, 200, ws, out=out, lse=lse)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        gplan = q.WindowPlan(cache, 4, 200, ws)
        gplan.decode(q1)
        q.window_prefill(cache, qn, 4, 200, ws, out=out, lse=lse)
    for _ in range(3):
        q1.copy_(torch.randn_like(q1))
        qn.copy_(torch.randn_like(qn))
        graph.replay()
        torch.cuda.synchronize()
        ok(ws)
        check(cache, q1[:, None], gplan.out[:, None], gplan.lse[:, None], 4, 200, False)
        check(cache, qn, out, lse, 4, 200, True)


def test_faults_are_reported():
    cache = make([100, 50], 4, 2, 16, seed=13)
    cache.block_table[1, 2] = cache.k_pool.shape[0]
    qq = torch.randn((2, 3, 4, 128), device="cuda").half()
    ws = q.window_workspace(cache, 3)
    q.window_prefill(cache, qq, 0, 10, ws)
    rc, detail = q.read_status(ws)
    assert rc == q.QUEST_ERR_BAD_PAGE and detail[:2] == (1, 2)
    q.workspace_init(ws)
    cache.block_table[1, 2] = 0
    cache.seq_lens[0] = -5
    q.window_decode(cache, qq[:, 0].contiguous(), 0, 10, ws)
    rc, detail = q.read_status(ws)
    assert rc == q.QUEST_ERR_BAD_LENGTH and detail[0] == 0


def test_empty_batch_and_no_lse():
    cache = make([64], 4, 4, 16)
    ws = q.window_workspace(cache, 2)
    qq = torch.randn((1, 2, 4, 128), device="cuda").half()
    a, z = q.window_prefill(cache, qq, 0, 9, ws, want_lse=False)
    assert z is None
    b, _ = q.window_prefill(cache, qq, 0, 9, ws)
    assert torch.equal(a, b)
    out, lse = q.window_prefill(cache, qq[:, :0].contiguous(), 0, 9, ws)
    assert out.numel() == 0 and lse.numel() == 0


def test_offsets_past_32_bits():
    """Pages beyond the first 4 GiB of each pool, and the last page of it."""
    hkv, P, hq, L, n = 8, 32, 16, 300, 20
    nph = (5 << 30) // (hkv * P * 128 * 2)
    k = torch.empty((nph, hkv, P, 128), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    pages = -(-L // P)
    bt = torch.arange(nph - pages, nph, device="cuda").int().flip(0)[None].contiguous()
    k[-pages:] = torch.randn((pages, hkv, P, 128), device="cuda").half()
    v[-pages:] = torch.randn((pages, hkv, P, 128), device="cuda").half()
    cache = q.PagedCache.allocate_meta(k, v, bt, torch.tensor([L], dtype=torch.int32).cuda(), hq)
    ws = q.window_workspace(cache, n)
    qq = torch.randn((1, n, hq, 128), device="cuda").half()
    out, lse = q.window_prefill(cache, qq, 4, 90, ws)
    ok(ws)
    check(cache, qq, out, lse, 4, 90, True)
    out, lse = q.window_decode(cache, qq[:, -1].contiguous(), 4, 90, ws)
    ok(ws)
    check(cache, qq[:, -1:], out[:, None], lse[:, None], 4, 90, False)


@pytest.mark.parametrize("batch,hkv", [(20, 8), (70, 16)], ids=["160_rows", "1120_rows"])
def test_many_rows(batch, hkv):
    """More rows than SMs (CTAs of four warps), and more than are ever split."""
    lens = [(37 * b) % 211 for b in range(batch)]
    cache = make(lens, hkv, hkv, 16, seed=15)
    ws = q.window_workspace(cache)
    qq = torch.randn((batch, hkv, 128), device="cuda").half()
    out, lse = q.window_decode(cache, qq, 3, 50, ws)
    ok(ws)
    check(cache, qq[:, None], out[:, None], lse[:, None], 3, 50, False)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (6, 3), (8, 2), (8, 1)])
@pytest.mark.parametrize("window", [600, 5000, 12000])
def test_a_row_over_many_work_items(hq, hkv, window):
    """Rows that a few work items share, those that many do, and one that sees one token."""
    lens = [12500, 1]
    cache = make(lens, hq, hkv, 16, seed=17)
    ws = q.window_workspace(cache)
    qq = torch.randn((2, hq, 128), device="cuda").half()
    out, lse = q.window_decode(cache, qq, 4, window, ws)
    ok(ws)
    check(cache, qq[:, None], out[:, None], lse[:, None], 4, window, False)


@pytest.mark.parametrize("hq,hkv,pps", [(8, 1, 2), (8, 1, 0), (4, 2, 1), (1, 1, 3)])
def test_many_split_rows(hq, hkv, pps):
    """More rows than SMs, each over several work items."""
    batch = 200
    lens = [(37 * b) % 411 for b in range(batch)]
    cache = make(lens, hq, hkv, 16, seed=18)
    o = q.opts(pages_per_split=pps)
    ws = q.window_workspace(cache, 1, o)
    qq = torch.randn((batch, hq, 128), device="cuda").half()
    out, lse = q.window_decode(cache, qq, 3, 350, ws, o)
    ok(ws)
    check(cache, qq[:, None], out[:, None], lse[:, None], 3, 350, False)


def test_one_workspace_for_every_length():
    """A workspace sized for a long chunk serves shorter ones, split or not, in any order."""
    cache = make([1500, 800], 8, 2, 16, seed=16)
    ws = q.window_workspace(cache, 600)
    for n in (600, 1, 7, 300, 1, 600, 40):
        qq = torch.randn((2, n, 8, 128), device="cuda").half()
        out, lse = q.window_prefill(cache, qq, 4, 900, ws)
        ok(ws)
        check(cache, qq, out, lse, 4, 900, True)
