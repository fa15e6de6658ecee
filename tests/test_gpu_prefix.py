"""Attention over prefixes that sequences share (quest_prefix_decode) against the plain 64-bit form,
and a serving step made of rotary writes and shared-prefix attention."""
import pytest
import torch

import query_aware_kv_gb300 as q
import rotary_reference as RR
import span_reference as R
from test_gpu_window import check, logical, ok

pytestmark = pytest.mark.gpu
BIG = 2 ** 31 - 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(0)


def make(groups, hq, hkv, P, seed=0, spare=3):
    """groups: (prefix tokens, [length of each sequence]).  A cache whose groups share their
    prefixes' whole pages; every slot that holds no token of any sequence is NaN."""
    g = torch.Generator().manual_seed(seed)
    lens = [L for _, ls in groups for L in ls]
    mp = max(max([*lens, *(p for p, _ in groups)]) // P + 1, 1)
    rows, free_page = [], 0
    for prefix, ls in groups:
        shared = list(range(free_page, free_page + prefix // P))
        free_page += len(shared)
        for L in ls:
            mine = mp - len(shared)
            rows.append(shared + list(range(free_page, free_page + mine)))
            free_page += mine
    nph = free_page + spare
    bt = torch.randperm(nph, generator=g)[torch.tensor(rows)].int().view(len(lens), mp)
    k = torch.randn((nph, hkv, P, 128), generator=g).half()
    v = torch.randn((nph, hkv, P, 128), generator=g).half()
    free = torch.ones((nph, P), dtype=torch.bool)
    for b, L in enumerate(lens):
        for p in range(-(-L // P)):
            free[bt[b, p].long(), :min(P, L - p * P)] = False
    k.masked_fill_(free[:, None, :, None], NAN)
    v.masked_fill_(free[:, None, :, None], NAN)
    cache = q.PagedCache.allocate_meta(k.cuda(), v.cuda(), bt.cuda(),
                                       torch.tensor(lens, dtype=torch.int32).cuda(), hq)
    return cache, [(len(ls), prefix) for prefix, ls in groups]


def queries(cache):
    return torch.randn((cache.batch, cache.desc.num_q_heads, 128), device="cuda").half()


def run(cache, groups, qq, pps=0, **kw):
    o = q.opts(pages_per_split=pps, **kw)
    ws = q.prefix_workspace(cache, groups, o)
    out, lse = q.prefix_decode(cache, qq, groups, ws, o)
    ok(ws)
    return out, lse


def right(cache, qq, out, lse):
    check(cache, qq[:, None], out[:, None], lse[:, None], 0, BIG, True)


GEOMS = [(4, 4, 16), (8, 1, 32), (8, 2, 16), (6, 3, 32)]
BATCHES = {
    "one": [(40, [50])],
    "pair": [(64, [64, 65])],
    "few": [(300, [301, 330, 512, 300])],
    "many": [(1000, [1000 + 13 * i for i in range(40)])],
    "groups": [(200, [210, 300]), (0, [77]), (129, [129, 700, 200]), (31, [40, 50]), (64, [64, 64])],
    "alone": [(100, [120]), (0, [5, 9, 300])],
    "short": [(500, [600, 3, 0, 499, 500, 17]), (260, [300, 0])],
    "empty": [(64, [0, 0]), (0, [0])],
    "blocks": [(150, [160 + i for i in range(70)]), (700, [701] * 33)],
}


@pytest.mark.parametrize("pps", [0, 1, 6, 100])
@pytest.mark.parametrize("geom", GEOMS, ids=str)
@pytest.mark.parametrize("batch", BATCHES)
def test_matches_64_bits(batch, geom, pps):
    cache, groups = make(BATCHES[batch], *geom, seed=len(batch) + pps)
    qq = queries(cache)
    out, lse = run(cache, groups, qq, pps)
    right(cache, qq, out, lse)


@pytest.mark.parametrize("geom", GEOMS, ids=str)
@pytest.mark.parametrize("tokens", [200, 700, 1900])
def test_scores_that_grow_along_the_prefix(tokens, geom):
    """The running maximum moves again and again (also within a work item, and in one half of a
    tile alone): large queries against keys that grow."""
    cache, groups = make([(tokens, [tokens + 9] * 6)], *geom, seed=tokens)
    P = cache.page_size
    qq = queries(cache) * 3
    for page in range(-(-(tokens + 9) // P)):
        for b in range(cache.batch if page * P >= tokens // P * P else 1):
            cache.k_pool[int(cache.block_table[b, page])] *= 0.25 + 2.5 * page * P / tokens
    for pps in (0, 1000):
        out, lse = run(cache, groups, qq, pps)
        right(cache, qq, out, lse)


@pytest.mark.parametrize("rows", [32, 9])
def test_work_items_of_many_tiles(rows):
    """Sixteen tiles a work item, all of its rows in use, or a few."""
    cache, groups = make([(2100, [2100 + 7 * i for i in range(rows)])], 8, 2, 16, seed=rows)
    qq = queries(cache) * 2
    out, lse = run(cache, groups, qq, 2048 // 16)
    right(cache, qq, out, lse)


def test_long_prefixes_and_pools_past_4_gib():
    """16K-token prefixes at the end of pools of 4.6 GB each."""
    cache, groups = make([(16400, [16500, 16401, 17000, 16400, 16899]), (8000, [8001, 9000])], 32, 8, 16)
    nph = 140000
    pools = []
    move = nph - cache.k_pool.shape[0]
    for name in ("k_pool", "v_pool"):
        pool = torch.empty((nph, 8, 16, 128), dtype=torch.float16, device="cuda")
        pool[:1] = NAN
        pool[move:] = getattr(cache, name)
        pools.append(pool)
    assert move * 8 * 16 * 128 * 2 > 2 ** 32
    far = q.PagedCache(*pools, cache.meta, cache.block_table + move, cache.seq_lens, 32)
    qq = queries(far)
    out, lse = run(far, groups, qq)
    right(far, qq, out, lse)


@pytest.mark.parametrize("pps", [0, 1, 6])
@pytest.mark.parametrize("geom,n", [((4, 4, 16), 2), ((4, 4, 16), 128), ((8, 1, 32), 16), ((8, 1, 32), 3),
                                    ((8, 2, 16), 5), ((8, 2, 16), 1), ((6, 3, 32), 33)], ids=str)
@pytest.mark.parametrize("batch", ["one", "few", "groups", "short", "empty", "blocks"])
def test_the_last_tokens_of_every_sequence(batch, geom, n, pps):
    """Drafted tokens: each sees what comes before it, in the prefix and in the tail; rows at negative
    positions see nothing."""
    if n * len(BATCHES[batch]) > 100 and batch == "blocks":
        pytest.skip("the same rows as the other batches, many times")
    cache, groups = make(BATCHES[batch], *geom, seed=n)
    qq = torch.randn((cache.batch, n, geom[0], 128), device="cuda").half()
    o = q.opts(pages_per_split=pps)
    ws = q.prefix_workspace(cache, groups, o, n)
    out, lse = q.prefix_decode(cache, qq, groups, ws, o)
    ok(ws)
    assert out.shape == qq.shape and lse.shape == qq.shape[:3]
    check(cache, qq, out, lse, 0, BIG, True)
    if n == 1:
        one, one_lse = run(cache, groups, qq[:, 0].contiguous(), pps or 1000)
        if pps:
            assert torch.equal(one, out[:, 0]) and torch.equal(one_lse, lse[:, 0])


def test_drafted_tokens_and_odd_values():
    """An infinity at a drafted token reaches the tokens from it on, no other row."""
    cache, groups = make([(200, [230, 215])], 8, 2, 16, seed=4)
    n = 12
    qq = torch.randn((2, n, 8, 128), device="cuda").half()
    o = q.opts(pages_per_split=4)
    ws = q.prefix_workspace(cache, groups, o, n)
    want, want_lse = (t.clone() for t in q.prefix_decode(cache, qq, groups, ws, o))
    at = 230 - 5
    cache.v_pool[int(cache.block_table[0, at // 16]), :, at % 16, 9] = INF
    out, lse = q.prefix_decode(cache, qq, groups, ws, o)
    ok(ws)
    assert torch.equal(lse, want_lse)
    sees = torch.zeros((2, n), dtype=torch.bool, device="cuda")
    sees[0, n - 5:] = True
    assert bool((out[..., 9][sees] == INF).all())
    out[..., 9][sees] = want[..., 9][sees]
    for b in range(2):
        L = int(cache.seq_lens[b])
        allowed = R.window_mask(L, n, 0, BIG, "cuda")
        for h in range(8):
            k, v = logical(cache, b, h // 4, "k_pool"), logical(cache, b, h // 4, "v_pool")
            v = torch.where(torch.isinf(v), 0.0, v)
            ref = R.attend(qq[b, :, h], k, v, allowed)
            ref[0][sees[b], 9] = want[b, sees[b], h, 9].double()
            R.assert_close(out[b, :, h], lse[b, :, h], ref, True, f"{b} {h}")


def test_without_lse_and_into_given_outputs():
    cache, groups = make(BATCHES["few"], 8, 2, 16)
    qq = queries(cache)
    want, want_lse = run(cache, groups, qq, 4)
    o = q.opts(pages_per_split=4)
    ws = q.prefix_workspace(cache, groups, o)
    out, lse = torch.full_like(want, NAN), torch.full_like(want_lse, NAN)
    got = q.prefix_decode(cache, qq, groups, ws, o, out=out, lse=lse)
    assert got[0] is out and got[1] is lse and torch.equal(out, want) and torch.equal(lse, want_lse)
    out, lse = q.prefix_decode(cache, qq, groups, ws, o, want_lse=False)
    assert lse is None and torch.equal(out, want)


def test_sharing_reads_the_first_row_once_and_repeats_exactly():
    """The same bits every time: no order of arrival enters a result."""
    cache, groups = make(BATCHES["blocks"], 8, 2, 16)
    qq = queries(cache)
    first = run(cache, groups, qq, 3)
    for _ in range(5):
        again = run(cache, groups, qq, 3)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def odd_rows(cache, groups, qq, at, value, name, rows):
    """`value` at dim 5 of the token `at` (page entry of sequence 0's table): the rows that see it."""
    out, lse = run(cache, groups, qq, 2)
    for b in range(cache.batch):
        sees = rows[b]
        if name == "k_pool" and sees:
            assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all(), b
        elif name == "v_pool" and sees:
            want = torch.full((cache.desc.num_q_heads,), value, device="cuda").half()
            assert torch.equal(torch.nan_to_num(out[b, :, 5], nan=7.0), torch.nan_to_num(want, nan=7.0)), b
            assert torch.isfinite(out[b, :, :5]).all() and torch.isfinite(out[b, :, 6:]).all()
        else:
            assert torch.isfinite(out[b]).all() and torch.isfinite(lse[b]).all(), b
    return out, lse


@pytest.mark.parametrize("geom", [(4, 4, 16), (8, 1, 32)], ids=str)
@pytest.mark.parametrize("at", [0, 255, 299, 310])
@pytest.mark.parametrize("value,name", [(NAN, "k_pool"), (NAN, "v_pool"), (INF, "v_pool"), (-INF, "v_pool")])
def test_odd_values_reach_the_rows_that_see_them(geom, at, value, name):
    """Sequences of 340, 256, 300 and 30 tokens behind a prefix of 320: a row sees a token of the
    prefix if its sequence has it, no other row does."""
    hq, hkv, P = geom
    lens = [340, 256, 300, 30]
    cache, groups = make([(320, lens)], hq, hkv, P, seed=at)
    qq = queries(cache)
    clean = getattr(cache, name).clone()
    phys = int(cache.block_table[0, at // P])
    # (the other sequences hold the same pages: they see the token if they are long enough)
    getattr(cache, name)[phys, :, at % P, 5] = value
    out, lse = odd_rows(cache, groups, qq, at, value, name, [L > at for L in lens])
    getattr(cache, name).copy_(clean)
    unseen = torch.tensor([L <= at for L in lens], device="cuda")
    if name == "v_pool":
        out[~unseen, :, 5] = run(cache, groups, qq, 2)[0][~unseen, :, 5]
        right(cache, qq, out, lse)
    elif bool(unseen.any()):
        want, want_lse = run(cache, groups, qq, 2)
        assert torch.equal(out[unseen], want[unseen]) and torch.equal(lse[unseen], want_lse[unseen])


@pytest.mark.parametrize("geom", [(4, 4, 16), (8, 1, 32), (8, 2, 16)], ids=str)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [64, 200, 333, 900])
def test_odd_values_in_a_tail_stay_in_its_sequence(geom, at, value):
    """A value of one sequence's own tokens (in either half of a tile, in any of its jobs)."""
    hq, hkv, P = geom
    cache, groups = make([(64, [1000, 980, 70])], hq, hkv, P, seed=at)
    qq = queries(cache)
    want, want_lse = run(cache, groups, qq, 6)
    phys = int(cache.block_table[1, at // P])
    clean = cache.v_pool.clone()
    cache.v_pool[phys, :, at % P, 5] = value
    out, lse = run(cache, groups, qq, 6)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1, :, 5] = False
    got = out[1, :, 5]
    assert torch.isnan(got).all() if value != value else bool((got == value).all())
    cache.v_pool.copy_(clean)
    out[~keep] = want[~keep]
    right(cache, qq, out, lse)
    assert torch.equal(lse, want_lse)
    assert torch.equal(out[[0, 2]], want[[0, 2]])


@pytest.mark.parametrize("lens", [[3, 600, 200], [0, 130, 600], [64, 64, 64]])
def test_a_first_sequence_shorter_than_its_prefix(lens):
    """The others read the prefix through its row of the block table all the same."""
    cache, groups = make([(192, lens), (256, [300] * 3)], 8, 2, 16, seed=lens[0])
    qq = queries(cache)
    for pps in (0, 3):
        out, lse = run(cache, groups, qq, pps)
        right(cache, qq, out, lse)


def test_many_groups_and_many_sequences():
    """128 groups (the most there are), and 300 short sequences in a few: the queue's chunks of 32
    sequences, jobs without a token, tails of every number of tiles."""
    cache, groups = make([(130 + 16 * (i % 5), [150 + 40 * (i % 7), 200]) for i in range(128)], 4, 2, 16)
    qq = queries(cache)
    for pps in (0, 2):
        out, lse = run(cache, groups, qq, pps)
        right(cache, qq, out, lse)
    cache, groups = make([(1040, [1040 + (i * 37) % 700 for i in range(150)]),
                          (0, [(i * 53) % 300 for i in range(100)]),
                          (2000, [2000 - 9 * i for i in range(50)])], 4, 1, 32)
    qq = queries(cache)
    out, lse = run(cache, groups, qq)
    right(cache, qq, out, lse)


def test_a_query_with_nan_stays_in_its_row():
    cache, groups = make(BATCHES["few"], 8, 2, 16)
    qq = queries(cache)
    want, want_lse = run(cache, groups, qq, 3)
    qq[1, 3, 100] = NAN
    out, lse = run(cache, groups, qq, 3)
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
    keep = torch.ones((4, 8), dtype=torch.bool, device="cuda")
    keep[1, 3] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])


@pytest.mark.parametrize("pps", [0, 2])
def test_a_plan_in_a_graph_while_sequences_grow(pps):
    """Append and attend, captured once on a stream of its own, replayed while the sequences grow
    past page ends."""
    cache, groups = make([(200, [210, 200, 333]), (64, [70, 80])], 8, 2, 16)
    cache.k_pool.nan_to_num_(0.0), cache.v_pool.nan_to_num_(0.0)
    o = q.opts(pages_per_split=pps)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ws, wws = q.prefix_workspace(cache, groups, o), q.window_workspace(cache)
        plan = q.PrefixPlan(cache, groups, ws, o)
        write = q.RotaryPlan(cache, q.Rope(), wws)
        new = [torch.randn((5, h, 128), device="cuda").half() for h in (8, 2, 2)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            plan.decode(write.append(*new))
        start = cache.seq_lens.clone()
        for step in range(20):
            if int(cache.seq_lens.max()) == cache.max_pages * 16:
                break
            for x in new:
                x.normal_()
            graph.replay()
            if step % 6 == 0:
                assert torch.equal(cache.seq_lens, start + step + 1)
                right(cache, write.q_out, plan.out, plan.lse)
        ok(ws), ok(wws)


def test_two_plans_on_two_streams():
    """Calls at the same time, with a workspace each."""
    made = [make(BATCHES[n], 8, 2, 16, seed=i) for i, n in enumerate(("many", "blocks"))]
    qs = [queries(c) for c, _ in made]
    want = [run(c, g, x, 5) for (c, g), x in zip(made, qs)]
    o = q.opts(pages_per_split=5)
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    plans = [q.PrefixPlan(c, g, q.prefix_workspace(c, g, o), o, stream=s) for (c, g), s in zip(made, streams)]
    torch.cuda.synchronize()
    for _ in range(30):
        for p, x in zip(plans, qs):
            p.decode(x)
    torch.cuda.synchronize()
    for p, (out, lse) in zip(plans, want):
        assert torch.equal(p.out, out) and torch.equal(p.lse, lse)


@pytest.mark.parametrize("entry", [-1, 2 ** 31 - 1])
def test_unmapped_pages_and_bad_lengths_are_reported(entry):
    for where in ("prefix", "tail", "length"):
        cache, groups = make([(400, [500, 450, 410])], 8, 2, 16)
        qq = queries(cache)
        if where == "prefix":
            cache.block_table[:, 7] = entry
        elif where == "tail":
            cache.block_table[1, 26] = entry
        else:
            cache.seq_lens[2] = entry
        o = q.opts(pages_per_split=3)
        ws = q.prefix_workspace(cache, groups, o)
        q.prefix_decode(cache, qq, groups, ws, o)
        rc, detail = q.read_status(ws)
        assert rc == (q.QUEST_ERR_BAD_LENGTH if where == "length" else q.QUEST_ERR_BAD_PAGE)
        if where != "length":
            assert detail[:2] == ((0, 7) if where == "prefix" else (1, 26))


@pytest.mark.parametrize("batch,pps", [("few", 0), ("many", 4), ("blocks", 0), ("short", 2)])
def test_a_wait_that_runs_out_ends_the_call(batch, pps):
    cache, groups = make(BATCHES[batch], 8, 2, 16)
    qq = queries(cache)
    kw = dict(wait_limit_ns=5_000_000, debug_flags=q.QUEST_DEBUG_WITHHOLD_VALUES)
    o = q.opts(pages_per_split=pps or 64, **kw)
    ws = q.prefix_workspace(cache, groups, o)
    for _ in range(2):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        q.prefix_decode(cache, qq, groups, ws, o)
        end.record()
        assert q.read_status(ws)[0] == q.QUEST_ERR_TIMEOUT
        assert 4 < start.elapsed_time(end) < 500
        q.workspace_init(ws)
    o = q.opts(pages_per_split=pps or 64)
    out, lse = q.prefix_decode(cache, qq, groups, ws, o)
    ok(ws)
    right(cache, qq, out, lse)


def test_a_short_limit_is_no_limit_on_work():
    """A limit far below a job's own time (uncut prefixes and tails) changes nothing."""
    cache, groups = make([(60000, [60100] * 40), (30000, [90000, 30001])], 8, 1, 32)
    qq = queries(cache)
    o = q.opts(pages_per_split=16384, wait_limit_ns=200_000)
    ws = q.prefix_workspace(cache, groups, o)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    out, lse = q.prefix_decode(cache, qq, groups, ws, o)
    start.record()
    q.prefix_decode(cache, qq, groups, ws, o, out=out, lse=lse)
    end.record()
    ok(ws)
    assert start.elapsed_time(end) > 0.3
    right(cache, qq, out, lse)


def test_a_short_limit_is_no_limit_on_rows_taken_again():
    """An infinite value makes every row of a job be taken again, a token at a time, while the CTA's
    other warps are at its next job (the prefixes' jobs alone are more than there are CTAs)."""
    cache, groups = make([(60000, [60030] * 4)] * 20, 64, 8, 32)
    at = int(cache.block_table[0, 3])
    cache.v_pool[at, :, 5, 9] = INF
    qq = queries(cache)
    o = q.opts(pages_per_split=16384, wait_limit_ns=300_000)
    ws = q.prefix_workspace(cache, groups, o)
    out, lse = q.prefix_decode(cache, qq, groups, ws, o)
    ok(ws)
    assert bool((out[:4, :, 9] == INF).all()) and bool(torch.isfinite(out[4:]).all())
    cache.v_pool[at, :, 5, 9] = 0
    out[..., 9] = run(cache, groups, qq, 16384)[0][..., 9]
    right(cache, qq, out, lse)


@pytest.mark.parametrize("hq,hkv,P,rope", [(8, 2, 16, dict()), (4, 4, 32, dict(rotary_dim=64, interleaved=True))])
def test_a_serving_step_from_projections(hq, hkv, P, rope):
    """A shared prompt written once with turned keys, every sequence's own question behind it, then
    decode steps (turn, append, attend): outputs against 64 bits from the raw projections."""
    r = q.Rope(**rope)
    prompt, asks, steps, B = 150, 20, 5, 3
    whole = prompt // P
    mp = -(-(prompt + asks + steps) // P)
    total = prompt + asks + steps
    x = torch.randn((B, total, hq + 2 * hkv, 128), device="cuda").half()
    x[:, :prompt] = x[:1, :prompt]  # the same prompt
    own = torch.arange(B * (mp - whole)).view(B, -1) + whole
    bt = torch.cat([torch.arange(whole).expand(B, -1), own], 1).int().cuda()
    pool = torch.full((int(bt.max()) + 1, hkv, P, 128), NAN, dtype=torch.float16, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    # the prompt's whole pages through the first sequence, the rest by each for itself
    one = q.PagedCache.allocate_meta(pool, pool.clone(), bt[:1].contiguous(), lens[:1].clone(), hq)
    wws = q.window_workspace(one)
    part = lambda t: (t[..., :hq, :], t[..., hq:hq + hkv, :], t[..., hq + hkv:, :])  # noqa: E731
    q.prefill_rotary(one, r, *part(x[:1, :whole * P]), wws)
    ok(wws)
    lens.fill_(whole * P)
    cache = q.PagedCache.allocate_meta(one.k_pool, one.v_pool, bt, lens, hq)
    cws = q.window_workspace(cache)
    q.prefill_rotary(cache, r, *part(x[:, whole * P:prompt + asks]), cws)
    groups = [(B, prompt)]
    o = q.opts(pages_per_split=2)
    ws = q.prefix_workspace(cache, groups, o)
    attend, write = q.PrefixPlan(cache, groups, ws, o), q.RotaryPlan(cache, r, cws)
    pos = torch.arange(total)
    turned = torch.stack([RR.turned(r, x[b, :, :hq + hkv], pos)[0] for b in range(B)])
    tq, tk, tv = turned[:, :, :hq].cuda(), turned[:, :, hq:].cuda(), x[:, :, hq + hkv:].double()
    for t in range(prompt + asks, total):
        out, lse = attend.decode(write.append(*part(x[:, t])))
        ok(ws), ok(cws)
        for b in range(B):
            for h in range(hq):
                g = h // (hq // hkv)
                k, v = tk[b, :t + 1, g], tv[b, :t + 1, g]
                ref = R.attend(tq[b, t, h][None], k, v, torch.ones((1, t + 1), dtype=torch.bool, device="cuda"))
                # keys and queries are what fp16 holds of the turned ones: each product of a score is
                # off by 2 * 2^-11 (and 2^-20s of the turn), a score by 2^-9.9 U, a weight by twice that
                e = 2.0 ** -9.9 * ref[3][:, None]
                tol = 2 * e * ref[2] + 2.0 ** -10 * ref[2] + 2.0 ** -11 * ref[0].abs() + 2.0 ** -24
                assert bool(((out[b, h].double() - ref[0]).abs() <= tol).all())
                assert float((lse[b, h].double() - ref[1]).abs()) <= float(e) + 1e-5
        # and exactly so from the cache as it is
        right(cache, write.q_out, out, lse)
    assert lens.tolist() == [total] * B


def test_refusals():
    cache, groups = make(BATCHES["few"], 8, 2, 16)
    ws = q.prefix_workspace(cache, groups)
    qq = queries(cache)
    for bad in ([], [(3, 10)], [(5, 10)], [(4, -1)], [(0, 0), (4, 8)], [(4, 10 ** 6)], [(-1, 0), (5, 0)],
                [(1, 0)] * 129):
        with pytest.raises(q.QuestError):
            q.prefix_decode(cache, qq, bad, ws)
        with pytest.raises(q.QuestError):
            q.prefix_workspace(cache, bad)
    with pytest.raises(q.QuestError):
        q.prefix_decode(cache, qq, groups, ws[:1024])
    for bad in (qq.float(), qq[:, :4], qq.cpu(), qq.transpose(0, 1)):
        with pytest.raises((ValueError, TypeError)):
            q.prefix_decode(cache, bad, groups, ws)
    with pytest.raises(q.QuestError, match="128"):
        q.prefix_workspace(cache, groups, None, 33)
    with pytest.raises(q.QuestError):
        q.prefix_decode(cache, queries(cache)[:, None][:, :0], groups, ws)
    with pytest.raises(ValueError):
        q.PrefixPlan(cache, groups, ws, n_tokens=-1)
    o = q.opts(pages_per_split=1)
    with pytest.raises(q.QuestError):  # a workspace for one token
        q.prefix_decode(cache, qq[:, None].repeat(1, 32, 1, 1), groups, q.prefix_workspace(cache, groups, o), o)
    nar = q.NarrowCache.allocate(9, 2, 16, cache.block_table, cache.seq_lens, 8)
    with pytest.raises(TypeError):
        q.PrefixPlan(nar, groups, ws)
