"""GPU parity of the narrow (8-bit) cache: its writes bit for bit against the definition of
the format, its attention against the plain 64-bit form over the stored values, a decode loop
of all of it together."""
import pytest
import torch

import query_aware_kv_gb300 as q
import span_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(0)


def empty(batch, hq, hkv, P, pages, seed=0):
    g = torch.Generator().manual_seed(seed)
    nph = batch * pages + 2
    bt = torch.randperm(nph, generator=g)[:batch * pages].view(batch, pages).int().cuda()
    cache = q.NarrowCache.allocate(nph, hkv, P, bt,
                                   torch.zeros(batch, dtype=torch.int32, device="cuda"), hq)
    cache.k_open.fill_(float("nan"))  # rows behind the open page's tokens are never tokens
    cache.v_open.fill_(float("nan"))
    cache.k_pool.view(torch.uint8).fill_(0x7f)  # NaN codes
    cache.v_pool.view(torch.uint8).fill_(0x7f)
    cache.k_scale.fill_(float("nan"))
    cache.v_scale.fill_(float("nan"))
    return cache


def tokens(batch, n, hkv, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn((batch, n, hkv, 128), generator=g) * scale
    k[..., 5] *= 8
    v = torch.randn((batch, n, hkv, 128), generator=g) * 3 * scale
    return k.half(), v.half()


def ok(ws):
    rc, detail = q.read_status(ws)
    assert rc == 0, (rc, detail)


def assert_cache(cache, ref):
    P = cache.page_size
    assert cache.seq_lens.cpu().tolist() == [ref.length(b) for b in range(cache.batch)]
    for b in range(cache.batch):
        phys = cache.block_table[b].cpu().long()
        for name in ("k", "v"):
            code, s, rest = ref.pages(b, name)
            at = phys[:code.shape[0]]
            pool = getattr(cache, name + "_pool").cpu()
            scale = getattr(cache, name + "_scale").cpu()
            got = pool.view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
            assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(code, nan=1e9)), (b, name)
            assert torch.equal(scale[at].double(), s), (b, name)
            rows = getattr(cache, name + "_open").cpu()[b, :, :rest.shape[1]]
            assert torch.equal(torch.nan_to_num(rows, nan=999.0), torch.nan_to_num(rest, nan=999.0)), (b, name)
        k = ref.k[b]
        meta = cache.meta.cpu()
        for p in range(-(-k.shape[1] // P)):
            page = k[:, p * P:(p + 1) * P]
            assert torch.equal(meta[b, :, p, 0], page.amin(1)) and \
                torch.equal(meta[b, :, p, 1], page.amax(1)), (b, p)


GEOMS = [(4, 4, 16), (8, 1, 32), (8, 2, 16), (6, 3, 32), (12, 12, 16)]


@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_chunks_and_tokens_give_the_format(geom):
    """Chunks of 1, P - 1, P, 2P + 3, 100 and 3 tokens and single tokens, compared after each;
    then the same tokens in one chunk into another cache: the same bytes."""
    hq, hkv, P = geom
    sizes = [1, P - 1, P, 2 * P + 3, 100, 3]
    total = sum(sizes) + P + 2
    cache = empty(3, hq, hkv, P, total // P + 2, seed=hq)
    ws = q.narrow_workspace(cache)
    ref = R.NarrowReference(3, hkv, P)
    k, v = tokens(3, total, hkv, seed=1)
    at = 0
    for n in sizes:
        kc, vc = k[:, at:at + n].contiguous(), v[:, at:at + n].contiguous()
        q.narrow_prefill(cache, kc.cuda(), vc.cuda(), ws)
        ref.write(kc, vc)
        at += n
        ok(ws)
        assert_cache(cache, ref)
    while at < total:
        q.narrow_append(cache, k[:, at].contiguous().cuda(), v[:, at].contiguous().cuda(), ws)
        ref.write(k[:, at:at + 1], v[:, at:at + 1])
        at += 1
    ok(ws)
    assert_cache(cache, ref)
    whole = empty(3, hq, hkv, P, total // P + 2, seed=hq)
    q.narrow_prefill(whole, k.cuda(), v.cuda(), ws)
    ok(ws)
    assert_cache(whole, ref)


def test_values_of_every_kind():
    """Zeros, subnormals, the largest fp16 numbers, values on rounding borders (ties),
    infinities and NaN, one kind per page."""
    P, hkv = 16, 2
    kinds = [torch.zeros(P, hkv, 128), torch.full((P, hkv, 128), 2.0 ** -24),
             torch.full((P, hkv, 128), 65504.0), torch.linspace(-448, 448, P * hkv * 128).view(P, hkv, 128),
             torch.linspace(-2, 2, P * hkv * 128).view(P, hkv, 128) ** 9]
    ties = torch.arange(P * hkv * 128).view(P, hkv, 128) % 256
    kinds.append((1 + ties / 16.0) * 2.0 ** (ties % 11 - 8.0))
    kinds.append(torch.where(ties == 7, torch.tensor(float("inf")), torch.randn(P, hkv, 128)))
    kinds.append(torch.where(ties == 9, torch.tensor(-float("inf")), torch.full((P, hkv, 128), 3.0)))
    kinds.append(torch.where(ties == 9, torch.tensor(float("nan")), torch.randn(P, hkv, 128)))
    x = torch.cat(kinds).half()[None]
    cache = empty(1, 2, hkv, P, len(kinds) + 1)
    ws = q.narrow_workspace(cache)
    q.narrow_prefill(cache, x.cuda(), x.flip(2).contiguous().cuda(), ws)
    ok(ws)
    ref = R.NarrowReference(1, hkv, P)
    ref.write(x, x.flip(2))
    for name in ("k", "v"):
        code, s, _ = ref.pages(0, name)
        at = cache.block_table[0, :len(kinds)].cpu().long()
        got = getattr(cache, name + "_pool").cpu().view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
        assert torch.equal(getattr(cache, name + "_scale").cpu()[at].double(), s)
        for i in range(len(kinds) - 1):
            assert torch.equal(got[i], code[i]), i
        raw = x[0, -P:].transpose(0, 1) if name == "k" else x.flip(2)[0, -P:].transpose(0, 1)
        assert torch.equal(torch.isnan(got[-1]), torch.isnan(raw))


def filled(geom, lens, seed=2, pages=None):
    hq, hkv, P = geom
    cache = empty(len(lens), hq, hkv, P, pages or max(lens) // P + 2, seed=seed)
    ref = R.NarrowReference(len(lens), hkv, P)
    k, v = tokens(len(lens), max(lens), hkv, seed=seed)
    for b, L in enumerate(lens):  # one sequence at a time: rows of the descriptor
        if L:
            one = q.NarrowCache(cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale,
                                cache.k_open[b:b + 1], cache.v_open[b:b + 1], cache.meta[b:b + 1],
                                cache.block_table[b:b + 1], cache.seq_lens[b:b + 1], hq)
            ws = q.narrow_workspace(one)
            q.narrow_prefill(one, k[b:b + 1, :L].contiguous().cuda(), v[b:b + 1, :L].contiguous().cuda(), ws)
            ok(ws)
        ref.k[b], ref.v[b] = k[b, :L].transpose(0, 1), v[b, :L].transpose(0, 1)
    return cache, ref


def check(cache, ref, qq, out, lse, allowed_of):
    G = cache.desc.num_q_heads // cache.num_kv_heads
    for b in range(cache.batch):
        k, v = ref.values(b, "k"), ref.values(b, "v")
        for h in range(cache.desc.num_q_heads):
            g = h // G
            R.assert_close(out[b, h:h + 1].cpu(), lse[b, h:h + 1].cpu(),
                           R.attend(qq[b, h:h + 1].cpu(), k[g], v[g], allowed_of(b, g)),
                           what=f"sequence {b} head {h}")


LENS = [0, 1, 15, 16, 33, 64, 500, 1031]


@pytest.mark.parametrize("pps", [0, 1, 5])
@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_dense(geom, pps):
    cache, ref = filled(geom, LENS)
    o = q.opts(pages_per_split=pps)
    ws = q.narrow_workspace(cache, 1, o)
    qq = torch.randn((len(LENS), geom[0], 128), device="cuda").half()
    out, lse = q.narrow_dense_decode(cache, qq, ws, o)
    ok(ws)
    check(cache, ref, qq, out, lse, lambda b, g: torch.ones((1, LENS[b]), dtype=torch.bool))


@pytest.mark.parametrize("geom", [(2, 2, 16), (4, 2, 16), (4, 1, 32), (8, 1, 16)], ids=str)
@pytest.mark.parametrize("window", [700, 6000, 2 ** 31 - 1])
def test_a_row_over_many_work_items(geom, window):
    """A row that a few work items share (their CTAs a cluster), and one that many do."""
    lens = [11003]
    cache, ref = filled(geom, lens)
    ws = q.narrow_workspace(cache)
    qq = torch.randn((1, geom[0], 128), device="cuda").half()
    out, lse = q.narrow_window_decode(cache, qq, 3, window, ws)
    ok(ws)
    check(cache, ref, qq, out, lse, lambda b, g: R.window_mask(lens[b], 1, 3, window, "cpu"))


@pytest.mark.parametrize("sink,window", [(0, 1), (4, 7), (3, 100), (40, 33), (300, 64), (0, 2 ** 31 - 1)])
@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_window(geom, sink, window):
    cache, ref = filled(geom, LENS)
    ws = q.narrow_workspace(cache)
    qq = torch.randn((len(LENS), geom[0], 128), device="cuda").half()
    out, lse = q.narrow_window_decode(cache, qq, sink, window, ws)
    ok(ws)
    check(cache, ref, qq, out, lse, lambda b, g: R.window_mask(LENS[b], 1, sink, window, "cpu"))


@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_sparse(geom):
    """A selection per head, the open page among it or not, empty and full rows."""
    hq, hkv, P = geom
    cache, ref = filled(geom, LENS)
    K = 7
    g = torch.Generator().manual_seed(4)
    idx = torch.full((len(LENS), hkv, K), -1, dtype=torch.int32)
    cnt = torch.zeros((len(LENS), hkv), dtype=torch.int32)
    for b, L in enumerate(LENS):
        N = -(-L // P)
        for h in range(hkv):
            c = min(K, N) if h % 2 == 0 else min(N, 2)
            idx[b, h, :c] = torch.randperm(N, generator=g)[:c].sort().values.int()
            cnt[b, h] = c
    ws = q.narrow_workspace(cache, K)
    qq = torch.randn((len(LENS), hq, 128), device="cuda").half()
    out, lse = q.narrow_sparse_decode(cache, qq, idx.cuda(), cnt.cuda(), K, ws)
    ok(ws)

    def allowed(b, h):
        a = torch.zeros((1, LENS[b]), dtype=torch.bool)
        for p in idx[b, h, :cnt[b, h]].tolist():
            a[:, p * P:(p + 1) * P] = True
        return a

    check(cache, ref, qq, out, lse, allowed)


@pytest.mark.parametrize("geom", GEOMS[:4], ids=str)
@pytest.mark.parametrize("window", [(0, 0), (1, 1)])
def test_decode_steps(geom, window):
    """A decode loop over page borders: the appended state, the selection (the fp16 cache's,
    from the oracle's scores) and the attention of every step."""
    hq, hkv, P = geom
    lens, K = [60, 200, 333], 6
    cache, ref = filled(geom, lens, pages=16 if P == 32 else 30)
    idx = torch.empty((3, hkv, K), dtype=torch.int32, device="cuda")
    cnt = torch.empty((3, hkv), dtype=torch.int32, device="cuda")
    o = q.opts(sink_pages=window[0], local_pages=window[1])
    ws = q.narrow_workspace(cache, K, o)
    plan = q.NarrowPlan(cache, K, ws, o, idx_out=idx, count_out=cnt)
    G = hq // hkv
    for step in range(P + 3):
        kn, vn = tokens(3, 1, hkv, seed=100 + step)
        qq = torch.randn((3, hq, 128), device="cuda").half()
        ref.write(kn, vn)
        if step % 5 == 4:  # append, then decode, as two calls
            q.narrow_append(cache, kn[:, 0].cuda(), vn[:, 0].cuda(), ws)
            out, lse = plan.decode(qq)
        else:
            out, lse = plan.step(qq, kn[:, 0].cuda(), vn[:, 0].cuda())
        ok(ws)
        for b in range(3):
            L = ref.length(b)
            N = -(-L // P)
            for g in range(hkv):
                box = [ref.k[b][g, p * P:(p + 1) * P].double() for p in range(N)]
                heads = qq[b, g * G:g * G + G].cpu().double()
                ub = [max(float(torch.maximum(x * p.amin(0), x * p.amax(0)).sum()) for x in heads) for p in box]
                if N > K:
                    for p in list(range(window[0])) + [N - 1 - i for i in range(window[1])]:
                        ub[p] = float("inf")
                order = sorted(range(N), key=lambda p: (-ub[p], p))
                c = min(K, N)
                got = idx[b, g, :c].tolist()
                assert int(cnt[b, g]) == c and got == sorted(got)
                edge = ub[order[c - 1]]
                near = {p for p in range(N) if abs(ub[p] - edge) <= 1e-5 * abs(edge)}
                assert set(got) - near == set(order[:c]) - near, (step, b, g)
        sel, n = idx.cpu(), cnt.cpu()

        def allowed(b, g):
            a = torch.zeros((1, ref.length(b)), dtype=torch.bool)
            for p in sel[b, g, :n[b, g]].tolist():
                a[:, p * P:(p + 1) * P] = True
            return a

        check(cache, ref, qq, out, lse, allowed)
    assert_cache(cache, ref)


def test_other_scales():
    """Pages that come from elsewhere: any fp32 scales, per page and head."""
    cache, ref = filled((4, 2, 16), [300])
    g = torch.Generator(device="cuda").manual_seed(1)
    cache.k_scale.copy_(torch.rand(cache.k_scale.shape, device="cuda", generator=g) * 3e-3)
    cache.v_scale.copy_(torch.rand(cache.v_scale.shape, device="cuda", generator=g) * 1e4)
    cache.v_scale[cache.block_table[0, 3].long()] = 0.0
    ws = q.narrow_workspace(cache)
    qq = torch.randn((1, 4, 128), device="cuda").half()
    out, lse = q.narrow_dense_decode(cache, qq, ws)
    ok(ws)
    for h in range(4):
        def val(name):
            at = cache.block_table[0, :18].long()
            x = getattr(cache, name + "_pool").view(torch.uint8)[at, h // 2].view(torch.float8_e4m3fn).double()
            x = (x * getattr(cache, name + "_scale")[at, h // 2].double()[:, None, None]).reshape(-1, 128)
            return torch.cat([x, getattr(cache, name + "_open")[0, h // 2, :300 % 16].double()])
        r = R.attend(qq[0, h:h + 1], val("k"), val("v"), torch.ones((1, 300), dtype=torch.bool, device="cuda"))
        R.assert_close(out[0, h:h + 1], lse[0, h:h + 1], r)


def test_a_chunk_that_does_not_fit_changes_nothing_live():
    cache, ref = filled((4, 4, 16), [37, 20], pages=4)
    before = cache.k_open.clone(), cache.v_open.clone(), cache.seq_lens.clone()
    k, v = tokens(2, 40, 4, seed=9)
    ws = q.narrow_workspace(cache)
    q.narrow_prefill(cache, k.cuda(), v.cuda(), ws)  # sequence 0 has room for 27
    rc, detail = q.read_status(ws)
    assert rc == q.QUEST_ERR_BAD_LENGTH and detail[0] == 0
    assert cache.seq_lens.tolist() == [37, 60]
    assert torch.equal(cache.k_open[0, :, :5], before[0][0, :, :5])
    assert torch.equal(cache.v_open[0, :, :5], before[1][0, :, :5])
    cache.block_table[1, 3] = -1
    q.narrow_append(cache, k[:, 0].contiguous().cuda(), v[:, 0].contiguous().cuda(), ws)
    rc, detail = q.read_status(ws)
    assert rc == q.QUEST_ERR_BAD_PAGE and detail[:2] == (1, 3)
    assert cache.seq_lens.tolist() == [38, 60]


def test_a_chunk_that_meets_an_unmapped_page_leaves_the_sequence():
    """The first page that the chunk would complete is mapped, a later one is not: tokens, box
    and length stay, and the same chunk goes in once the page is mapped."""
    cache, ref = filled((8, 2, 16), [37, 21], pages=40)
    ws = q.narrow_workspace(cache)
    held = int(cache.block_table[0, 37])
    cache.block_table[0, 37] = -1
    box = cache.meta[0, :, 2].clone()
    k, v = tokens(2, 590, 2, seed=12)
    q.narrow_prefill(cache, k.cuda(), v.cuda(), ws)
    rc, detail = q.read_status(ws)
    assert rc == q.QUEST_ERR_BAD_PAGE and detail[:2] == (0, 37)
    assert cache.seq_lens.tolist() == [37, 611]
    assert torch.equal(cache.meta[0, :, 2], box)
    assert torch.equal(cache.k_open[0, :, :5].cpu(), ref.k[0][:, 32:37])
    assert torch.equal(cache.v_open[0, :, :5].cpu(), ref.v[0][:, 32:37])
    cache.block_table[0, 37] = held
    cache.seq_lens[1] = 37  # (any length with room: sequence 1 is not looked at again)
    q.narrow_prefill(cache, k.cuda(), v.cuda(), ws)
    ok(ws)
    both = torch.cat((ref.k[0], k[0].transpose(0, 1)), 1)
    for p in range(627 // 16):
        page = both[:, p * 16:p * 16 + 16]
        assert torch.equal(cache.meta[0, :, p, 0].cpu(), page.amin(1)), p


def test_bad_selection_is_reported():
    cache, _ = filled((4, 4, 16), [100])
    ws = q.narrow_workspace(cache, 3)
    idx = torch.tensor([[[0, 9, -1]] * 4], dtype=torch.int32, device="cuda")
    cnt = torch.full((1, 4), 2, dtype=torch.int32, device="cuda")
    qq = torch.randn((1, 4, 128), device="cuda").half()
    q.narrow_sparse_decode(cache, qq, idx, cnt, 3, ws)
    rc, _ = q.read_status(ws)
    assert rc == q.QUEST_ERR_BAD_SELECTION


def test_graph_of_steps_on_a_side_stream():
    """A captured step (append, bounds, top-K, attention) replayed with new tokens in place."""
    geom, lens = (8, 2, 16), [200, 90]
    cache, ref = filled(geom, lens, pages=20)
    ws = q.narrow_workspace(cache, 8)
    kn, vn = (x[:, 0].cuda() for x in tokens(2, 1, 2, seed=1))
    qq = torch.randn((2, 8, 128), device="cuda").half()
    idx = torch.empty((2, 2, 8), dtype=torch.int32, device="cuda")
    cnt = torch.empty((2, 2), dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        plan = q.NarrowPlan(cache, 8, ws, idx_out=idx, count_out=cnt)
        plan.step(qq, kn, vn)
    for step in range(20):
        k, v = tokens(2, 1, 2, seed=50 + step)
        kn.copy_(k[:, 0])
        vn.copy_(v[:, 0])
        qq.copy_(torch.randn_like(qq))
        graph.replay()
        torch.cuda.synchronize()
        ok(ws)
        ref.write(k, v)

        def allowed(b, g):
            a = torch.zeros((1, ref.length(b)), dtype=torch.bool)
            for p in idx[b, g, :cnt[b, g]].tolist():
                a[:, p * 16:(p + 1) * 16] = True
            return a

        check(cache, ref, qq, plan.out, plan.lse, allowed)
    assert_cache(cache, ref)


def test_workspace_shared_by_every_call():
    """One workspace, sized for the largest top_k, for calls with other options in turn."""
    cache, ref = filled((8, 2, 16), [900, 400])
    o = q.opts(pages_per_split=2)
    ws = q.narrow_workspace(cache, 40, o)
    qq = torch.randn((2, 8, 128), device="cuda").half()
    for _ in range(2):
        q.narrow_decode(cache, qq, 40, ws)
        out, lse = q.narrow_dense_decode(cache, qq, ws, o)
        check(cache, ref, qq, out, lse, lambda b, g: torch.ones((1, ref.length(b)), dtype=torch.bool))
        out, lse = q.narrow_window_decode(cache, qq, 4, 300, ws, o)
        check(cache, ref, qq, out, lse, lambda b, g: R.window_mask(ref.length(b), 1, 4, 300, "cpu"))
    ok(ws)


def test_selection_is_that_of_the_fp16_cache():
    """The boxes are those of the fp16 keys: the same selection from the same tokens."""
    hq, hkv, P, L, K = 8, 2, 16, 700, 9
    k, v = tokens(1, L, hkv, seed=21)
    narrow = empty(1, hq, hkv, P, L // P + 2, seed=3)
    nws = q.narrow_workspace(narrow, K)
    q.narrow_prefill(narrow, k.cuda(), v.cuda(), nws)
    wide = q.PagedCache.allocate_meta(
        torch.zeros(narrow.k_pool.shape, dtype=torch.float16, device="cuda"),
        torch.zeros(narrow.k_pool.shape, dtype=torch.float16, device="cuda"), narrow.block_table,
        torch.zeros(1, dtype=torch.int32, device="cuda"), hq)
    wws = q.workspace(wide, K)
    q.prefill(wide, k.cuda(), v.cuda(), wws)
    qq = torch.randn((1, hq, 128), device="cuda").half()
    sel = []
    for cache, ws, call in ((narrow, nws, q.narrow_decode), (wide, wws, q.decode)):
        idx = torch.empty((1, hkv, K), dtype=torch.int32, device="cuda")
        cnt = torch.empty((1, hkv), dtype=torch.int32, device="cuda")
        out, lse = call(cache, qq, K, ws, idx_out=idx, count_out=cnt)
        ok(ws)
        sel.append((idx, out, lse))
    assert torch.equal(narrow.meta, wide.meta)
    assert torch.equal(sel[0][0], sel[1][0])


def test_rows_behind_the_open_page_are_left_as_they_were():
    P = 16
    cache = empty(1, 2, 2, P, 6, seed=4)
    ws = q.narrow_workspace(cache)
    k, v = tokens(1, 60, 2, seed=31)
    at = 0
    for n in (5, 3, 20, 1):
        before = cache.k_open.clone(), cache.v_open.clone()
        q.narrow_prefill(cache, k[:, at:at + n].contiguous().cuda(), v[:, at:at + n].contiguous().cuda(), ws)
        at += n
        rows = at % P
        for now, was in ((cache.k_open, before[0]), (cache.v_open, before[1])):
            assert torch.equal(now[0, :, rows:].view(torch.int16), was[0, :, rows:].view(torch.int16))
    q.narrow_append(cache, k[:, at].contiguous().cuda(), v[:, at].contiguous().cuda(), ws)
    ok(ws)
    assert int(cache.seq_lens[0]) == 30


def test_offsets_past_32_bits():
    """Pages beyond the first 4 GiB of each pool: written, then read."""
    hkv, P, hq, L = 8, 32, 16, 300
    nph = (5 << 30) // (hkv * P * 128)
    pages = -(-L // P) + 1
    bt = torch.arange(nph - pages, nph, device="cuda").int().flip(0)[None].contiguous()
    cache = q.NarrowCache.allocate(nph, hkv, P, bt, torch.zeros(1, dtype=torch.int32, device="cuda"), hq)
    ws = q.narrow_workspace(cache)
    k, v = tokens(1, L, hkv, seed=41)
    q.narrow_prefill(cache, k.cuda(), v.cuda(), ws)
    ok(ws)
    ref = R.NarrowReference(1, hkv, P)
    ref.write(k, v)
    assert_cache(cache, ref)
    qq = torch.randn((1, hq, 128), device="cuda").half()
    out, lse = q.narrow_dense_decode(cache, qq, ws)
    ok(ws)
    check(cache, ref, qq, out, lse, lambda b, g: torch.ones((1, L), dtype=torch.bool))


def test_hidden_and_unwritten_slots_hold_anything():
    """NaN codes and scales in pages and slots that no call may read as tokens."""
    cache, ref = filled((8, 2, 32), [500, 90])
    lo = 500 - 70
    at = cache.block_table.long()
    pool = cache.k_pool.view(torch.uint8), cache.v_pool.view(torch.uint8)
    for t in range(lo // 32 * 32, lo):  # before the window, in its first page
        for x in pool:
            x[at[0, t // 32], :, t % 32] = 0x7f
    for p in range(1, lo // 32):  # between the sinks and the window
        cache.k_scale[at[0, p]] = float("nan")
        cache.v_scale[at[0, p]] = float("nan")
    ws = q.narrow_workspace(cache)
    qq = torch.randn((2, 8, 128), device="cuda").half()
    out, lse = q.narrow_window_decode(cache, qq, 4, 70, ws)
    ok(ws)
    check(cache, ref, qq, out, lse, lambda b, g: R.window_mask(ref.length(b), 1, 4, 70, "cpu"))


def test_a_step_without_room_keeps_its_length():
    cache, ref = filled((4, 4, 16), [64, 20], pages=4)
    ws = q.narrow_workspace(cache, 3)
    kn, vn = (x[:, 0].cuda() for x in tokens(2, 1, 4, seed=1))
    qq = torch.randn((2, 4, 128), device="cuda").half()
    q.narrow_decode_step(cache, qq, kn, vn, 3, ws)
    rc, detail = q.read_status(ws)
    assert rc == q.QUEST_ERR_BAD_LENGTH and detail[0] == 0
    assert cache.seq_lens.tolist() == [64, 21]
    q.workspace_init(ws)
    cache.block_table[1, 1] = cache.k_pool.shape[0]
    q.narrow_decode_step(cache, qq, kn, vn, 3, ws)
    rc, _ = q.read_status(ws)
    assert rc in (q.QUEST_ERR_BAD_LENGTH, q.QUEST_ERR_BAD_PAGE)
    assert cache.seq_lens.tolist() == [64, 21]
