"""The selection of a narrow cache's decode steps where several work items of a row take it for
themselves (MHA rows) and where a kernel of its own does, and its outputs beside the fp16 cache's."""
import math

import pytest
import torch

import query_aware_kv_gb300 as q
import span_reference as R
from test_gpu_narrow import assert_cache, check, empty, ok, tokens
from test_gpu_window import check as check_window

pytestmark = pytest.mark.gpu


def whole(shape, top, g):
    """Whole numbers of at most `top`: the bounds are then exact sums, many of them equal."""
    return torch.randint(-top, top + 1, shape, generator=g).half()


def filled(hq, hkv, P, lens, pages, g):
    cache = empty(len(lens), hq, hkv, P, pages, seed=3)
    ref = R.NarrowReference(len(lens), hkv, P)
    for b, L in enumerate(lens):
        k, v = whole((1, L, hkv, 128), 3, g), torch.randn((1, L, hkv, 128), generator=g).half()
        # pages whose boxes are the same: tied at every query
        k[0, P:2 * P] = k[0, 3 * P:4 * P] if L >= 4 * P else k[0, P:2 * P]
        one = q.NarrowCache(cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale,
                            cache.k_open[b:b + 1], cache.v_open[b:b + 1], cache.meta[b:b + 1],
                            cache.block_table[b:b + 1], cache.seq_lens[b:b + 1], hq)
        ws = q.narrow_workspace(one)
        q.narrow_prefill(one, k.cuda(), v.cuda(), ws)
        ok(ws)
        ref.k[b], ref.v[b] = k[0].transpose(0, 1), v[0].transpose(0, 1)
    return cache, ref


def selection(k, qs, P, K, sink, local):
    """The pages that one kv head keeps: k [L, 128], qs [G, 128]."""
    L = k.shape[0]
    N = -(-L // P)
    pad = torch.nn.functional.pad(k.double(), (0, 0, 0, N * P - L), value=math.nan).view(N, P, 128)
    lo = torch.nan_to_num(pad, nan=math.inf).amin(1)
    hi = torch.nan_to_num(pad, nan=-math.inf).amax(1)
    x = qs.double()[:, None]
    bound = torch.maximum(x * lo, x * hi).sum(-1).amax(0)
    if N > K:
        bound[:sink] = math.inf
        bound[N - local:] = math.inf
    order = bound.sort(descending=True, stable=True).indices  # ties: the lower page
    return order[:K].sort().values.tolist()


CASES = [
    # hq, hkv, lens, top_k, pages per split, pages of the table
    (4, 4, [5000, 2100, 200], 16, 0, 340), (4, 4, [5000, 2100, 200], 64, 0, 340),
    (4, 4, [5000, 2100, 200], 128, 0, 340), (4, 4, [5000, 2100, 200], 64, 3, 340),
    (4, 4, [5000, 2100, 200], 128, 50, 340), (1, 1, [12000], 600, 0, 780),
    (2, 2, [5000, 90], 64, 0, 4200), (16, 16, [2600] * 4, 100, 0, 200),
    (16, 16, [900] * 24, 40, 0, 70), (8, 2, [5000, 700], 64, 0, 340),
]


@pytest.mark.parametrize("window", [(0, 0), (2, 3)], ids=["plain", "kept_ends"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_steps_select_the_same_pages_everywhere(case, window):
    """Work items of a row that select for themselves (few MHA rows of up to 4096 pages: over a
    cluster, over a join, one alone), rows with fewer pages than top_k, and rows that a kernel of its
    own selects for: pages, counts, outputs and lengths of every step."""
    hq, hkv, lens, K, pps, pages = case
    P, B, G = 16, len(lens), hq // hkv
    g = torch.Generator().manual_seed(K + pps)
    cache, ref = filled(hq, hkv, P, lens, pages, g)
    o = q.opts(pages_per_split=pps, sink_pages=window[0], local_pages=window[1])
    ws = q.narrow_workspace(cache, K, o)
    idx = torch.empty((B, hkv, K), dtype=torch.int32, device="cuda")
    cnt = torch.empty((B, hkv), dtype=torch.int32, device="cuda")
    plan = q.NarrowPlan(cache, K, ws, o, idx_out=idx, count_out=cnt)
    for step in range(3 if B > 4 else 6):
        kn, vn = whole((B, 1, hkv, 128), 3, g), torch.randn((B, 1, hkv, 128), generator=g).half()
        qq = whole((B, hq, 128), 2, g)
        idx.fill_(-7)
        ref.write(kn, vn)
        out, lse = plan.step(qq.cuda(), kn[:, 0].cuda(), vn[:, 0].cuda())
        ok(ws)
        assert cache.seq_lens.tolist() == [ref.length(b) for b in range(B)]
        got, n = idx.cpu(), cnt.cpu()
        mask = {}
        for b in range(B):
            for h in range(hkv):
                want = selection(ref.k[b][h], qq[b, h * G:h * G + G], P, K, *window)
                assert int(n[b, h]) == len(want) and got[b, h, :len(want)].tolist() == want, (step, b, h)
                assert (got[b, h, len(want):] == -1).all()
                a = torch.zeros((1, ref.length(b)), dtype=torch.bool)
                for p in want:
                    a[:, p * P:(p + 1) * P] = True
                mask[b, h] = a
        check(cache, ref, qq.cuda(), out, lse, lambda b, h: mask[b, h])
        # the same selection and attention without the append
        again, lse2 = q.narrow_decode(cache, qq.cuda(), K, ws, o, idx_out=idx, count_out=cnt)
        ok(ws)
        assert torch.equal(idx.cpu(), got) and torch.equal(again, out) and torch.equal(lse2, lse)
    if B < 5:
        assert_cache(cache, ref)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 4)])
def test_outputs_are_near_the_fp16_caches(hq, hkv):
    """The same tokens in both caches, the same selection: the outputs differ by what the codes
    allow.  With E the largest |q . (k' - k)| / sqrt(128) of a token, its weight differs by a factor
    of at most exp(2 E); so out differs by (exp(2 E) - 1) sum w |v'| + sum w |v' - v| at most, and
    by both sides' roundings."""
    P, L, K, G = 16, 700, 9, hq // hkv
    k, v = tokens(1, L, hkv, seed=21)
    narrow = empty(1, hq, hkv, P, L // P + 2, seed=3)
    nws = q.narrow_workspace(narrow, K)
    q.narrow_prefill(narrow, k.cuda(), v.cuda(), nws)
    fp16 = [torch.zeros(narrow.k_pool.shape, dtype=torch.float16, device="cuda") for _ in range(2)]
    wide = q.PagedCache.allocate_meta(*fp16, narrow.block_table,
                                      torch.zeros(1, dtype=torch.int32, device="cuda"), hq)
    wws = q.workspace(wide, K)
    q.prefill(wide, k.cuda(), v.cuda(), wws)
    g = torch.Generator().manual_seed(8)
    qq = torch.randn((1, hq, 128), generator=g).half()
    idx, cnt = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((1, hkv, K), (1, hkv)))
    out, lse = q.narrow_decode(narrow, qq.cuda(), K, nws, idx_out=idx, count_out=cnt)
    ok(nws)
    idx2, cnt2 = torch.empty_like(idx), torch.empty_like(cnt)
    out2, lse2 = q.decode(wide, qq.cuda(), K, wws, idx_out=idx2, count_out=cnt2)
    ok(wws)
    assert torch.equal(idx, idx2) and torch.equal(cnt, cnt2)
    ref = R.NarrowReference(1, hkv, P)
    ref.write(k, v)
    for h in range(hq):
        at = torch.cat([torch.arange(p * P, min(L, p * P + P)) for p in idx[0, h // G].tolist()])
        kh, vh = k[0, at, h // G].double(), v[0, at, h // G].double()
        kn, vn = ref.values(0, "k")[h // G][at], ref.values(0, "v")[h // G][at]
        x = qq[0, h].double()
        w = torch.softmax(kh @ x / math.sqrt(128), 0)
        E = float(((kn - kh) @ x).abs().max()) / math.sqrt(128)
        U = float((torch.maximum(kh.abs(), kn.abs()) @ x.abs()).max()) / math.sqrt(128)
        A = (w @ vn.abs()) * math.exp(2 * E) + w @ vh.abs()
        a, z = out[0, h].double().cpu(), out2[0, h].double().cpu()
        tol = ((math.exp(2 * E) - 1) * (w @ vn.abs()) + w @ (vn - vh).abs() +
               (2 * 132 * 2.0 ** -24 * U + 2.0 ** -20) * A + 2.0 ** -11 * (a.abs() + z.abs()) + 2.0 ** -24)
        assert ((a - z).abs() <= tol).all()
        lim = E + 2 * (132 * 2.0 ** -24 * U + 2.0 ** -20) + 2.0 ** -21 * abs(float(lse2[0, h]))
        assert abs(float(lse[0, h]) - float(lse2[0, h])) <= lim


@pytest.mark.parametrize("pps", [16384, 16385, 2 ** 31 - 1])
def test_splits_longer_than_any_row(pps):
    """pages_per_split up to the largest number that it holds: one work item a row."""
    g = torch.Generator().manual_seed(1)
    cache, ref = filled(8, 2, 16, [900, 30], 60, g)
    o = q.opts(pages_per_split=pps)
    ws = q.narrow_workspace(cache, 1, o)
    qq = torch.randn((2, 8, 128), device="cuda").half()
    out, lse = q.narrow_dense_decode(cache, qq, ws, o)
    ok(ws)
    check(cache, ref, qq, out, lse, lambda b, h: torch.ones((1, ref.length(b)), dtype=torch.bool))
    fp16 = [torch.randn(cache.k_pool.shape, device="cuda").half() for _ in range(2)]
    wide = q.PagedCache.allocate_meta(*fp16, cache.block_table, cache.seq_lens, 8)
    qn = torch.randn((2, 5, 8, 128), device="cuda").half()
    wws = q.window_workspace(wide, 5, o)
    out, lse = q.window_prefill(wide, qn, 4, 700, wws, o)
    ok(wws)
    check_window(wide, qn, out, lse, 4, 700, True)
