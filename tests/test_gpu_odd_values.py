"""NaN and infinities that a row does see: in queries, keys and values, for windowed attention and
the narrow cache, however the row is split over work items."""
import pytest
import torch

import query_aware_kv_gb300 as q
import span_reference as R
from test_gpu_narrow import empty
from test_gpu_window import BIG, logical, make, ok

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(0)


def slot(cache, b, t):
    return int(cache.block_table[b, t // cache.page_size]), slice(None), t % cache.page_size


def assert_rows(cache, qq, out, lse, sink, window, odd_k=(), odd_v=(), odd_q=None):
    """qq, out [B, n, Hq, 128].  odd_k: (sequence, token) of NaN keys; odd_v: (sequence, token, dim,
    value); odd_q [B, n, Hq]: rows whose query holds a NaN.  Pools hold finite values in their
    places by now."""
    B, n, hq, _ = qq.shape
    G = hq // cache.num_kv_heads
    for b in range(B):
        allowed = R.window_mask(int(cache.seq_lens[b]), n, sink, window, "cuda")
        for h in range(hq):
            k, v = logical(cache, b, h // G, "k_pool"), logical(cache, b, h // G, "v_pool")
            o, z = out[b, :, h].clone(), lse[b, :, h].clone()
            lost = torch.zeros(n, dtype=torch.bool, device="cuda")
            for s, t in odd_k:
                if s == b:
                    lost |= allowed[:, t]
            if odd_q is not None:
                lost |= odd_q[b, :, h] & allowed.any(-1)
            assert torch.isnan(o[lost]).all() and torch.isnan(z[lost]).all(), (b, h)
            ref = R.attend(torch.nan_to_num(qq[b, :, h]), k, v, allowed)
            want = torch.zeros_like(o)  # sums of the infinities that a row sees
            for s, t, d, x in odd_v:
                if s == b:
                    want[allowed[:, t], d] += x
            odd = (want != 0) & ~lost[:, None]
            assert torch.equal(torch.nan_to_num(o[odd], nan=7.0), torch.nan_to_num(want[odd], nan=7.0)), (b, h)
            o[odd] = ref[0][odd].half()
            o[lost], z[lost] = ref[0][lost].half(), ref[1][lost].float()
            R.assert_close(o, z, ref, True, f"sequence {b} head {h}")


# rows in one work item, over a few (a cluster's or a join's), over many
SPLITS = [0, 1, 7, 40]
GEOMS = [(2, 2, 16), (8, 1, 32), (8, 2, 16)]


def run(cache, qq, sink, window, pps):
    n = qq.shape[1]
    o = q.opts(pages_per_split=pps)
    ws = q.window_workspace(cache, n, o)
    out, lse = q.window_prefill(cache, qq, sink, window, ws, o)
    ok(ws)
    return out, lse


@pytest.mark.parametrize("pps", SPLITS)
@pytest.mark.parametrize("geom", GEOMS, ids=str)
@pytest.mark.parametrize("n", [1, 3, 150])
def test_a_query_with_nan(geom, n, pps):
    """Its rows are NaN, those that see no token are 0 all the same; no other row changes."""
    hq, hkv, P = geom
    cache = make([700, 0, 90, 1], hq, hkv, P, seed=1)
    qq = torch.randn((4, n, hq, 128), device="cuda").half()
    odd = torch.rand((4, n, hq), device="cuda") < 0.3
    odd[:, -1, 0] = True
    odd[0, -1, -1] = False
    qq[..., 77][odd] = NAN
    for sink, window in [(4, 300), (0, BIG), (0, 1)]:
        out, lse = run(cache, qq, sink, window, pps)
        assert_rows(cache, qq, out, lse, sink, window, odd_q=odd)


@pytest.mark.parametrize("pps", SPLITS)
@pytest.mark.parametrize("geom", GEOMS, ids=str)
@pytest.mark.parametrize("n", [1, 3, 150])
def test_keys_with_nan(geom, n, pps):
    """One NaN key, and a run of them that fills whole work items of the row: rows that see one are
    NaN, the log-sum-exp with them."""
    hq, hkv, P = geom
    for first, count in [(650, 1), (640, 33), (128, 320)]:
        cache = make([700], hq, hkv, P, seed=2)
        clean = cache.k_pool.clone()
        for t in range(first, first + count):
            cache.k_pool[slot(cache, 0, t)] = NAN
        qq = torch.randn((1, n, hq, 128), device="cuda").half()
        got = [run(cache, qq, sink, window, pps) for sink, window in [(0, BIG), (3, 55)]]
        cache.k_pool.copy_(clean)
        for (sink, window), (out, lse) in zip([(0, BIG), (3, 55)], got):
            assert_rows(cache, qq, out, lse, sink, window,
                        odd_k=[(0, t) for t in range(first, first + count)])


@pytest.mark.parametrize("name", ["dense", "window", "sparse", "decode", "step"])
@pytest.mark.parametrize("pps", [0, 1, 20])
@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_a_query_with_nan_on_a_narrow_cache(geom, pps, name):
    hq, hkv, P = geom
    cache, _, _ = narrow(geom, 500)
    K = 500 // P + 2
    o = q.opts(pages_per_split=pps)
    ws = q.narrow_workspace(cache, K, o)
    qq = torch.randn((1, hq, 128), device="cuda").half()
    qq[0, hq - 1, 3] = NAN
    if name == "dense":
        out, lse = q.narrow_dense_decode(cache, qq, ws, o)
    elif name == "window":
        out, lse = q.narrow_window_decode(cache, qq, 4, 300, ws, o)
    elif name == "decode":
        out, lse = q.narrow_decode(cache, qq, K, ws, o)
    elif name == "step":
        new = torch.randn((2, 1, hkv, 128), device="cuda").half()
        out, lse = q.narrow_decode_step(cache, qq, new[0], new[1], K, ws, o)
    else:
        N = -(-500 // P)
        idx = torch.full((1, hkv, K), -1, dtype=torch.int32, device="cuda")
        idx[:, :, :N] = torch.arange(N, device="cuda").int()
        out, lse = q.narrow_sparse_decode(cache, qq, idx, torch.full((1, hkv), N, dtype=torch.int32, device="cuda"),
                                          K, ws, o)
    ok(ws)
    assert torch.isnan(out[0, -1]).all() and torch.isnan(lse[0, -1])
    assert torch.isfinite(out[0, :-1]).all() and torch.isfinite(lse[0, :-1]).all()


def narrow(geom, L, k_odd=(), v_odd=()):
    """A narrow cache of one sequence of L tokens, some of whose values are (token, dim, value)."""
    hq, hkv, P = geom
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn((1, L, hkv, 128), generator=g).half() for _ in range(2))
    for x, odd in ((k, k_odd), (v, v_odd)):
        for t, d, value in odd:
            x[0, t, :, d] = value
    cache = empty(1, hq, hkv, P, L // P + 2, seed=1)
    ws = q.narrow_workspace(cache)
    q.narrow_prefill(cache, k.cuda(), v.cuda(), ws)
    ok(ws)
    ref = R.NarrowReference(1, hkv, P)
    ref.write(k, v)
    return cache, ref, ws


@pytest.mark.parametrize("pps", [0, 1, 20])
@pytest.mark.parametrize("geom", GEOMS, ids=str)
@pytest.mark.parametrize("at", [33, 498])
def test_a_nan_key_in_a_narrow_cache(geom, at, pps):
    """In a complete page and in the open one."""
    cache, _, _ = narrow(geom, 500, k_odd=[(at, 9, NAN)])
    o = q.opts(pages_per_split=pps)
    ws = q.narrow_workspace(cache, 1, o)
    qq = torch.randn((1, geom[0], 128), device="cuda").half()
    out, lse = q.narrow_dense_decode(cache, qq, ws, o)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    out, lse = q.narrow_window_decode(cache, qq, 2, 20, ws, o)
    ok(ws)
    sees = at >= 480
    assert torch.isnan(out).all() == sees and torch.isnan(lse).all() == sees
    assert torch.isfinite(out).all() != sees


@pytest.mark.parametrize("pps", SPLITS)
@pytest.mark.parametrize("geom", GEOMS, ids=str)
@pytest.mark.parametrize("n", [1, 3, 150])
def test_infinities_among_the_values(geom, n, pps):
    """Rows that see one infinity get it in its dimension and nowhere else, rows that see both signs
    of it NaN, and one with a weight far below the largest counts like any other."""
    hq, hkv, P = geom
    odd = [(0, 690, 5, INF), (0, 3, 6, -INF), (0, 128, 77, INF), (0, 699, 77, -INF), (0, 400, 127, INF),
           (1, 1, 0, INF), (1, 1, 1, -INF)]
    cache = make([700, 2], hq, hkv, P, seed=4)
    qq = torch.randn((2, n, hq, 128), device="cuda").half()
    # the key of one of them: a score of about -60, far under fp16's smallest weight
    at = slot(cache, 0, 400)
    cache.k_pool[at] = 0
    cache.k_pool[at][:, 8] = -200
    qq[..., 8] = 3.5
    clean = cache.v_pool.clone()
    for b, t, d, x in odd:
        cache.v_pool[slot(cache, b, t)][:, d] = x
    visible = [(0, BIG), (4, 55), (3, 1)]
    got = [run(cache, qq, sink, window, pps) for sink, window in visible]
    cache.v_pool.copy_(clean)
    for (sink, window), (out, lse) in zip(visible, got):
        assert_rows(cache, qq, out, lse, sink, window, odd_v=odd)


@pytest.mark.parametrize("pps", SPLITS)
@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_an_infinity_of_little_weight(geom, pps):
    """The work item that holds the infinity has a maximum far below that of another (a factor of
    2^-170): its part is not multiplied away."""
    hq, hkv, P = geom
    cache = make([700], hq, hkv, P, seed=6)
    for t in range(700):
        cache.k_pool[slot(cache, 0, t)] = 0
        cache.k_pool[slot(cache, 0, t)][:, 8] = 200 if t >= 600 else -200
    cache.v_pool[slot(cache, 0, 100)][:, 9] = INF
    for n in (1, 3):
        qq = torch.randn((1, n, hq, 128), device="cuda").half()
        qq[..., 8] = 3.35
        out, lse = run(cache, qq, 0, BIG, pps)
        assert (out[..., 9] == INF).all() and torch.isfinite(lse).all()
        out[..., 9] = 0
        assert torch.isfinite(out).all()


def test_many_rows_with_an_infinity():
    """More rows than are ever split, and rows of CTAs of four warps."""
    for batch, hkv in [(20, 8), (70, 16)]:
        lens = [(37 * b) % 211 for b in range(batch)]
        cache = make(lens, hkv, hkv, 16, seed=15)
        odd = [(b, lens[b] - 7, b % 128, INF if b % 2 else -INF) for b in range(batch) if lens[b] > 7]
        clean = cache.v_pool.clone()
        for b, t, d, x in odd:
            cache.v_pool[slot(cache, b, t)][:, d] = x
        qq = torch.randn((batch, 1, hkv, 128), device="cuda").half()
        out, lse = run(cache, qq, 3, 50, 0)
        cache.v_pool.copy_(clean)
        assert_rows(cache, qq, out, lse, 3, 50, odd_v=odd)


@pytest.mark.parametrize("name", ["dense", "window", "decode", "step"])
@pytest.mark.parametrize("pps", [0, 1, 20])
@pytest.mark.parametrize("geom", GEOMS, ids=str)
def test_an_infinity_in_the_open_page(geom, pps, name):
    """The fp16 rows of a narrow cache's open page hold what was written: its infinity goes out,
    every other dimension is as if it were not there."""
    hq, hkv, P = geom
    L = 500  # 20 (P = 32) or 4 (P = 16) tokens in the open page
    cache, ref, _ = narrow(geom, L, v_odd=[(498, 9, INF), (497, 70, -INF)])
    K = L // P + 2
    o = q.opts(pages_per_split=pps)
    ws = q.narrow_workspace(cache, K, o)
    qq = torch.randn((1, hq, 128), device="cuda").half()
    new = torch.randn((2, 1, 1, hkv, 128)).half()
    if name == "dense":
        out, lse = q.narrow_dense_decode(cache, qq, ws, o)
    elif name == "window":
        out, lse = q.narrow_window_decode(cache, qq, 4, 300, ws, o)
    elif name == "decode":
        out, lse = q.narrow_decode(cache, qq, K, ws, o)
    else:
        out, lse = q.narrow_decode_step(cache, qq, new[0, 0].cuda(), new[1, 0].cuda(), K, ws, o)
        ref.write(new[0], new[1])
        L += 1
    ok(ws)
    assert (out[:, :, 9] == INF).all() and (out[:, :, 70] == -INF).all()
    allowed = R.window_mask(L, 1, 4, 300 if name == "window" else BIG, "cpu")
    for h in range(hq):
        k, v = ref.values(0, "k")[h // (hq // hkv)], torch.nan_to_num(ref.values(0, "v")[h // (hq // hkv)], posinf=0, neginf=0)
        r = R.attend(qq[0, h:h + 1].cpu(), k, v, allowed)
        got = out[0, h:h + 1].cpu().clone()
        got[:, [9, 70]] = r[0][:, [9, 70]].half()
        R.assert_close(got, lse[0, h:h + 1].cpu(), r)
