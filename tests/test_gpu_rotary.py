"""Rotary positions on the GPU: rotate against 64 bits, cache writes that turn their keys against
rotate followed by the plain writes (bit for bit) and against 64 bits."""
import itertools

import pytest
import torch

import query_aware_kv_gb300 as q
import rotary_reference as R

pytestmark = pytest.mark.gpu
D = 128


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.float16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


ROPES = {
    "plain": lambda: q.Rope(),
    "inter": lambda: q.Rope(interleaved=True),
    "part": lambda: q.Rope(64, base=500000.0),
    "part_inter": lambda: q.Rope(24, interleaved=True, scaling="linear", factor=4.0),
    "least": lambda: q.Rope(8),
    "odd_part": lambda: q.Rope(104, scaling="ntk", factor=3.0),
    "yarn": lambda: q.Rope(scaling="yarn", factor=8.0, original_length=4096),
    "bands": lambda: q.Rope(96, interleaved=True, scaling="bands", factor=8.0, original_length=4096),
    "own": lambda: q.Rope.from_frequencies([3.0, -0.5, 0.0, 1e-7], magnitude=0.75),
}


@pytest.mark.parametrize("rope", ROPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=str)
def test_rotate_matches_64_bits(rope, dtype):
    r, g = ROPES[rope](), gen(1)
    for (n, heads), transposed in itertools.product([(1, 1), (3, 2), (7, 5), (33, 40)], [False, True]):
        x = normal(g, n, heads, D, dtype=dtype)
        pos = torch.randint(0, 5000, (n,), generator=g, device="cuda", dtype=torch.int32)
        y, bound = R.turned(r, x, pos, transposed)
        got = q.rotate(r, x, pos, transposed=transposed)
        assert got.dtype == dtype and got.shape == x.shape
        R.check(got, y, bound)
        rd = r.rotary_dim
        assert torch.equal(got[..., rd:], x[..., rd:])


def test_rotate_is_exact_at_far_and_negative_positions():
    r, g = q.Rope(), gen(2)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 0, 1 << 20, 123456789, -7654321], dtype=torch.int32,
                       device="cuda")
    x = normal(g, len(pos), 3, D, dtype=torch.float32)
    R.check(q.rotate(r, x, pos), *R.turned(r, x, pos))


@pytest.mark.parametrize("name", ["plain", "yarn", "bands", "own"])
def test_cosines_and_sines_lose_only_their_last_rounding(name):
    """Of pairs (1, 0) the turn is m cos and m sin themselves.  Next to half a unit in the last place
    (2^-24 of the value) there are the angle's cut (1.5e-9), and in the sine products of at most a
    tenth that are rounded three times (1.8e-8): below 2e-8 together, and little in the mean."""
    r, g = ROPES[name](), gen(5)
    a, b = R.pairs(r)
    pos = torch.randint(-2 ** 20, 2 ** 20, (2000,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.zeros((2000, 1, D), device="cuda")
    x[..., a] = 1.0
    y = q.rotate(r, x, pos)[:, 0].double().cpu()
    t, m = R.angles(r, pos.cpu()), r.magnitude
    for got, want in ((y[:, a], torch.cos(t) * m), (y[:, b], torch.sin(t) * m)):
        far, nearest = (got - want).abs(), (want.float().double() - want).abs()
        assert bool((far <= 2.0 ** -24 * want.abs() + 2e-8 * abs(m)).all())
        assert float(far.square().mean().sqrt()) <= 1.1 * float(nearest.square().mean().sqrt()) + 1.5e-9


def test_rotate_takes_strided_rows_and_writes_in_place():
    r, g = q.Rope(), gen(3)
    rows = normal(g, 2, 9, 12, D)
    pos = torch.arange(18, device="cuda", dtype=torch.int32).view(2, 9)
    part = rows[:, :, 2:7]
    want = q.rotate(r, part.contiguous(), pos)
    assert torch.equal(q.rotate(r, part, pos), want)
    before = rows.clone()
    out = torch.zeros_like(rows)
    q.rotate(r, part, pos, out=out[:, :, 5:10])
    assert torch.equal(out[:, :, 5:10], want)
    assert not out[:, :, :5].any() and not out[:, :, 10:].any()
    assert q.rotate(r, part, pos, out=part) is part
    assert torch.equal(rows[:, :, 2:7], want)
    assert torch.equal(rows[:, :, :2], before[:, :, :2]) and torch.equal(rows[:, :, 7:], before[:, :, 7:])
    one = normal(g, 1, 4, D).expand(6, 4, D)  # the same token at six positions
    pos6 = torch.arange(6, device="cuda", dtype=torch.int32)
    assert torch.equal(q.rotate(r, one, pos6), q.rotate(r, one.contiguous(), pos6))
    assert q.rotate(r, rows[:0], pos[:0]).shape == (0, 9, 12, D)


def test_rotate_keeps_infinities_to_their_pair():
    r, g = q.Rope(64), gen(4)
    x = normal(g, 2, 2, D)
    x[0, 0, 3], x[1, 1, 100] = float("inf"), float("nan")
    y = q.rotate(r, x, torch.tensor([5, 6], device="cuda", dtype=torch.int32))
    odd = ~torch.isfinite(y)
    assert odd.nonzero().tolist() == [[0, 0, 3], [0, 0, 35], [1, 1, 100]]


@pytest.mark.parametrize("inter", [False, True])
def test_transposed_is_the_gradient(inter):
    """<w, rotate(x)> has the gradient rotate(w, transposed) in x: against differences, which are the
    derivative itself for a linear map (in 64 bits, of the definition)."""
    r, g = q.Rope(72, interleaved=inter, scaling="yarn", factor=4.0, original_length=512), gen(5)
    x, w = normal(g, 3, 2, D, dtype=torch.float32), normal(g, 3, 2, D, dtype=torch.float32)
    pos = torch.tensor([0, 11, 70000], dtype=torch.int32, device="cuda")
    grad = q.rotate(r, w, pos, transposed=True).double().cpu()
    y, bound = R.turned(r, x, pos)
    for at in [(0, 0, 5), (1, 1, 0), (1, 0, 71), (2, 1, 40), (2, 0, 100)]:
        moved = x.double().cpu()
        moved[at] += 1.0
        diff = ((R.turned(r, moved, pos)[0] - y) * w.double().cpu()).sum()
        # grad's own error: as turned() bounds it for w, and one rounding to fp32
        room = float(R.turned(r, w, pos, True)[1][at]) + abs(float(diff)) * 2.0 ** -23 + 1e-12
        assert abs(float(grad[at] - diff)) <= room


# ------------------------------------------------------------------ writes
def paged(g, B, Hq, Hkv, P, lens, mp, narrow):
    nph = B * mp + 2
    bt = torch.randperm(nph, generator=g, device="cuda")[:B * mp].view(B, mp).to(torch.int32)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if narrow:
        c = q.NarrowCache.allocate(nph, Hkv, P, bt, sl, Hq)
        c.k_open.copy_(normal(g, B, Hkv, P, D))
        c.v_open.copy_(normal(g, B, Hkv, P, D))
        c.meta.copy_(normal(g, *c.meta.shape))
        return c, q.narrow_workspace(c)
    c = q.PagedCache.allocate_meta(normal(g, nph, Hkv, P, D), normal(g, nph, Hkv, P, D), bt, sl, Hq)
    c.meta.copy_(normal(g, *c.meta.shape))
    return c, q.window_workspace(c)


NAMES = ("k_pool", "v_pool", "meta", "seq_lens", "k_scale", "v_scale", "k_open", "v_open")


def copy_of(c):
    t = {n: getattr(c, n).clone() for n in NAMES if hasattr(c, n)}
    return type(c)(**t, block_table=c.block_table, num_q_heads=c.desc.num_q_heads)


def same(a, b, behind=True):
    """Bit for bit; `behind`: the open pages' rows behind the sequences' ends too (a page filled in
    one call never goes through them, one filled in several does)."""
    live = torch.arange(a.page_size, device="cuda") < (a.seq_lens % a.page_size)[:, None]
    for n in NAMES:
        if hasattr(a, n):
            x, y = getattr(a, n), getattr(b, n)
            if n.endswith("open") and not behind:
                x, y = (torch.where(live[:, None, :, None], t, 0.0) for t in (x, y))
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), n


WRITES = [  # lens, n, Hq, Hkv
    ([0], 1, 1, 1), ([0, 5, 15, 31, 47], 1, 8, 2), ([16, 32, 0], 1, 4, 4), ([31] * 3, 1, 32, 32),
    ([0, 1, 30], 2, 8, 1), ([0, 17], 40, 6 * 2, 6), ([3, 16, 31, 0], 33, 8, 8), ([5], 100, 40, 5),
    ([64], 64, 16, 16), ([15, 14], 17, 3, 3)]


@pytest.mark.parametrize("narrow", [False, True], ids=["paged", "narrow"])
@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("lens,n,Hq,Hkv", WRITES)
def test_writes_are_rotate_then_write(lens, n, Hq, Hkv, P, narrow):
    g, B = gen(len(lens) * 1000 + n * 10 + P), len(lens)
    c, ws = paged(g, B, Hq, Hkv, P, lens, 12, narrow)
    for rope, offsets in ((q.Rope(), False), (q.Rope(40, interleaved=True), True)):
        rows = normal(g, B, n, Hq + 2 * Hkv, D)
        qq, k, v = rows[:, :, :Hq], rows[:, :, Hq:Hq + Hkv], rows[:, :, Hq + Hkv:]
        off = (torch.randint(-1000, 100000, (B,), generator=g, device="cuda", dtype=torch.int32)
               if offsets else None)
        a, b = copy_of(c), copy_of(c)
        pos = c.seq_lens[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
        if offsets:
            pos = pos + off[:, None]
        pos = pos.to(torch.int32).contiguous()
        want_q, turned_k = q.rotate(rope, qq, pos), q.rotate(rope, k, pos)
        write = q.narrow_prefill if narrow else q.prefill
        write(a, turned_k, v.contiguous(), ws)
        call = q.narrow_prefill_rotary if narrow else q.prefill_rotary
        got_q = call(b, rope, qq, k, v, ws, offsets=off)
        assert torch.equal(got_q, want_q)
        same(a, b)
        if n == 1:  # the single-token forms
            one = q.narrow_append_rotary if narrow else q.append_rotary
            d = copy_of(c)
            assert torch.equal(one(d, rope, qq[:, 0], k[:, 0], v[:, 0], ws, offsets=off), want_q[:, 0])
            same(a, d)
            d = copy_of(c)
            plan = q.RotaryPlan(d, rope, ws, offsets=off)
            assert plan.append(qq[:, 0], k[:, 0], v[:, 0]) is plan.q_out
            assert torch.equal(plan.q_out, want_q[:, 0])
            same(a, d)
        d = copy_of(c)  # keys and values alone
        assert call(d, rope, None, k, v, ws, offsets=off) is None
        same(a, d)
        if n > 1:  # in chunks
            d, cut = copy_of(c), n // 3 + 1
            parts = [call(d, rope, qq[:, s], k[:, s], v[:, s], ws, offsets=off)
                     for s in (slice(0, cut), slice(cut, n)) if s.start < n]
            assert torch.equal(torch.cat(parts, 1), want_q)
            same(a, d, behind=False)
    assert q.read_status(ws)[0] == 0


@pytest.mark.parametrize("n", [1, 21])
def test_writes_of_bf16_match_64_bits(n):
    """bf16 heads are turned in fp32 and rounded to fp16 once."""
    g, B, Hq, Hkv, P = gen(9), 3, 8, 2, 16
    c, ws = paged(g, B, Hq, Hkv, P, [0, 13, 16], 8, False)
    rows = normal(g, B, n, Hq + 2 * Hkv, D, dtype=torch.bfloat16)
    qq, k, v = rows[:, :, :Hq], rows[:, :, Hq:Hq + Hkv], rows[:, :, Hq + Hkv:]
    rope = q.Rope(64, scaling="yarn", factor=8.0, original_length=64)
    pos = c.seq_lens[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    got = q.prefill_rotary(c, rope, qq, k, v, ws)
    R.check(got, *R.turned(rope, qq, pos))
    phys = c.block_table.long().gather(1, (pos // P).long())
    slot = (pos % P).long()
    R.check(c.k_pool[phys, :, slot], *R.turned(rope, k, pos))
    assert torch.equal(c.v_pool[phys, :, slot], v.to(torch.float16))
    # the boxes of the pages that began empty, from the keys as stored
    for b, L in enumerate([0, 13, 16]):
        for page in range(-(-L // P), -(-(L + n) // P)):
            rows = c.k_pool[c.block_table[b, page].long(), :, :min(P, L + n - page * P)]
            assert torch.equal(c.meta[b, :, page, 0], rows.amin(1))
            assert torch.equal(c.meta[b, :, page, 1], rows.amax(1))


def test_queries_may_be_turned_in_place():
    g = gen(10)
    c, ws = paged(g, 2, 8, 2, 16, [3, 20], 8, False)
    rope = q.Rope()
    k, v, qq = normal(g, 2, 19, 2, D), normal(g, 2, 19, 2, D), normal(g, 2, 19, 8, D)
    want = q.prefill_rotary(copy_of(c), rope, qq, k, v, ws)
    assert q.prefill_rotary(copy_of(c), rope, qq, k, v, ws, q_out=qq) is qq
    assert torch.equal(qq, want)


@pytest.mark.parametrize("narrow", [False, True], ids=["paged", "narrow"])
@pytest.mark.parametrize("n", [1, 20])
def test_a_sequence_that_does_not_fit_is_reported(narrow, n):
    """No room, an unmapped page: the status says so, that sequence's length stays, the others are
    written."""
    for fault in ("room", "page", "length"):
        g = gen(11)
        c, ws = paged(g, 3, 4, 2, 16, [16, 30, 5], 4, narrow)
        if fault == "room":
            c.seq_lens[1] = 64 - n + 1
        elif fault == "length":
            c.seq_lens[1] = -3
        else:
            c.block_table[1, 1 if n == 1 else 3] = c.k_pool.shape[0]
        L1 = int(c.seq_lens[1])
        k, v, qq = normal(g, 3, n, 2, D), normal(g, 3, n, 2, D), normal(g, 3, n, 4, D)
        call = q.narrow_prefill_rotary if narrow else q.prefill_rotary
        got = call(c, q.Rope(), qq, k, v, ws)
        rc, detail = q.read_status(ws)
        assert rc == (q.QUEST_ERR_BAD_PAGE if fault == "page" else q.QUEST_ERR_BAD_LENGTH)
        assert detail[0] == 1
        assert c.seq_lens.tolist() == [16 + n, L1, 5 + n]
        pos = torch.tensor([[16], [5]], device="cuda") + torch.arange(n, device="cuda")
        R.check(got[[0, 2]], *R.turned(q.Rope(), qq[[0, 2]], pos))


def test_rotary_calls_are_captured_and_replayed():
    """A decode step's writes in a CUDA graph on a stream of its own: every replay appends."""
    g = gen(12)
    c, ws = paged(g, 2, 8, 2, 16, [14, 31], 8, False)
    ref = copy_of(c)
    rope = q.Rope()
    qq, k, v = normal(g, 2, 8, D), normal(g, 2, 2, D), normal(g, 2, 2, D)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        plan = q.RotaryPlan(c, rope, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            plan.append(qq, k, v)
            once_more = q.rotate(rope, qq, c.seq_lens)
        for _ in range(4):
            graph.replay()
    torch.cuda.synchronize()
    for _ in range(4):
        want = q.append_rotary(ref, rope, qq, k, v, ws)
    torch.cuda.synchronize()
    same(c, ref)
    assert torch.equal(plan.q_out, want)
    assert torch.equal(once_more, q.rotate(rope, qq, ref.seq_lens))


def test_refusals():
    g = gen(13)
    c, ws = paged(g, 2, 8, 2, 16, [3, 20], 8, False)
    rope = q.Rope()
    x = normal(g, 4, 3, D)
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    for bad in (lambda: q.rotate(rope, x, pos.long()), lambda: q.rotate(rope, x, pos[:3]),
                lambda: q.rotate(rope, x.double(), pos), lambda: q.rotate(rope, x[..., ::2], pos),
                lambda: q.rotate(rope, x[:, ::2], pos), lambda: q.rotate(rope, x[..., :64], pos),
                lambda: q.rotate(rope, x, pos.cpu()), lambda: q.rotate(rope, x.cpu(), pos),
                lambda: q.rotate(rope, x, pos, out=x.float()), lambda: q.rotate(rope, x, pos, out=x[:3]),
                lambda: q.rotate(rope, x, pos, out=x[:1].expand(4, 3, D)),
                lambda: q.rotate(rope, x.transpose(0, 1), pos[:3])):
        with pytest.raises((ValueError, TypeError, q.QuestError)):
            bad()
    flat = normal(g, 4 * 3 * D + 64)
    with pytest.raises(q.QuestError, match="aligned"):
        q.rotate(rope, flat[1:1 + 4 * 3 * D].view(4, 3, D), pos)
    odd = torch.as_strided(flat, (2, 3, D), (3 * D + 4, D, 1))
    with pytest.raises(q.QuestError, match="multiples of 8"):
        q.rotate(rope, odd, pos[:2])
    k, v, qq = normal(g, 2, 5, 2, D), normal(g, 2, 5, 2, D), normal(g, 2, 5, 8, D)
    for bad in (lambda: q.prefill_rotary(c, rope, qq[:, :4], k, v, ws),
                lambda: q.prefill_rotary(c, rope, qq, k, v.bfloat16(), ws),
                lambda: q.prefill_rotary(c, rope, qq.float(), k.float(), v.float(), ws),
                lambda: q.prefill_rotary(c, rope, qq, k[:, :, :1], v, ws),
                lambda: q.prefill_rotary(c, rope, None, k, v, ws, q_out=qq),
                lambda: q.prefill_rotary(c, rope, qq, k, v, ws, q_out=qq.transpose(1, 2)),
                lambda: q.prefill_rotary(c, rope, qq, k, v, ws, offsets=pos),
                lambda: q.prefill_rotary(c, rope, qq, k, v, ws[:64]),
                lambda: q.prefill_rotary(c, rope, qq, k.cpu(), v, ws),
                lambda: q.append_rotary(c, rope, qq, k, v, ws),
                lambda: q.RotaryPlan(c, rope, ws).append(qq[:, 0], k[:, 0], v[:, 0].bfloat16()),
                lambda: q.RotaryPlan(c, rope, ws).append(qq[:, 0], k[:, 0, :1], v[:, 0]),
                lambda: q.RotaryPlan(c, rope, ws).append(None, k[:, 0], v[:, 0]),
                lambda: q.RotaryPlan(c, rope, ws).append(*(t[:, 0].float() for t in (qq, k, v)))):
        with pytest.raises((ValueError, TypeError, q.QuestError)):
            bad()
    with pytest.raises(q.QuestError, match="max_pages"):
        big = normal(g, 2, 129, 2, D)
        q.prefill_rotary(c, rope, None, big, big, ws)
    assert c.seq_lens.tolist() == [3, 20]
    assert q.read_status(ws)[0] == 0
