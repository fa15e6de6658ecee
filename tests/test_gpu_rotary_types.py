"""Rotary writes of bf16, into every kind of cache, and of odd numbers: against 64 bits where they go
into an fp16 cache, and bit for bit against the plain writes of the fp16 rows that they leave there."""
import pytest
import torch

import query_aware_kv_gb300 as q
import rotary_reference as R
from test_gpu_rotary import copy_of, gen, normal, paged, same

pytestmark = pytest.mark.gpu
D = 128
INF, NAN = float("inf"), float("nan")
ROPES = {"halves": lambda: q.Rope(64, scaling="yarn", factor=8.0, original_length=64),
         "inter": lambda: q.Rope(96, interleaved=True), "all": lambda: q.Rope()}
LENS = [0, 13, 31, 15]


def parts(rows, hq, hkv):
    return rows[..., :hq, :], rows[..., hq:hq + hkv, :], rows[..., hq + hkv:, :]


def stored(c, pos, name):
    """[B][n][Hkv][128]: the rows of an fp16 cache at these positions."""
    phys = c.block_table.long().gather(1, (pos // c.page_size).long())
    return getattr(c, name)[phys, :, (pos % c.page_size).long()]


@pytest.mark.parametrize("n", [1, 2, 40])
@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("rope", ROPES, ids=str)
def test_bf16_rows_in_both_caches(rope, P, n):
    """Turned in fp32 and rounded to fp16 once; a narrow cache is that of narrow_prefill of the same
    fp16 rows (n = 1: among others a token that completes a page, with rows that are fp16 already)."""
    g, B, hq, hkv = gen(P + n), len(LENS), 8, 2
    c, ws = paged(g, B, hq, hkv, P, LENS, 8, False)
    rows = normal(g, B, n, hq + 2 * hkv, D, dtype=torch.bfloat16)
    qq, k, v = parts(rows, hq, hkv)
    r = ROPES[rope]()
    off = torch.randint(-1000, 100000, (B,), generator=g, device="cuda", dtype=torch.int32)
    pos = c.seq_lens[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    at = (pos + off[:, None]).to(torch.int32)
    got = q.prefill_rotary(c, r, qq, k, v, ws, offsets=off)
    R.check(got, *R.turned(r, qq, at))
    kept = stored(c, pos, "k_pool"), stored(c, pos, "v_pool")
    R.check(kept[0], *R.turned(r, k, at))
    assert torch.equal(kept[1], v.to(torch.float16))
    assert q.read_status(ws)[0] == 0

    nar, nws = paged(g, B, hq, hkv, P, LENS, 8, True)
    want, mine = copy_of(nar), copy_of(nar)
    q.narrow_prefill(want, *(t.contiguous() for t in kept), nws)
    assert torch.equal(q.narrow_prefill_rotary(mine, r, qq, k, v, nws, offsets=off), got)
    same(want, mine)
    if n == 1:
        mine = copy_of(nar)
        plan = q.RotaryPlan(mine, r, nws, offsets=off)
        assert torch.equal(plan.append(qq[:, 0], k[:, 0], v[:, 0]), got[:, 0])
        same(want, mine)
    assert q.read_status(nws)[0] == 0


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_numbers_beyond_fp16_infinities_and_nan(dtype, P, n):
    """A bf16 number beyond fp16's range is stored as an infinity (keys, values, turned queries), NaN
    stays one; boxes, and narrow pages' scales and codes, are those of the plain writes of such rows."""
    g, B, hq, hkv = gen(7 * P + n), len(LENS), 4, 2
    c, ws = paged(g, B, hq, hkv, P, LENS, 8, False)
    rows = normal(g, B, n, hq + 2 * hkv, D, dtype=dtype)
    r = q.Rope(64)
    big = 1e5 if dtype is torch.bfloat16 else INF
    # token 0 of sequences 1 .. 3, every head; the dims from 64 on pass through
    rows[1, 0, :, 70], rows[1, 0, :, 71], rows[2, 0, :, 100] = big, -big, NAN
    rows[3, 0, :, 3], rows[3, n - 1, :, 120] = NAN, -INF
    qq, k, v = parts(rows, hq, hkv)
    pos = c.seq_lens[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    before = copy_of(c)
    got = q.prefill_rotary(c, r, qq, k, v, ws)
    kept = stored(c, pos, "k_pool"), stored(c, pos, "v_pool")
    for x in (got, kept[0], kept[1]):
        assert bool((x[1, 0, :, 70] == INF).all()) and bool((x[1, 0, :, 71] == -INF).all())
        assert bool(torch.isnan(x[2, 0, :, 100]).all()) and bool(torch.isnan(x[3, 0, :, 3]).all())
        assert bool((x[3, n - 1, :, 120] == -INF).all())
    # its pair's other dim takes the NaN too, values are not turned; nothing else is odd
    assert int((~torch.isfinite(kept[0])).sum()) == int((~torch.isfinite(kept[1])).sum()) + hkv
    assert int((~torch.isfinite(kept[1])).sum()) == 5 * hkv
    plain = before
    q.prefill(plain, *(t.contiguous() for t in kept), ws)
    same(plain, c)
    nar, nws = paged(g, B, hq, hkv, P, LENS, 8, True)
    want, mine = copy_of(nar), copy_of(nar)
    q.narrow_prefill(want, *(t.contiguous() for t in kept), nws)
    assert torch.equal(q.narrow_prefill_rotary(mine, r, qq, k, v, nws).view(torch.int16), got.view(torch.int16))
    same(want, mine)
    assert q.read_status(ws)[0] == 0 and q.read_status(nws)[0] == 0


def test_a_turn_that_leaves_fp16s_range():
    """60000 turned by an eighth of a turn leaves 84853 in one dim of its pair and nothing in the other:
    the first is an infinity in fp16, in bf16 it is a number (input and output are rounded: 2^-8)."""
    r = q.Rope.from_frequencies([3.141592653589793 / 4] * 4)
    x = torch.zeros((1, 1, 1, D), device="cuda")
    x[..., 0], x[..., 4] = 60000.0, -60000.0
    pos = torch.ones((1, 1), dtype=torch.int32, device="cuda")
    y = q.rotate(r, x.half(), pos)
    assert float(y[0, 0, 0, 0]) == INF
    assert abs(float(y[0, 0, 0, 4])) < 120000 * 2.0 ** -20  # (rotary_reference's bound)
    y = q.rotate(r, x.bfloat16(), pos)
    assert abs(float(y[0, 0, 0, 0]) / 84853 - 1) < 2 ** -8 + 2 ** -9
    g = gen(3)
    for dtype in (torch.float16, torch.bfloat16):
        c, ws = paged(g, 1, 1, 1, 16, [1], 2, False)
        h = x.to(dtype)
        got = q.prefill_rotary(c, r, h, h, h, ws)
        at = c.block_table[0, 0].long()
        assert float(got[0, 0, 0, 0]) == INF and float(c.k_pool[at, 0, 1, 0]) == INF
        assert float(c.v_pool[at, 0, 1, 0]) == float(h[0, 0, 0, 0].half())


def test_strides_past_31_bits():
    """Tokens and sequences 2.3 G elements apart."""
    g, r, far = gen(5), q.Rope(), 2_300_000_000 // 8 * 8
    base = torch.empty(far + 4096, dtype=torch.float16, device="cuda")
    x = torch.as_strided(base, (2, 3, D), (far, D, 1))
    x.copy_(normal(g, 2, 3, D))
    pos = torch.tensor([5, 70000], dtype=torch.int32, device="cuda")
    want = q.rotate(r, x.contiguous(), pos)
    assert torch.equal(q.rotate(r, x, pos), want)
    for narrow in (False, True):
        for n in (1, 2):
            shape, step = (2, n, 3, D), (far, 3 * D, D, 1)
            k = torch.as_strided(base, shape, step)
            k.copy_(normal(g, *shape))
            c, ws = paged(g, 2, 3, 3, 16, [3, 15], 4, narrow)
            a, b = copy_of(c), copy_of(c)
            call = q.narrow_prefill_rotary if narrow else q.prefill_rotary
            assert torch.equal(call(a, r, k, k, k, ws), call(b, r, *[k.contiguous()] * 3, ws))
            same(a, b)
    x.copy_(normal(g, 2, 3, D))
    want = q.rotate(r, x.contiguous(), pos)
    assert q.rotate(r, x, pos, out=x) is x and torch.equal(x, want)


def test_writes_on_two_streams_at_once():
    """Caches of their own, each written by its stream, beside turns on both."""
    g, r = gen(6), q.Rope(96)
    made = [paged(g, 3, 8, 2, 16, [0, 9, 30], 40, narrow) for narrow in (False, True)]
    rows = [[normal(g, 3, n, 12, D) for n in (100, 1, 37, 1, 200)] for _ in made]
    calls = q.prefill_rotary, q.narrow_prefill_rotary
    want = []
    for (c, ws), xs, call in zip(made, rows, calls):
        a = copy_of(c)
        want.append((a, [call(a, r, *parts(x, 8, 2), ws) for x in xs]))
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [(copy_of(c), []) for c, _ in made]
        outs = [[torch.empty_like(t) for t in w[1]] for w in want]
        torch.cuda.synchronize()
        for i in range(5):
            for (c, _), xs, call, s, o, (_, ws) in zip(got, rows, calls, streams, outs, made):
                call(c, r, *parts(xs[i], 8, 2), ws, q_out=o[i], stream=s)
        torch.cuda.synchronize()
        for (a, t), (b, _), o in zip(want, got, outs):
            same(a, b)
            assert all(torch.equal(x, y) for x, y in zip(t, o))
    assert all(q.read_status(ws)[0] == 0 for _, ws in made)
