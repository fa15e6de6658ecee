"""Host side of rotary positions (no GPU): the descriptor's layout and exactness, the scalings'
frequencies, and the entry points' refusals."""
import ctypes
import math
import random

import pytest

import query_aware_kv_gb300 as q
import rotary_reference as R
from query_aware_kv_gb300 import build as cuda_build
from test_abi import _c_layout, desc
from test_span_abi import narrow

BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()
    return q.load()


@pytest.mark.parametrize("cls,name", [(q.QuestRope, "quest_rope_t"), (q.QuestRotaryIo, "quest_rotary_io_t")])
def test_structs_match_the_header(tmp_path, cls, name):
    fields = [f for f, _ in cls._fields_]
    size, offsets = _c_layout(tmp_path, name, fields)
    assert ctypes.sizeof(cls) == size
    assert [getattr(cls, f).offset for f in fields] == offsets


def test_turns_are_exact():
    rng = random.Random(1)
    f = [1.0, 0.0, -1.0, 2 * math.pi, math.pi, 1e-300, 1e6, -1e6, 1e-19, 5e-20] + \
        [rng.uniform(-4, 4) * 10 ** rng.randint(-9, 5) for _ in range(54)]
    r = q.Rope.from_frequencies(f)
    for x, got in zip(f, r.desc.turns):
        far = ((got << 64) - R._turn(x)) % R.ONE  # in 2^-128ths of a turn
        assert min(far, R.ONE - far) <= 0.51 * 2 ** 64, x
    assert r.rotary_dim == 128 and list(r.inv_freq) == f


def test_a_magnitude_has_two_parts():
    for m in (1.0, 0.75, 0.1 * math.log(8) + 1, -1 / 3, 1e-30):
        d = q.Rope(magnitude=m).desc
        assert d.magnitude == ctypes.c_float(m).value
        assert abs(d.magnitude + d.magnitude_low - m) <= abs(m) * 2.0 ** -48 + 1e-45
    assert q.Rope().desc.magnitude_low == 0.0


def test_scalings():
    base, m = q.rope_frequencies(64, 10000.0)
    assert m == 1.0 and base[0] == 1.0 and base[16] == pytest.approx(0.01, rel=1e-14)
    f, _ = q.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert f == [x / 4 for x in base]
    f, _ = q.rope_frequencies(64, 10000.0, "ntk", 4.0)
    assert f[0] == 1.0 and f[-1] == pytest.approx(base[-1] / 4, rel=1e-12)
    f, m = q.rope_frequencies(64, 10000.0, "bands", 4.0, original_length=1000)
    turns = [1000 * x / (2 * math.pi) for x in base]
    for x, y, t in zip(base, f, turns):
        if t >= 4:
            assert y == x
        elif t <= 1:
            assert y == pytest.approx(x / 4, rel=1e-14)
        else:
            assert x / 4 < y < x
    assert m == 1.0
    f, m = q.rope_frequencies(64, 10000.0, "yarn", 4.0, original_length=1000)
    assert m == pytest.approx(0.1 * math.log(4) + 1)
    assert f[0] == base[0] and f[-1] == pytest.approx(base[-1] / 4)
    assert all(x / 4 <= y * (1 + 1e-14) and y <= x for x, y in zip(base, f))
    assert q.Rope(64, scaling="yarn", factor=4.0, original_length=1000, magnitude=1.0).magnitude == 1.0


@pytest.mark.parametrize("bad", [
    dict(rotary_dim=12), dict(rotary_dim=0), dict(rotary_dim=136), dict(rotary_dim=-8),
    dict(scaling="other"), dict(base=1.0), dict(base=float("inf")), dict(factor=0.0),
    dict(factor=float("nan")), dict(scaling="yarn"), dict(scaling="bands", original_length=0),
    dict(scaling="bands", original_length=10, low_turns=4.0, high_turns=4.0),
    dict(scaling="yarn", original_length=10, beta_fast=1.0), dict(magnitude=float("inf"))])
def test_ropes_are_checked(bad):
    with pytest.raises((ValueError, q.QuestError)):
        q.Rope(**bad)


def test_frequencies_are_checked():
    for f in ([1.0] * 3, [1.0] * 65, [], [float("nan")] * 4, [2e6] * 4):
        with pytest.raises((ValueError, q.QuestError)):
            q.Rope.from_frequencies(f)


def io(**kw):
    base = dict(q=256, k=256, v=256, dtype=0, n_tokens=4, q_out=256)
    strides = {s: kw.pop(s, (1024, 512)) for s in ("q_stride", "k_stride", "v_stride")}
    base.update(kw)
    x = q.QuestRotaryIo(**base)
    for s, v in strides.items():
        getattr(x, s)[:] = v
    return x


def test_rotate_refuses_bad_arguments(lib):
    r, bad = q.Rope(), q.QUEST_ERR_INVALID_ARG
    good = [r.ref, 256, 512, 256, 4, 4, 0, 0, 512, 512, None]
    for at, value in ((0, None), (1, None), (1, 264), (2, 516), (3, None), (3, 258), (4, -1), (5, 0),
                      (6, 3), (6, -1), (7, 2), (8, None), (8, 520), (9, 500), (9, 504), (9, -512)):
        args = list(good)
        args[at] = value
        assert lib.quest_rotate(*args) == bad, (at, value)
    args = list(good)
    args[8], args[9] = 256, 1024  # in place with another stride
    assert lib.quest_rotate(*args) == bad
    args = list(good)
    args[4] = 0
    assert lib.quest_rotate(*args) == q.QUEST_OK
    raw = q.QuestRope()
    args[0], args[4] = ctypes.byref(raw), 4
    assert lib.quest_rotate(*args) == bad
    assert "quest_rope_init" in lib.quest_last_error().decode()


@pytest.mark.parametrize("is_narrow", [False, True])
def test_writes_refuse_bad_arguments(lib, is_narrow):
    r, bad = q.Rope(), q.QUEST_ERR_INVALID_ARG
    fn = lib.quest_narrow_prefill_rotary if is_narrow else lib.quest_prefill_rotary
    d = ctypes.byref(narrow() if is_narrow else desc())

    def call(x, ws=256, n=BIG, rope=r.ref, cache=d):
        return fn(cache, rope, None if x is None else ctypes.byref(x), ws, n, None)

    assert call(None) == bad and call(io(), rope=None) == bad and call(io(), cache=None) == bad
    for kw in (dict(dtype=2), dict(dtype=-1), dict(n_tokens=-1), dict(n_tokens=1 << 30), dict(k=None),
               dict(v=None), dict(k=260), dict(v=264), dict(q=264), dict(q_out=264), dict(q=None),
               dict(q_out=None), dict(q_stride=(4, 8)), dict(k_stride=(8, 4)), dict(v_stride=(3, 8)),
               dict(position_offsets=258)):
        assert call(io(**kw)) == bad, kw
    assert call(io(), ws=None) == q.QUEST_ERR_WORKSPACE
    assert call(io(), n=64) == q.QUEST_ERR_WORKSPACE
    assert call(io(n_tokens=0), ws=None, n=0) == q.QUEST_OK
    odd = narrow(head_dim=64) if is_narrow else desc(head_dim=64)
    assert call(io(), cache=ctypes.byref(odd)) == q.QUEST_ERR_UNSUPPORTED
