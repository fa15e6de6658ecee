"""Host side of attention over shared prefixes (no GPU): the entry points' refusals, and workspaces
over many cuts of the work."""
import ctypes
import random

import pytest

import query_aware_kv_gb300 as q
from query_aware_kv_gb300 import _lib
from query_aware_kv_gb300 import build as cuda_build
from test_abi import desc
from test_span_devices import Elsewhere

BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()
    return q.load()


def groups(*rows):
    return (q.QuestPrefixGroup * max(1, len(rows)))(*rows), len(rows)


def test_bad_groups_are_refused(lib):
    d = ctypes.byref(desc(batch=4, num_q_heads=8, num_kv_heads=2, max_pages=64))
    for rows in ([], [(3, 0)], [(5, 0)], [(4, -1)], [(4, 64 * 16 + 1)], [(0, 0), (4, 0)], [(-4, 0), (8, 0)],
                 [(2 ** 31 - 1, 0)] * 4, [(1, 0)] * 129):
        arr, n = groups(*rows)
        assert lib.quest_prefix_workspace_size(d, arr, n, 1, None) == 0
        code = lib.quest_prefix_decode(d, 256, 1, arr, n, 256, None, 256, BIG, None, None)
        assert code == (q.QUEST_ERR_UNSUPPORTED if len(rows) > 128 else q.QUEST_ERR_INVALID_ARG)
    assert lib.quest_prefix_workspace_size(d, None, 1, 1, None) == 0


def test_bad_arguments_are_refused(lib):
    c = desc(batch=4, num_q_heads=8, num_kv_heads=2, max_pages=64)
    d, (arr, n) = ctypes.byref(c), groups((4, 500))
    need = lib.quest_prefix_workspace_size(d, arr, n, 1, None)
    assert need > 0
    for args in ((None, 256, None), (256, None, None), (264, 256, None), (256, 264, None), (256, 256, 258)):
        assert lib.quest_prefix_decode(d, args[0], 1, arr, n, args[1], args[2], 256, BIG, None,
                                       None) == q.QUEST_ERR_INVALID_ARG
    assert lib.quest_prefix_decode(d, 256, 1, arr, n, 256, None, 256, need - 1, None, None) == q.QUEST_ERR_WORKSPACE
    assert lib.quest_prefix_decode(d, 256, 1, arr, n, 256, None, None, need, None, None) == q.QUEST_ERR_WORKSPACE
    assert lib.quest_prefix_decode(None, 256, 1, arr, n, 256, None, 256, BIG, None, None) == q.QUEST_ERR_INVALID_ARG
    odd = ctypes.byref(desc(batch=4, num_q_heads=8, num_kv_heads=2, max_pages=64, head_dim=64))
    assert lib.quest_prefix_decode(odd, 256, 1, arr, n, 256, None, 256, BIG, None, None) == q.QUEST_ERR_UNSUPPORTED
    for tokens, code in ((0, q.QUEST_ERR_INVALID_ARG), (-1, q.QUEST_ERR_INVALID_ARG), (33, q.QUEST_ERR_UNSUPPORTED)):
        assert lib.quest_prefix_workspace_size(d, arr, n, tokens, None) == 0
        assert lib.quest_prefix_decode(d, 256, tokens, arr, n, 256, None, 256, BIG, None, None) == code
    assert lib.quest_prefix_workspace_size(d, arr, n, 32, None) >= need
    none = ctypes.byref(desc(batch=0))
    assert lib.quest_prefix_decode(none, None, 1, None, 0, None, None, None, 0, None, None) == q.QUEST_OK


def test_workspaces_stay_in_proportion(lib):
    """Over drawn batches the parts hold every row's shares and no more than a few of the GPU's worth."""
    rng = random.Random(3)
    for _ in range(300):
        G, hkv = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 8, 32])
        rows = [(rng.choice([1, 2, 7, 40, 300]), rng.choice([0, 1, 15, 16, 500, 9000, 200000]))
                for _ in range(rng.randint(1, 6))]
        batch = sum(c for c, _ in rows)
        d = ctypes.byref(desc(batch=batch, num_q_heads=G * hkv, num_kv_heads=hkv, max_pages=16384, num_phys=1 << 20))
        arr, n = groups(*rows)
        for pps in (0, 1, 300):
            o = ctypes.byref(q.opts(pages_per_split=pps))
            size = lib.quest_prefix_workspace_size(d, arr, n, 1, o)
            heads = batch * G * hkv
            assert size > heads * 520  # a share a row at least
            least = heads * 130 * 4 * (65 + 64 if pps else 2 + 64)
            assert size <= least + 4 * 152 * 256 * 520 + (1 << 20)


def test_a_prefix_plan_is_not_launched_on_another_device(monkeypatch):
    monkeypatch.setattr(_lib, "_current_device", lambda: 1)
    for cls, call in ((q.PrefixPlan, lambda p: p.decode(None)), (q.RotaryPlan, lambda p: p.append(None, None, None))):
        p = object.__new__(cls)
        p._dev, p._many = 0, True
        with pytest.raises(ValueError, match="current"):
            call(p)
    assert Elsewhere((1,), 0).get_device() == 0
