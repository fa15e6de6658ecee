"""Host-side checks of the narrow-cache and window entry points (no GPU), and the plain forms
that the GPU tests compare with."""
import ctypes

import pytest
import torch

import query_aware_kv_gb300 as q
import span_reference as R
from query_aware_kv_gb300 import build as cuda_build
from test_abi import _c_layout, desc


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return q.load()


def narrow(**kw):
    base = dict(batch=1, num_q_heads=4, num_kv_heads=4, head_dim=128, page_size=16, max_pages=64,
                num_phys=64, k_pool=16, v_pool=32, k_scale=16, v_scale=32, k_open=16, v_open=32,
                meta=48, block_table=64, seq_lens=80)
    base.update(kw)
    return q.QuestNarrowCacheDesc(*[base[f] for f, _ in q.QuestNarrowCacheDesc._fields_])


def test_narrow_struct_matches_the_header(tmp_path):
    fields = [f for f, _ in q.QuestNarrowCacheDesc._fields_]
    size, offsets = _c_layout(tmp_path, "quest_narrow_cache_t", fields)
    assert ctypes.sizeof(q.QuestNarrowCacheDesc) == size
    assert [getattr(q.QuestNarrowCacheDesc, f).offset for f in fields] == offsets


@pytest.mark.parametrize("kw,needle", [
    (dict(head_dim=64), "head_dim"), (dict(page_size=8), "page_size"),
    (dict(num_q_heads=12), "group size"), (dict(max_pages=q.QUEST_MAX_PAGES + 1), "max_pages"),
    (dict(k_scale=0), "NULL"), (dict(v_open=0), "NULL"), (dict(k_open=24), "aligned"),
    (dict(v_scale=18), "aligned"), (dict(k_pool=8), "aligned"), (dict(seq_lens=0), "NULL")])
def test_narrow_descriptors_are_checked(lib, kw, needle):
    d = ctypes.byref(narrow(**kw))
    assert lib.quest_narrow_workspace_size(d, 16, None) == 0
    assert needle in lib.quest_last_error().decode()
    big = 1 << 40
    for rc in (lib.quest_narrow_prefill(d, 16, 16, 8, 256, big, None),
               lib.quest_narrow_append(d, 16, 16, 256, big, None),
               lib.quest_narrow_dense_decode(d, 16, 16, None, 256, big, None, None),
               lib.quest_narrow_decode(d, 16, 4, 16, None, None, None, 256, big, None, None),
               lib.quest_narrow_window_decode(d, 16, 0, 9, 16, None, 256, big, None, None)):
        assert rc in (q.QUEST_ERR_INVALID_ARG, q.QUEST_ERR_UNSUPPORTED)


def test_narrow_calls_refuse_bad_arguments(lib):
    d = ctypes.byref(narrow())
    big = 1 << 40
    bad, ws_bad = q.QUEST_ERR_INVALID_ARG, q.QUEST_ERR_WORKSPACE
    assert lib.quest_narrow_workspace_size(d, 0, None) == 0
    assert lib.quest_narrow_workspace_size(None, 4, None) == 0
    assert lib.quest_narrow_prefill(d, 16, 16, -1, 256, big, None) == bad
    assert lib.quest_narrow_prefill(d, 16, 16, 64 * 16 + 1, 256, big, None) == bad
    assert lib.quest_narrow_prefill(d, 16, 24, 8, 256, big, None) == bad
    assert lib.quest_narrow_prefill(d, None, 16, 8, 256, big, None) == bad
    assert lib.quest_narrow_prefill(d, 16, 16, 8, None, big, None) == ws_bad
    assert lib.quest_narrow_prefill(d, 16, 16, 8, 256, 64, None) == ws_bad
    assert lib.quest_narrow_prefill(d, 16, 16, 0, None, 0, None) == q.QUEST_OK
    assert lib.quest_narrow_append(d, 16, None, 256, big, None) == bad
    assert lib.quest_narrow_sparse_decode(d, 16, None, 16, 4, 16, None, 256, big, None, None) == bad
    assert lib.quest_narrow_sparse_decode(d, 16, 16, 16, 0, 16, None, 256, big, None, None) == bad
    assert lib.quest_narrow_dense_decode(d, 18, 16, None, 256, big, None, None) == bad
    assert lib.quest_narrow_dense_decode(d, 16, 16, None, 256, 1024, None, None) == ws_bad
    assert lib.quest_narrow_decode_step(d, 16, None, 16, 4, 16, None, None, None, 256, big, None,
                                        None) == bad
    assert lib.quest_narrow_decode(d, 16, 4, 16, 2, None, None, 256, big, None, None) == bad
    for kw in (dict(gqa_union=True), dict(path=q.QUEST_PATH_FUSED), dict(path=q.QUEST_PATH_STREAM),
               dict(cluster_size=2)):
        o = ctypes.byref(q.opts(**kw))
        assert lib.quest_narrow_decode(d, 16, 4, 16, None, None, None, 256, big, o, None) == \
            q.QUEST_ERR_UNSUPPORTED
    o = ctypes.byref(q.opts(sink_pages=3, local_pages=2))
    assert lib.quest_narrow_decode(d, 16, 4, 16, None, None, None, 256, big, o, None) == bad
    for sink, window in ((-1, 5), (0, 0), (2, -3)):
        assert lib.quest_narrow_window_decode(d, 16, sink, window, 16, None, 256, big, None,
                                              None) == bad
    none = ctypes.byref(narrow(batch=0))
    assert lib.quest_narrow_append(none, 16, 16, 256, big, None) == q.QUEST_OK
    assert lib.quest_narrow_decode(none, 16, 4, 16, None, None, None, 256, big, None, None) == q.QUEST_OK


def test_window_calls_refuse_bad_arguments(lib):
    d = ctypes.byref(desc())
    big = 1 << 40
    bad = q.QUEST_ERR_INVALID_ARG
    assert lib.quest_window_workspace_size(d, 0, None) == 0
    assert lib.quest_window_workspace_size(d, 64 * 16 + 1, None) == 0
    assert 0 < lib.quest_window_workspace_size(d, 1, None)
    for sink, window in ((-1, 5), (0, 0), (2, -3)):
        assert lib.quest_window_decode(d, 16, sink, window, 16, None, 256, big, None, None) == bad
        assert lib.quest_window_prefill(d, 16, 4, sink, window, 16, None, 256, big, None, None) == bad
    assert "window" in lib.quest_last_error().decode()
    assert lib.quest_window_decode(d, 16, 0, 5, 24, None, 256, big, None, None) == bad
    assert lib.quest_window_decode(d, None, 0, 5, 16, None, 256, big, None, None) == bad
    assert lib.quest_window_decode(d, 16, 0, 5, 16, 2, 256, big, None, None) == bad
    assert lib.quest_window_prefill(d, 16, -1, 0, 5, 16, None, 256, big, None, None) == bad
    assert lib.quest_window_prefill(d, 16, 64 * 16 + 1, 0, 5, 16, None, 256, big, None, None) == bad
    assert lib.quest_window_decode(d, 16, 0, 5, 16, None, None, 0, None, None) == \
        q.QUEST_ERR_WORKSPACE
    assert lib.quest_window_prefill(d, 16, 4, 0, 5, 16, None, 256, 64, None, None) == \
        q.QUEST_ERR_WORKSPACE
    assert lib.quest_window_prefill(d, 16, 0, 0, 5, 16, None, None, 0, None, None) == q.QUEST_OK
    none = ctypes.byref(desc(batch=0))
    assert lib.quest_window_decode(none, 16, 0, 5, 16, None, None, 0, None, None) == q.QUEST_OK
    unsupported = ctypes.byref(desc(page_size=64))
    assert lib.quest_window_decode(unsupported, 16, 0, 5, 16, None, 256, big, None, None) == \
        q.QUEST_ERR_UNSUPPORTED


def test_e4m3_reference_rounds_to_nearest_even():
    y = torch.tensor([0.0, 448, 500, 2 ** -9, 2 ** -10, 1.5 * 2 ** -9, 1 + 1 / 16, 1 + 3 / 16, -17.0, 19.0])
    want = torch.tensor([0.0, 448, 448, 2 ** -9, 0, 2 ** -8, 1.0, 1.25, -16.0, 20.0])
    assert torch.equal(R.e4m3(y.double()), want.double())
    x = torch.randn(5000) * 30
    assert torch.equal(R.e4m3(x.half().double()), x.half().float().to(torch.float8_e4m3fn).double())


def test_scale_reference():
    top = torch.tensor([0.0, 448, 449, 224, 2.0 ** -24, 65504]).double()
    assert R.pow2_scale(top).tolist() == [1.0, 1.0, 2.0, 0.5, 2.0 ** -32, 256.0]


def test_window_mask_by_hand():
    m = R.window_mask(6, 3, 1, 2, "cpu")
    assert m.tolist() == [[True, False, True, True, False, False],
                          [True, False, False, True, True, False],
                          [True, False, False, False, True, True]]
    assert R.window_mask(1, 3, 4, 9, "cpu").tolist() == [[False], [False], [True]]


def test_binding_refuses_what_is_not_a_cuda_cache():
    """Tensors of the host, another type, another shape or another order are refused before any
    call of the library."""
    bt, sl = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        q.NarrowCache.allocate(4, 2, 16, bt, sl, 4)
    from query_aware_kv_gb300 import _lib
    with pytest.raises(TypeError, match="torch.Tensor"):
        _lib._need([1], "q", torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        _lib._need(torch.zeros(2, dtype=torch.float16), "q", torch.float16)


def test_workspaces_do_not_shrink_with_more_tokens(lib):
    """A workspace for n query tokens holds what fewer need; options that split more need more."""
    d = ctypes.byref(desc(batch=2, num_q_heads=8, num_kv_heads=4))
    sizes = [lib.quest_window_workspace_size(d, n, None) for n in (1, 2, 5, 31, 64, 300, 1000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert lib.quest_window_workspace_size(d, 5, ctypes.byref(q.opts(pages_per_split=1))) >= sizes[2]
    n = ctypes.byref(narrow())
    assert lib.quest_narrow_workspace_size(n, 64, None) > lib.quest_narrow_workspace_size(n, 1, None)
