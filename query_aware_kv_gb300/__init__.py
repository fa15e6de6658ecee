"""Quest decode-time hot path for GB300 (sm_103a): paged fp16 KV cache with per-page key
min/max boxes, query-aware page scoring, per-head top-K page selection and split-K
sparse flash-decode, as a C-ABI library (``libquest.so``) with a thin ctypes binding; caches
of 8-bit pages (``NarrowCache``), attention with a sliding window and sink tokens, rotary
positions (``Rope``) turned on the way into a cache, and attention over prefixes that sequences
share.

The names below mirror the C entry points of ``include/quest.h``.
"""
from ._lib import (  # noqa: F401
    EXPORTS, HEAD_DIM, QUEST_DEBUG_WITHHOLD_SELECTION, QUEST_DEBUG_WITHHOLD_VALUES, QUEST_ERR_BAD_LENGTH,
    QUEST_ERR_BAD_PAGE, QUEST_ERR_BAD_SELECTION, QUEST_ERR_CUDA, QUEST_ERR_INVALID_ARG,
    QUEST_ERR_TIMEOUT, QUEST_ERR_UNSUPPORTED, QUEST_ERR_WORKSPACE, QUEST_MAX_PAGES, QUEST_OK,
    QUEST_PATH_AUTO, QUEST_PATH_CHAIN, QUEST_PATH_FUSED, QUEST_PATH_STREAM,
    DecodePlan, PagedCache, QuestCacheDesc, QuestError, QuestLayer, QuestOpts, append, build_meta, decode,
    decode_launches, decode_layers, decode_path, decode_step,
    dense_decode, estimate, estimate_heads, load, opts, prefill, read_status, sparse_decode, topk, workspace,
    workspace_init, workspace_size,
    NarrowCache, NarrowPlan, QuestNarrowCacheDesc, WindowPlan, narrow_append, narrow_decode,
    narrow_decode_step, narrow_dense_decode, narrow_prefill, narrow_sparse_decode,
    narrow_window_decode, narrow_workspace, window_decode, window_prefill, window_workspace,
    QuestRope, QuestRotaryIo, RotaryPlan, append_rotary, narrow_append_rotary,
    narrow_prefill_rotary, prefill_rotary, rotate,
    QUEST_MAX_PREFIX_GROUPS, PrefixPlan, QuestPrefixGroup, prefix_decode, prefix_workspace,
)
from .rope import Rope, rope_frequencies  # noqa: F401
