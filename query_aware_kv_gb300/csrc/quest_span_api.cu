// quest_span_api.cu - the C entry points of narrow (8-bit) caches and of windowed attention
// (declared in include/quest.h): argument checks, workspace layout and dispatch.  No call
// allocates memory or synchronises.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "quest_internal.h"

using namespace quest;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
int bad(const char* message) { return set_last_error(QUEST_ERR_INVALID_ARG, message); }

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return QUEST_OK;
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return set_last_error(QUEST_ERR_CUDA, msg);
}

int group_of(const quest_cache_t& c) { return c.num_q_heads / c.num_kv_heads; }

// The shape, boxes, block table and lengths of a narrow cache as the checks and kernels
// shared with the fp16 cache take them (its pools are not fp16: no kernel reads them there).
quest_cache_t shared_part(const quest_narrow_cache_t& n) {
  return quest_cache_t{n.batch,     n.num_q_heads, n.num_kv_heads, n.head_dim, n.page_size,
                       n.max_pages, n.num_phys,    n.k_pool,       n.v_pool,   n.meta,
                       n.block_table, n.seq_lens};
}

NarrowPtrs narrow_ptrs(const quest_narrow_cache_t& n) {
  return NarrowPtrs{static_cast<unsigned char*>(n.k_pool), static_cast<unsigned char*>(n.v_pool),
                    n.k_scale, n.v_scale, static_cast<__half*>(n.k_open),
                    static_cast<__half*>(n.v_open)};
}

int check_narrow(const quest_narrow_cache_t* n) {
  if (!n) return bad("cache descriptor is NULL");
  const quest_cache_t c = shared_part(*n);
  int rc = check_cache_desc(&c);
  if (rc || n->batch == 0) return rc;
  if (!n->k_scale || !n->v_scale || !n->k_open || !n->v_open)
    return bad("a cache pointer is NULL (k_scale, v_scale, k_open, v_open)");
  if (!aligned(n->k_scale, 4) || !aligned(n->v_scale, 4) || !aligned(n->k_open, 16) ||
      !aligned(n->v_open, 16))
    return bad("k_open / v_open must be 16-byte aligned, k_scale / v_scale 4-byte aligned");
  return QUEST_OK;
}

int user_split(const quest_opts_t* o) {
  return o && o->pages_per_split > 0 ? std::min(o->pages_per_split, QUEST_MAX_PAGES) : 0;
}

// Workspace: the header and the counters (zero between calls, and at the same place for every
// top_k, n_tokens and opts), what a chain step keeps between its kernels, and the parts of
// split rows.
struct SpanLayout {
  size_t seq_done, arrive, scores, sel_idx, sel_count, part_ml, part_acc, total;
};

SpanLayout span_layout(const quest_cache_t& c, int top_k, const quest_opts_t* o,
                       int n_tokens = 1) {
  SpanLayout L{};
  const size_t nbg = (size_t)c.batch * c.num_kv_heads;
  size_t parts = span_max_parts(c.batch, c.num_kv_heads, user_split(o) > 0) * group_of(c);
  if (n_tokens > 1)
    parts = std::max(parts, (size_t)(user_split(o) ? kPromptParts : kPromptParts / 2) *
                                prompt_part_rows(group_of(c), n_tokens));
  size_t off = sizeof(WsHeader);
  L.seq_done = off;  off = up256(off + (size_t)c.batch * 4);
  L.arrive = off;    off = up256(off + (size_t)kSplitRows * 4);
  L.scores = off;    off = up256(off + (top_k ? nbg * c.max_pages * 4 : 0));
  L.sel_idx = off;   off = up256(off + nbg * (size_t)top_k * 4);
  L.sel_count = off; off = up256(off + (top_k ? nbg * 4 : 0));
  L.part_ml = off;   off = up256(off + parts * 2 * 4);
  L.part_acc = off;  off = up256(off + parts * kHeadDim * 4);
  L.total = off;
  return L;
}

Params make_params(const quest_cache_t& c, void* ws, const SpanLayout& L, const quest_opts_t* o) {
  Params p{};
  p.B = c.batch;
  p.Hq = c.num_q_heads;
  p.Hkv = c.num_kv_heads;
  p.P = c.page_size;
  p.max_pages = c.max_pages;
  p.num_phys = c.num_phys;
  p.k_pool = static_cast<__half*>(c.k_pool);
  p.v_pool = static_cast<__half*>(c.v_pool);
  p.meta = static_cast<__half*>(c.meta);
  p.block_table = c.block_table;
  p.seq_lens = c.seq_lens;
  unsigned char* w = static_cast<unsigned char*>(ws);
  p.status = &reinterpret_cast<WsHeader*>(w)->status;
  p.exited = &reinterpret_cast<WsHeader*>(w)->exited;
  p.seq_done = reinterpret_cast<unsigned*>(w + L.seq_done);
  p.decode_arrive = reinterpret_cast<unsigned*>(w + L.arrive);
  p.scores = reinterpret_cast<float*>(w + L.scores);
  p.sel_idx = reinterpret_cast<int*>(w + L.sel_idx);
  p.sel_count = reinterpret_cast<int*>(w + L.sel_count);
  p.part_ml = reinterpret_cast<float*>(w + L.part_ml);
  p.part_acc = reinterpret_cast<float*>(w + L.part_acc);
  p.wait_limit_ns = kDefaultWaitNs;
  p.qscale = (float)(1.4426950408889634 / std::sqrt((double)kHeadDim));
  int stp = o && o->score_tile_pages > 0 ? o->score_tile_pages : kDefaultScoreTilePages;
  stp = std::min(stp, (int)c.max_pages);
  p.score_tile_pages = stp;
  p.n_score_tiles = (c.max_pages + stp - 1) / stp;
  if (o) {
    p.sink_pages = o->sink_pages;
    p.local_pages = o->local_pages;
  }
  return p;
}

int check_io(const void* q, const void* out, const float* lse) {
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return bad("q / out must be non-NULL and 16-byte aligned, lse 4-byte aligned");
  return QUEST_OK;
}

int check_visible(int sink_tokens, int window) {
  if (sink_tokens >= 0 && window >= 1) return QUEST_OK;
  char msg[128];
  snprintf(msg, sizeof(msg), "sink_tokens %d must be >= 0 and window %d >= 1", sink_tokens, window);
  return bad(msg);
}

// The most pages a window row reads: the sinks', and the window's, whose ends lie inside a
// page each.
int window_pages(const quest_cache_t& c, int sink, int window) {
  const long long P = c.page_size;
  const long long n = (sink + P - 1) / P + ((long long)window + P - 1) / P + 1;
  return (int)std::min<long long>(n, c.max_pages);
}

// The same for the rows of a prompt work item, up to 256 query tokens.
int prompt_pages(const quest_cache_t& c, int n_tokens, int sink, int window) {
  return window_pages(c, sink, (int)std::min<long long>((long long)window + std::min(n_tokens, 256),
                                                        0x7fffffff));
}

// One span-decode launch over rows of at most `pages` pages.
int run_span(SpanParams& sp, bool narrow, int pages, const quest_opts_t* o, const void* q,
             void* out, float* lse, quest_stream_t stream, const char* what) {
  sp.p.q = static_cast<const __half*>(q);
  sp.p.out = static_cast<__half*>(out);
  sp.p.lse = lse;
  sp.run_pages = user_split(o);
  return launched(launch_span(sp, narrow, pages, static_cast<cudaStream_t>(stream)), what);
}

int check_narrow_opts(const quest_opts_t* o, int top_k) {
  if (!o) return QUEST_OK;
  if (o->gqa_union || o->cluster_size > 0 ||
      (o->path != QUEST_PATH_AUTO && o->path != QUEST_PATH_CHAIN))
    return set_last_error(QUEST_ERR_UNSUPPORTED,
                          "narrow caches decode on the chain path, one selection per kv head");
  if (o->sink_pages < 0 || o->local_pages < 0 ||
      (long long)o->sink_pages + o->local_pages > (long long)top_k)
    return bad("sink_pages and local_pages must be >= 0 with a sum <= top_k");
  return QUEST_OK;
}

int narrow_decode(const quest_narrow_cache_t* cache, const void* q, const void* k_new,
                  const void* v_new, int32_t top_k, void* out, float* lse, int32_t* idx_out,
                  int32_t* count_out, void* ws, size_t ws_bytes, const quest_opts_t* opts,
                  quest_stream_t stream, const char* what) {
  int rc = check_narrow(cache);
  if (rc) return rc;
  if ((rc = check_top_k(top_k))) return rc;
  if ((rc = check_narrow_opts(opts, top_k))) return rc;
  if (cache->batch == 0) return QUEST_OK;
  if ((rc = check_io(q, out, lse))) return rc;
  if (!aligned(idx_out, 4) || !aligned(count_out, 4))
    return bad("idx_out / count_out must be 4-byte aligned");
  if (!aligned(k_new, 16) || !aligned(v_new, 16))
    return bad("k_new / v_new must be 16-byte aligned");
  const quest_cache_t c = shared_part(*cache);
  const SpanLayout L = span_layout(c, top_k, opts);
  if ((rc = check_workspace(ws, ws_bytes, L.total))) return rc;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  SpanParams sp{};
  sp.p = make_params(c, ws, L, opts);
  sp.nar = narrow_ptrs(*cache);
  sp.mode = kSpanList;
  if (idx_out) sp.p.sel_idx = idx_out;
  if (count_out) sp.p.sel_count = count_out;
  sp.p.top_k = top_k;
  sp.p.q = static_cast<const __half*>(q);
  // a step that appends writes the token in the estimate and advances the lengths at its end
  sp.p.k_new = static_cast<const __half*>(k_new);
  sp.p.v_new = static_cast<const __half*>(v_new);
  sp.p.chain_append = k_new ? 1 : 0;
  cudaError_t e = k_new ? launch_narrow_estimate(sp.p, sp.nar, group_of(c), s)
                        : launch_estimate(sp.p, group_of(c), false, s);
  const int pages = std::min(top_k, c.max_pages);
  sp.run_pages = user_split(opts);
  sp.p.chain_select = span_selects(sp, pages) ? 1 : 0;
  if (e == cudaSuccess && !sp.p.chain_select) e = launch_topk(sp.p, s);
  if (e != cudaSuccess) return launched(e, what);
  return run_span(sp, true, pages, opts, q, out, lse, stream, what);
}

}  // namespace

extern "C" {

size_t quest_narrow_workspace_size(const quest_narrow_cache_t* cache, int32_t top_k,
                                   const quest_opts_t* opts) {
  if (check_narrow(cache) || check_top_k(top_k)) return 0;
  const quest_cache_t c = shared_part(*cache);
  return span_layout(c, top_k, opts).total;
}

int quest_narrow_prefill(const quest_narrow_cache_t* cache, const void* k, const void* v,
                         int32_t n_tokens, void* ws, size_t ws_bytes, quest_stream_t stream) {
  int rc = check_narrow(cache);
  if (rc) return rc;
  if (n_tokens < 0) return bad("n_tokens must be >= 0");
  if (cache->batch == 0 || n_tokens == 0) return QUEST_OK;
  if ((long long)n_tokens > (long long)cache->max_pages * cache->page_size)
    return bad("n_tokens exceeds max_pages * page_size");
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16))
    return bad("k / v must be non-NULL and 16-byte aligned");
  const quest_cache_t c = shared_part(*cache);
  const SpanLayout L = span_layout(c, 1, nullptr);
  if ((rc = check_workspace(ws, ws_bytes, L.arrive))) return rc;
  const Params p = make_params(c, ws, L, nullptr);
  return launched(launch_narrow_prefill(p, narrow_ptrs(*cache), static_cast<const __half*>(k),
                                        static_cast<const __half*>(v), n_tokens,
                                        static_cast<cudaStream_t>(stream)),
                  "quest_narrow_prefill");
}

int quest_narrow_append(const quest_narrow_cache_t* cache, const void* k_new, const void* v_new,
                        void* ws, size_t ws_bytes, quest_stream_t stream) {
  int rc = check_narrow(cache);
  if (rc) return rc;
  if (cache->batch == 0) return QUEST_OK;
  if (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16))
    return bad("k_new / v_new must be non-NULL and 16-byte aligned");
  const quest_cache_t c = shared_part(*cache);
  const SpanLayout L = span_layout(c, 1, nullptr);
  if ((rc = check_workspace(ws, ws_bytes, L.arrive))) return rc;
  const Params p = make_params(c, ws, L, nullptr);
  return launched(launch_narrow_append(p, narrow_ptrs(*cache), static_cast<const __half*>(k_new),
                                       static_cast<const __half*>(v_new),
                                       static_cast<cudaStream_t>(stream)),
                  "quest_narrow_append");
}

int quest_narrow_sparse_decode(const quest_narrow_cache_t* cache, const void* q,
                               const int32_t* idx, const int32_t* count, int32_t top_k, void* out,
                               float* lse, void* ws, size_t ws_bytes, const quest_opts_t* opts,
                               quest_stream_t stream) {
  int rc = check_narrow(cache);
  if (rc) return rc;
  if ((rc = check_top_k(top_k))) return rc;
  if (cache->batch == 0) return QUEST_OK;
  if ((rc = check_io(q, out, lse))) return rc;
  if (!idx || !count || !aligned(idx, 4) || !aligned(count, 4))
    return bad("idx / count must be non-NULL and 4-byte aligned");
  const quest_cache_t c = shared_part(*cache);
  const SpanLayout L = span_layout(c, top_k, opts);
  if ((rc = check_workspace(ws, ws_bytes, L.total))) return rc;
  SpanParams sp{};
  sp.p = make_params(c, ws, L, nullptr);
  sp.nar = narrow_ptrs(*cache);
  sp.mode = kSpanList;
  sp.p.sel_idx = const_cast<int*>(idx);
  sp.p.sel_count = const_cast<int*>(count);
  sp.p.top_k = top_k;
  return run_span(sp, true, std::min(top_k, c.max_pages), opts, q, out, lse, stream,
                  "quest_narrow_sparse_decode");
}

int quest_narrow_dense_decode(const quest_narrow_cache_t* cache, const void* q, void* out,
                              float* lse, void* ws, size_t ws_bytes, const quest_opts_t* opts,
                              quest_stream_t stream) {
  int rc = check_narrow(cache);
  if (rc) return rc;
  if (cache->batch == 0) return QUEST_OK;
  if ((rc = check_io(q, out, lse))) return rc;
  const quest_cache_t c = shared_part(*cache);
  const SpanLayout L = span_layout(c, 1, opts);
  if ((rc = check_workspace(ws, ws_bytes, L.total))) return rc;
  SpanParams sp{};
  sp.p = make_params(c, ws, L, nullptr);
  sp.nar = narrow_ptrs(*cache);
  sp.mode = kSpanDense;
  return run_span(sp, true, c.max_pages, opts, q, out, lse, stream, "quest_narrow_dense_decode");
}

int quest_narrow_decode(const quest_narrow_cache_t* cache, const void* q, int32_t top_k,
                        void* out, float* lse, int32_t* idx_out, int32_t* count_out, void* ws,
                        size_t ws_bytes, const quest_opts_t* opts, quest_stream_t stream) {
  return narrow_decode(cache, q, nullptr, nullptr, top_k, out, lse, idx_out, count_out, ws,
                       ws_bytes, opts, stream, "quest_narrow_decode");
}

int quest_narrow_decode_step(const quest_narrow_cache_t* cache, const void* q, const void* k_new,
                             const void* v_new, int32_t top_k, void* out, float* lse,
                             int32_t* idx_out, int32_t* count_out, void* ws, size_t ws_bytes,
                             const quest_opts_t* opts, quest_stream_t stream) {
  if (!k_new || !v_new) return bad("quest_narrow_decode_step needs k_new and v_new");
  return narrow_decode(cache, q, k_new, v_new, top_k, out, lse, idx_out, count_out, ws, ws_bytes,
                       opts, stream, "quest_narrow_decode_step");
}

int quest_narrow_window_decode(const quest_narrow_cache_t* cache, const void* q,
                               int32_t sink_tokens, int32_t window, void* out, float* lse,
                               void* ws, size_t ws_bytes, const quest_opts_t* opts,
                               quest_stream_t stream) {
  int rc = check_narrow(cache);
  if (rc) return rc;
  if ((rc = check_visible(sink_tokens, window))) return rc;
  if (cache->batch == 0) return QUEST_OK;
  if ((rc = check_io(q, out, lse))) return rc;
  const quest_cache_t c = shared_part(*cache);
  const SpanLayout L = span_layout(c, 1, opts);
  if ((rc = check_workspace(ws, ws_bytes, L.total))) return rc;
  SpanParams sp{};
  sp.p = make_params(c, ws, L, nullptr);
  sp.nar = narrow_ptrs(*cache);
  sp.mode = kSpanWindow;
  sp.sink = sink_tokens;
  sp.window = window;
  return run_span(sp, true, window_pages(c, sink_tokens, window), opts, q, out, lse, stream,
                  "quest_narrow_window_decode");
}

size_t quest_window_workspace_size(const quest_cache_t* cache, int32_t n_tokens,
                                   const quest_opts_t* opts) {
  if (check_cache_desc(cache)) return 0;
  if (n_tokens < 1 || (long long)n_tokens > (long long)cache->max_pages * cache->page_size) {
    bad("n_tokens must be in [1, max_pages * page_size]");
    return 0;
  }
  return span_layout(*cache, 0, opts, n_tokens).total;
}

static int window_rows(const quest_cache_t* cache, const void* q, int32_t n_tokens,
                       int32_t sink_tokens, int32_t window, void* out, float* lse, void* ws,
                       size_t ws_bytes, const quest_opts_t* opts, quest_stream_t stream,
                       const char* what) {
  int rc = check_cache_desc(cache);
  if (rc) return rc;
  if ((rc = check_visible(sink_tokens, window))) return rc;
  if (n_tokens < 0 || (long long)n_tokens > (long long)cache->max_pages * cache->page_size)
    return bad("n_tokens must be in [0, max_pages * page_size]");
  if (cache->batch == 0 || n_tokens == 0) return QUEST_OK;
  if ((rc = check_io(q, out, lse))) return rc;
  const SpanLayout L = span_layout(*cache, 0, opts, n_tokens);
  if ((rc = check_workspace(ws, ws_bytes, L.total))) return rc;
  SpanParams sp{};
  sp.p = make_params(*cache, ws, L, nullptr);
  if (n_tokens > 1) {
    sp.p.q = static_cast<const __half*>(q);
    sp.p.out = static_cast<__half*>(out);
    sp.p.lse = lse;
    if (opts && opts->wait_limit_ns > 0) sp.p.wait_limit_ns = opts->wait_limit_ns;
    sp.p.debug_flags = opts ? opts->debug_flags : 0;
    sp.p.n_splits =
        prompt_splits(sp.p, n_tokens, prompt_pages(*cache, n_tokens, sink_tokens, window),
                      user_split(opts));
    return launched(launch_prompt(sp.p, n_tokens, sink_tokens, window,
                                  static_cast<cudaStream_t>(stream)),
                    what);
  }
  sp.mode = kSpanWindow;
  sp.sink = sink_tokens;
  sp.window = window;
  return run_span(sp, false, window_pages(*cache, sink_tokens, window), opts, q, out, lse, stream,
                  what);
}

int quest_window_decode(const quest_cache_t* cache, const void* q, int32_t sink_tokens,
                        int32_t window, void* out, float* lse, void* ws, size_t ws_bytes,
                        const quest_opts_t* opts, quest_stream_t stream) {
  return window_rows(cache, q, 1, sink_tokens, window, out, lse, ws, ws_bytes, opts, stream,
                     "quest_window_decode");
}

int quest_window_prefill(const quest_cache_t* cache, const void* q, int32_t n_tokens,
                         int32_t sink_tokens, int32_t window, void* out, float* lse, void* ws,
                         size_t ws_bytes, const quest_opts_t* opts, quest_stream_t stream) {
  return window_rows(cache, q, n_tokens, sink_tokens, window, out, lse, ws, ws_bytes, opts,
                     stream, "quest_window_prefill");
}

}  // extern "C"
