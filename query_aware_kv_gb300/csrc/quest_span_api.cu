// quest_span_api.cu - the C entry points of narrow (8-bit) caches and of windowed attention
// (declared in include/quest.h): argument checks, workspace layout and dispatch.  No call
// allocates memory or synchronises.
#include <algorithm>
#include <climits>
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
                       int n_tokens = 1, size_t prefix_parts = 0) {
  SpanLayout L{};
  const size_t nbg = (size_t)c.batch * c.num_kv_heads;
  size_t parts = span_max_parts(c.batch, c.num_kv_heads, user_split(o) > 0) * group_of(c);
  if (n_tokens > 1)
    parts = std::max(parts, (size_t)(user_split(o) ? kPromptParts : kPromptParts / 2) *
                                prompt_part_rows(group_of(c), n_tokens));
  parts = std::max(parts, prefix_parts);
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

// ---- prefixes that sequences share
int check_groups(const quest_cache_t& c, const quest_prefix_group_t* groups, int n) {
  if (!groups || n < 1) return bad("groups must be non-NULL, n_groups >= 1");
  if (n > QUEST_MAX_PREFIX_GROUPS)
    return set_last_error(QUEST_ERR_UNSUPPORTED, "n_groups exceeds QUEST_MAX_PREFIX_GROUPS");
  long long total = 0;
  for (int i = 0; i < n; ++i) {
    if (groups[i].count < 1 || groups[i].prefix_tokens < 0 ||
        groups[i].prefix_tokens > (long long)c.max_pages * c.page_size)
      return bad("a group needs count >= 1 and prefix_tokens in [0, max_pages * page_size]");
    total += groups[i].count;
  }
  return total == c.batch ? QUEST_OK : bad("the groups' counts must sum to the batch");
}

// The query tokens of a sequence: a tail's rows are one work item's.
int check_query_tokens(const quest_cache_t& c, int n) {
  if (n < 1) return bad("n_tokens must be >= 1");
  if ((long long)n * group_of(c) <= kPrefixRows) return QUEST_OK;
  return set_last_error(QUEST_ERR_UNSUPPORTED,
                        "n_tokens * (num_q_heads / num_kv_heads) exceeds 128 (quest_window_prefill "
                        "takes any number of query tokens)");
}

// Whether sharing pays: a long prefix, or many tokens that sequences would read again.  Two launches
// and a job's start and end cost some 8 us, and a short prefix comes from L2: 16 sequences of 32 / 8
// heads behind 512 tokens take 9.6 us each for itself and 11.0 shared, 32 behind 256 tokens 13.3 and
// 17.8, 4 of 32 MHA heads behind 1024 tokens 14.3 and 16.4; 32 of 32 / 8 heads behind 512 tokens 15.8
// and 13.4, 4 behind 2048 12.3 and 11.3, 2 behind 8192 17.4 and 14.4.
constexpr int kShareTokens = 1536, kShareTokensInAll = 12288;
// Each for itself, rows are split as the span decode splits them, but for two of its choices, which get
// one wave of plain parts instead.  Clusters on more than 120 SMs (16 rows of eight): their last waits
// for the first (16 rows of 612 tokens 11.7 us, 8.2 in nine parts; of 2248 16.6 and 10.9, of 8000 28.2
// and 17.8).  And a second wave of CTAs, which it takes where the first leaves many SMs empty (22, 26,
// 32, 33, 41 rows, ...), for parts of less than 64 blocks of 16 tokens.  In two waves and in one: 32
// rows of 612 tokens 13.6 and 9.7 us, of up to 8000 26.0 and 25.5, of up to 16000 38.9 and 41.3, of up
// to 64000 116 and 140 (lengths from a quarter of that on; all as long: 15.9 and 11.3 at 1200, 49.6 and
// 45.3 at 16000); 60 rows of up to 2248 20.9 and 17.6, of 8000 36.1 and 38.7; 96 rows of up to 1200
// 19.4 and 14.5, of 4000 31.2 and 34.8; 192 rows of up to 1200 24.1 and 22.0, of 2248 32.4 and 36.4 (all
// as long: 44.5 and 41.0).
constexpr int kClusterCtas = 120, kWaveBlocks = 64;
int one_wave_split(const SpanParams& sp, int pages) {
  const SpanChoice own = span_choice(sp, false, pages);
  const long long rows = (long long)sp.p.B * sp.p.Hkv, ctas = rows * own.splits;
  const bool late = ctas > own.slots && pages * (sp.p.P / 16) < kWaveBlocks * own.splits;
  if (own.splits == 1 || !(late || (own.cluster && ctas > kClusterCtas))) return 0;
  const int parts = (int)std::max(1LL, own.slots / rows);
  return (pages + parts - 1) / parts;
}
constexpr int kPrefixJobs = 96;  // of the prefixes, in one go: five eighths of the SMs, the others
                                 // begin with tails (152: 45.2 us for 40.0 at 32 tails of 512 tokens
                                 // behind 32K, 42.2 for 34.7 at tails of 16)
constexpr int kPrefixStart = 3;  // what a job's start and end cost, in tiles

// How the prefixes are cut.  A job takes `per` K / V tiles, so that the jobs fill the SMs once, or
// twice, ..., whichever takes the fewest tiles one after another.
PrefixTable prefix_cut(const quest_cache_t& c, const quest_prefix_group_t* groups, int n,
                       int n_tokens, const quest_opts_t* o) {
  PrefixTable t{};
  t.n = n;
  const int user = user_split(o);
  const long long token_rows = (long long)n_tokens * group_of(c);
  int first = 0, longest = 0;
  long long again = 0;  // tokens that would be read again
  for (int i = 0; i < n; ++i) {
    const int pages = groups[i].count > 1 ? groups[i].prefix_tokens / c.page_size : 0;
    t.group[i] = PrefixTable::Group{first, groups[i].count, pages, 1, 0, 0};
    first += groups[i].count;
    longest = std::max(longest, pages * c.page_size);
    again += (groups[i].count - 1LL) * pages * c.page_size;
  }
  for (int i = 0; i < n && !user; ++i)  // (where some group shares, any that has a tile does)
    if ((longest < kShareTokens && again < kShareTokensInAll) ||
        t.group[i].pages * c.page_size < kPrefixTokens)
      t.group[i].pages = 0;
  int tiles[QUEST_MAX_PREFIX_GROUPS], items[QUEST_MAX_PREFIX_GROUPS], most = 0;
  for (int i = 0; i < n; ++i) {
    tiles[i] = (t.group[i].pages * c.page_size + kPrefixTokens - 1) / kPrefixTokens;
    items[i] = (int)(c.num_kv_heads *
                     ((t.group[i].count * token_rows + kPrefixRows - 1) / kPrefixRows));
    most = std::max(most, tiles[i]);
  }
  auto ctas = [&](int per) {
    long long sum = 0;
    for (int i = 0; i < n; ++i) sum += (long long)items[i] * ((tiles[i] + per - 1) / per);
    return sum;
  };
  const int least = std::max(2, (most + kPrefixSplits - 1) / kPrefixSplits);
  int per = std::max(1, most);
  if (user) {
    per = std::max(1, user * c.page_size / kPrefixTokens);
    per = std::max(per, (most + kPrefixSplits - 1) / kPrefixSplits);
  } else if (most > least) {
    long long best = 0;
    for (int waves = 1; waves <= 4; ++waves) {
      int lo = least, hi = most;  // the fewest tiles a CTA with that many waves (hi: all of them)
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (ctas(mid) <= (long long)waves * kPrefixJobs) hi = mid;
        else lo = mid + 1;
      }
      const long long cost = (ctas(lo) + kPrefixJobs - 1) / kPrefixJobs * (lo + kPrefixStart);
      if (best == 0 || cost < best) {
        best = cost;
        per = lo;
      }
    }
  }
  long long jobs = 0, parts = 0;
  for (int i = 0; i < n; ++i) {
    PrefixTable::Group& g = t.group[i];
    g.splits = std::max(1, (tiles[i] + per - 1) / per);
    g.cta0 = (int)std::min<long long>(jobs, INT_MAX);
    g.part0 = (int)std::min<long long>(parts, INT_MAX);
    if (g.pages > 0) {
      const long long mine = (long long)items[i] * g.splits;
      jobs += mine;
      parts += mine * std::min<long long>(kPrefixRows, g.count * token_rows);
    }
    t.most_pages = std::max(t.most_pages, c.max_pages - g.pages);
  }
  t.ctas = (int)std::min<long long>(jobs, INT_MAX);
  t.parts = (int)std::min<long long>(parts, INT_MAX);
  return t;
}

// Jobs of a tail: six tiles each.  How many there can be is bound by the table's rows, and to ten
// jobs an SM where every row is as long (then they are longer).
int tail_piece(const quest_cache_t& c, const quest_opts_t* o) {
  const int user = user_split(o);
  return user ? user : 6 * kPrefixTokens / c.page_size;
}
int tail_splits(const quest_cache_t& c, const PrefixTable& t, const quest_opts_t* o) {
  const long long rows = (long long)c.batch * c.num_kv_heads;
  const int piece = tail_piece(c, o);
  long long n = (t.most_pages + piece - 1) / piece;
  if (!user_split(o)) n = std::min(n, 10 * kPrefixSms / rows);
  return (int)std::max(1LL, std::min<long long>(n, kPrefixSplits));
}

// Places of all shares; the kernels count them in 32 bits.
int prefix_parts(const quest_cache_t& c, const PrefixTable& t, int n_tokens, int splits,
                 size_t* parts) {
  const long long tails = (long long)c.batch * n_tokens * c.num_q_heads * splits;
  if (t.parts + tails + t.ctas >= INT_MAX)
    return set_last_error(QUEST_ERR_UNSUPPORTED, "the batch has too many rows for its splits");
  *parts = (size_t)(t.parts + tails);
  return QUEST_OK;
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

namespace quest {

int narrow_write_params(const quest_narrow_cache_t* cache, void* ws, size_t ws_bytes, Params* p,
                        NarrowPtrs* nar) {
  const quest_cache_t c = shared_part(*cache);
  const SpanLayout L = span_layout(c, 1, nullptr);
  const int rc = check_workspace(ws, ws_bytes, L.arrive);
  if (rc) return rc;
  *p = make_params(c, ws, L, nullptr);
  *nar = narrow_ptrs(*cache);
  return QUEST_OK;
}
int check_narrow_desc(const quest_narrow_cache_t* cache) { return check_narrow(cache); }

}  // namespace quest

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

size_t quest_prefix_workspace_size(const quest_cache_t* cache, const quest_prefix_group_t* groups,
                                   int32_t n_groups, int32_t n_tokens, const quest_opts_t* opts) {
  if (check_cache_desc(cache)) return 0;
  if (cache->batch == 0) return span_layout(*cache, 0, opts).total;
  if (check_query_tokens(*cache, n_tokens) || check_groups(*cache, groups, n_groups)) return 0;
  const PrefixTable t = prefix_cut(*cache, groups, n_groups, n_tokens, opts);
  size_t parts = 0;
  if (prefix_parts(*cache, t, n_tokens, tail_splits(*cache, t, opts), &parts)) return 0;
  return span_layout(*cache, 0, opts, 1, parts).total;
}

int quest_prefix_decode(const quest_cache_t* cache, const void* q, int32_t n_tokens,
                        const quest_prefix_group_t* groups, int32_t n_groups, void* out, float* lse,
                        void* ws, size_t ws_bytes, const quest_opts_t* opts,
                        quest_stream_t stream) {
  int rc = check_cache_desc(cache);
  if (rc || cache->batch == 0) return rc;
  if ((rc = check_query_tokens(*cache, n_tokens))) return rc;
  if ((rc = check_groups(*cache, groups, n_groups))) return rc;
  if ((rc = check_io(q, out, lse))) return rc;
  const PrefixTable t = prefix_cut(*cache, groups, n_groups, n_tokens, opts);
  SpanParams sp{};
  const int splits = tail_splits(*cache, t, opts);
  size_t parts = 0;
  if ((rc = prefix_parts(*cache, t, n_tokens, splits, &parts))) return rc;
  const SpanLayout L = span_layout(*cache, 0, opts, 1, parts);
  if ((rc = check_workspace(ws, ws_bytes, L.total))) return rc;
  sp.p = make_params(*cache, ws, L, opts);
  if (t.ctas == 0 && n_tokens == 1) {  // nothing is shared: every sequence on its own
    sp.mode = kSpanDense;
    quest_opts_t some{};
    if (!user_split(opts) && (some.pages_per_split = one_wave_split(sp, cache->max_pages)) > 0)
      opts = &some;
    return run_span(sp, false, cache->max_pages, opts, q, out, lse, stream, "quest_prefix_decode");
  }
  sp.p.q = static_cast<const __half*>(q);
  sp.p.out = static_cast<__half*>(out);
  sp.p.lse = lse;
  if (opts && opts->wait_limit_ns > 0) sp.p.wait_limit_ns = opts->wait_limit_ns;
  if (opts) sp.p.debug_flags = opts->debug_flags;
  return launched(launch_prefix(sp.p, t, n_tokens, splits, tail_piece(*cache, opts),
                                static_cast<cudaStream_t>(stream)),
                  "quest_prefix_decode");
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
