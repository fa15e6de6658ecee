// quest_internal.h - declarations shared by the CUDA translation units of libquest.so.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "quest.h"

namespace quest {

constexpr int kHeadDim = 128;
constexpr int kConsumerWarps = 8;           // warps that compute
constexpr int kConsumerThreads = kConsumerWarps * 32;
constexpr int kDecodeThreads = kConsumerThreads + 32;  // + one copy-producer warp
constexpr int kStages = 8;                  // smem ring depth (pages in flight per CTA)
constexpr int kMaxSplits = 256;             // split-K partials per (sequence, q head)
constexpr int kDefaultPagesPerSplit = 8;    // dense decode work items (at least)
constexpr int kMinSparsePagesPerSplit = 16;  // sparse decode work items, by default
constexpr int kDefaultScoreTilePages = 128;
constexpr long long kDefaultWaitNs = 1000000000LL;

// Places in the code that record a device fault (third detail word).
enum FaultSite : int {
  kSiteMeta = 1, kSiteAppend = 2, kSiteScore = 3, kSiteTopk = 4, kSiteDecode = 5,
  kSiteWaitSelection = 6, kSiteWaitStage = 7, kSiteWaitSlot = 8, kSiteSelection = 9,
  kSiteSpan = 10, kSitePrompt = 11, kSitePrefix = 12,
};

// First 256 bytes of the workspace.
struct WsHeader {
  int status;        // QUEST_OK or the first QUEST_ERR_* the device saw
  int detail[3];     // sequence, logical page, fault site
  unsigned exited;   // cluster kernel: CTAs that have left (the last advances the lengths)
  unsigned started;  // stream kernel: CTAs that have read the lengths of an appending step
  unsigned pad[58];
};
static_assert(sizeof(WsHeader) == 256, "header is 256 bytes");

struct Tiling {
  int topk_cap;          // slots per selection row: top_k (min(G * top_k, max_pages) for the
                         // union form of a fused call)
  int score_rows;        // score rows per (b, kv head): 1, or G for the union form
  int score_tile_pages;  // pages per scoring work item
  int n_score_tiles;     // scoring work items per (b, g)
  int pps_sparse, n_splits_sparse;  // selected pages per decode item, items per (b, g)
  int pps_dense, n_splits_dense;
  int max_splits;
};

struct WsLayout {
  size_t score_arrive, ready, decode_arrive;  // u32 [B*Hkv] each
  size_t seq_done;                            // u32 [B]
  size_t skeys;                               // u32 [B*Hkv*max_pages] stream kernel's key
                                              // rows (0 = not written yet; kept zero)
  size_t scores;                              // f32 [B*Hkv*score_rows*max_pages]
  size_t sel_idx, sel_count;                  // i32 [B*Hkv*topk_cap], [B*Hkv]
  size_t part_ml, part_acc;                   // f32 [B*Hq*max_splits*2], [..*128]
  size_t sel_pair;                            // i32x2 [B*Hkv*topk_cap] (logical, physical)
  size_t total;
};

// Everything a kernel needs, passed by value.
struct Params {
  int B, Hq, Hkv, P, max_pages, num_phys;
  __half* k_pool;
  __half* v_pool;
  __half* meta;
  const int* block_table;
  int* seq_lens;

  const __half* q;       // [B][Hq][128]
  __half* out;           // [B][Hq][128]
  float* lse;            // [B][Hq] or null
  float* scores;         // [B][Hkv][max_pages]
  int* sel_idx;          // [B][Hkv][top_k]
  int* sel_count;        // [B][Hkv]
  int top_k;             // row length of sel_idx (= requested K, capped at max_pages)
  int sink_pages, local_pages;  // pages always kept at the start / end of a long sequence

  int score_tile_pages, n_score_tiles;
  int pps, n_splits;     // decode work-item size and count per (b, g)
  int dense;             // decode every page instead of a selection

  int* status;           // -> WsHeader::status (detail follows it)
  unsigned* exited;
  unsigned* score_arrive;
  unsigned* ready;
  unsigned* decode_arrive;
  float* part_ml;        // [B][Hq][n_splits][2]  (running max in log2 units, sum)
  float* part_acc;       // [B][Hq][n_splits][128]

  long long wait_limit_ns;
  int debug_flags;
  float qscale;          // log2(e) / sqrt(128)

  unsigned* seq_done;    // chain decode: kv heads of a sequence merged so far
  int chain_append;      // chain and stream kernel: the step appends k_new; every kernel
                         // sees seq_lens + 1 (when there is room) and the last step of the
                         // call advances seq_lens
  int* sel_pair;         // stream kernel and chain: [B][Hkv][top_k] (logical, physical page)
  int chain_pairs;       // chain: topk_kernel also writes sel_pair, decode_kernel reads it
  int chain_select;      // chain: every decode work item takes its pair's top-K itself
  unsigned* skeys;       // stream kernel: [B][Hkv][max_pages] page keys, 0 until written
  unsigned* started;     // stream kernel: CTAs that have read the lengths
  int hold_lengths;      // stream kernel: append, but leave seq_lens to a later launch
  int sel_ctas;          // stream kernel: the last sel_ctas CTAs of the grid select and merge
  int ring_slots;        // stream kernel: stages in each streaming CTA's ring
                         // (every layer but the last of a multi-layer step)
  const __half* k_new;   // fused step: token appended per (b, g) before scoring, or null
  const __half* v_new;
  unsigned long long* trace;  // one-launch kernels: optional timeline (quest_opts_t.trace)
  int trace_capacity;
};

// Launch with programmatic dependent launch allowed: the kernel may start while the
// previous kernel on the stream finishes; every kernel calls griddepcontrol.wait before
// touching memory an earlier kernel wrote.
inline cudaError_t launch_pdl(const void* fn, dim3 grid, dim3 block, size_t smem,
                              cudaStream_t s, void** args, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

// Dynamic shared memory of the decode-capable kernels (bytes), see quest_device.cuh.
size_t decode_smem_bytes(int G, int P, int topk_keys, int score_tile_pages);
// Raise a kernel's dynamic shared-memory cap (once per device and kernel).
// Per-layer tensors of a multi-layer fused step (the shape, block table and lengths are
// shared by every layer).  Passed by value as a kernel parameter.
struct LayerPtrs {
  __half* k_pool;
  __half* v_pool;
  __half* meta;
  const __half* q;
  const __half* k_new;
  const __half* v_new;
  __half* out;
  float* lse;
};
constexpr int kMaxLayers = 32;
struct LayerTable {
  int n;
  int pad;
  LayerPtrs l[kMaxLayers];
};

cudaError_t ensure_smem(const void* fn, size_t bytes);

// Host-side checks of quest_decode's cache / top_k arguments (status code, error text
// set), and the workspace bytes it needs: `total`, of which the first `zeroed` bytes
// (header, arrival counters, ready flags, key rows) must be zero when a call starts.
int decode_workspace_requirement(const quest_cache_t* cache, int top_k, size_t* total,
                                 size_t* zeroed);
// Record a failure for quest_last_error(); returns `code`.
int set_last_error(int code, const char* message);

cudaError_t launch_build_meta(const Params& p, cudaStream_t s);
cudaError_t launch_append(const Params& p, const __half* k_new, const __half* v_new,
                          cudaStream_t s, bool advance = true);
// seq_lens[b] += n for every sequence with room whose touched pages are mapped.
cudaError_t launch_advance_lengths(const Params& p, int n, cudaStream_t s);
cudaError_t launch_estimate(const Params& p, int G, bool per_head, cudaStream_t s);
cudaError_t launch_topk_union(const Params& p, int row_cap, cudaStream_t s);
cudaError_t launch_prefill(const Params& p, const __half* k, const __half* v, int n,
                           cudaStream_t s);
// Whether QUEST_PATH_AUTO takes the one-launch cluster kernel for this step (see quest.h).
cudaError_t cluster_preferred(int G, int P, int max_pages, int top_k, int nbg, bool* out);
cudaError_t launch_topk(const Params& p, cudaStream_t s);
cudaError_t launch_decode(const Params& p, int G, cudaStream_t s);
size_t cluster_smem_bytes(int G, int P, int max_pages, int cs, int top_k);
bool cluster_any_fits(int G, int P, int max_pages, int top_k);
cudaError_t launch_cluster(const Params& p, const LayerTable& lt, int G, int cs, int max_clusters,
                           cudaStream_t s);
constexpr int kMaxClusterSize = 16;
// The stream kernel (one persistent launch, every CTA on every pair): ring slots for this
// shape (0 if it does not fit), its shared memory, and its launch.
int stream_slots(int G, int P, int max_pages, int top_k, int batch, int hq);
size_t stream_smem_bytes(int G, int P, int max_pages, int top_k, int batch, int hq);
cudaError_t launch_stream(const Params& p, const LayerPtrs& lay, int G, int max_ctas,
                          cudaStream_t s);
// A narrow (8-bit) cache's own tensors (quest_narrow_cache_t); shape, boxes, block table
// and lengths travel in Params.
struct NarrowPtrs {
  unsigned char* k_pool;  // e4m3 [num_phys][Hkv][P][128]
  unsigned char* v_pool;
  float* k_scale;         // [num_phys][Hkv]
  float* v_scale;
  __half* k_open;         // [B][Hkv][P][128]: the rows of each sequence's open page
  __half* v_open;
};

// Which pages a span-decode row attends over.
enum SpanMode : int { kSpanDense = 0, kSpanList = 1, kSpanWindow = 2 };

// One launch of the span decode (quest_span_kernel.cu): one query token per sequence, a row
// per (sequence, kv head).
struct SpanParams {
  Params p;               // part_ml, part_acc: G slots per CTA; decode_arrive: one per row;
                          // with chain_append the launch advances the lengths (exited)
  NarrowPtrs nar;         // narrow caches only
  int mode;               // SpanMode
  int sink, window;       // kSpanWindow, in tokens
  int run_pages;          // pages of a split (0: the launch's choice)
  int cluster;            // a row's CTAs are a cluster (the launch's choice)
};

constexpr int kSplitRows = 1024;  // rows of a launch that splits them, at most (its counters)
// The most parts (rows * splits) that a launch writes; `user`: with run_pages given.
size_t span_max_parts(int batch, int hkv, bool user);
// `pages`: the most that a row has.
// Whether the launch of a narrow chain step takes the selection itself (p.chain_select).
bool span_selects(const SpanParams& sp, int pages);
cudaError_t launch_span(const SpanParams& sp, bool narrow, int pages, cudaStream_t s);
// How that launch would split its rows: CTAs a row, whether they are a cluster, and how many CTAs the
// GPU holds at once.
struct SpanChoice {
  int splits;
  bool cluster;
  int slots;
};
SpanChoice span_choice(const SpanParams& sp, bool narrow, int pages);

// ---- prefixes that sequences share
constexpr int kPrefixRows = 128;    // query rows (sequence, head) of a work item of the prefixes
constexpr int kPrefixTokens = 128;  // tokens of its K / V tiles
// The groups of a batch, in order; passed by value.  A group without pages shares nothing.
struct PrefixTable {
  struct Group {
    int first, count;  // sequences
    int pages;         // of the prefix that is read once
    int splits;        // of its K / V tiles
    int cta0;          // the group's first job
    int part0;         // its first row of part_ml / part_acc
  };
  int n, ctas;    // groups; jobs of the prefixes (0: nothing is shared)
  int parts;      // rows of part_ml / part_acc of the prefixes' shares
  int most_pages; // of a sequence behind its prefix
  Group group[QUEST_MAX_PREFIX_GROUPS];

  // The last group with value(group) <= x.
  template <class F>
  __host__ __device__ int last(int x, F value) const {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (value(group[mid]) <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  }
  // (a group without jobs starts where the next one does)
  __host__ __device__ int group_of_cta(int c) const {
    return last(c, [](const Group& g) { return g.cta0; });
  }
  __host__ __device__ int group_of_seq(int b) const {
    return last(b, [](const Group& g) { return g.first; });
  }
};

constexpr int kPrefixSms = 152;     // CTAs that take jobs (a GB300's SMs)
constexpr int kPrefixSplits = 64;   // of a prefix, and of a tail
// The cuts of the prefixes (t.ctas jobs), then every sequence's and kv head's tail in jobs of
// piece_pages pages, `splits` of them at most (part_ml / part_acc rows from t.parts on), then all
// shares into out and lse: two launches.
cudaError_t launch_prefix(const Params& p, const PrefixTable& t, int n_tokens, int splits,
                          int piece_pages, cudaStream_t s);

// Windowed attention of the last n_tokens tokens of every sequence (quest_prompt_kernel.cu):
// p.n_splits CTAs per work item of 256 query rows, whose shares take prompt_part_rows rows of
// part_ml / part_acc each; splits only while items * splits is at most kPromptParts.  Two
// launches where rows are split (the second joins their shares), one otherwise.
constexpr int kPromptParts = 304;
int prompt_part_rows(int G, int n_tokens);
int prompt_splits(const Params& p, int n_tokens, int pages, int user_pps);
cudaError_t launch_prompt(const Params& p, int n_tokens, int sink, int window, cudaStream_t s);
cudaError_t launch_narrow_prefill(const Params& p, const NarrowPtrs& nar, const __half* k,
                                  const __half* v, int n, cudaStream_t s);
// The estimate of a step that appends p.k_new / p.v_new (p.chain_append).
cudaError_t launch_narrow_estimate(const Params& p, const NarrowPtrs& nar, int G, cudaStream_t s);
cudaError_t launch_narrow_append(const Params& p, const NarrowPtrs& nar, const __half* k_new,
                                 const __half* v_new, cudaStream_t s);
// ---- rotary positions (quest_rotary_kernels.cu)
struct RotateCall {
  const quest_rope_t* rope;
  const void* x;
  void* out;
  const int* positions;
  long long x_stride, out_stride;
  int tokens, heads, dtype, transposed;
};
cudaError_t launch_rotate(const RotateCall& r, cudaStream_t s);
// A chunk into an fp16 cache (nar null) or a narrow one.
cudaError_t launch_rotary_write(const Params& p, const NarrowPtrs* nar, const quest_rope_t& rope,
                                const quest_rotary_io_t& io, cudaStream_t s);

int check_narrow_desc(const quest_narrow_cache_t* cache);
// The cache's part of a narrow write's parameters, after its checks (quest_span_api.cu).
int narrow_write_params(const quest_narrow_cache_t* cache, void* ws, size_t ws_bytes, Params* p,
                        NarrowPtrs* nar);

// Host checks shared with quest_api.cu (status code, error text set).
int check_cache_desc(const quest_cache_t* cache);
int check_top_k(int top_k);
int check_workspace(void* ws, size_t ws_bytes, size_t need);

constexpr int kStreamPiecePages = 8;  // kept pages per decode piece of the stream kernel
constexpr size_t kMaxSmem = 227 * 1024;  // dynamic shared memory of one CTA

}  // namespace quest
