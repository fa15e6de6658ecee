// quest_prompt_kernel.cu - windowed attention of prompt tokens over a paged fp16 cache, on
// the fifth-generation tensor cores (tcgen05, accumulators in TMEM, operands by TMA).
//
// The last n tokens of a sequence are queries; token at position i sees j <= i with j < sink
// or i - j < window.  One CTA owns 256 query rows of one (sequence, kv head): two tiles of
// 128 rows, a row being (token, query head) with the G heads of the group side by side, so
// that a group shares every K / V tile.  The CTA's visible pages form a list (the sinks'
// pages, then the window's), cut into tiles of 128 tokens; each page is fetched by TMA with
// its own coordinates, so a tile is any 8 (or 4) pages and a handful of sinks costs one page
// instead of a tile.
//
// Per K / V tile and query tile, with the running maximum and sum of a softmax:
//   S = Q K^T            tcgen05.mma, both operands in shared memory, S in TMEM
//   P = 2^(S c - m + 8)  the tile's 128 softmax threads, one row each (no shuffles), written
//                        back over S as fp16
//   O += P V             tcgen05.mma, P from TMEM, V in shared memory (MN-major), O in TMEM
// Warps 0-3 and 4-7 are the softmax of the two tiles, warps 8 and 10 fetch, warps 9 and 11
// issue the products of a tile each: while one tile is in its softmax, the tensor core works
// for the other.  The order of issue P V (t, j), Q K^T (t, j + 1) per tile t lets P live in S's
// columns.  Few query rows leave most SMs without work, so then the K / V tiles of a work item
// are shared by several CTAs, whose shares a second kernel joins.
// The maximum m moves only when a row exceeds it by more than 2^6 (then O is rescaled in
// TMEM by the softmax threads themselves), so weights reach 2^14 at most and keep fp16's full
// precision down to 2^-22 of the largest.  P enters the second product as one fp16 number:
// a rounding of 2^-11 per weight, random in sign, against the final rounding to fp16 of the
// same size; its sum l is taken in fp32 before that rounding.  Measured, the distance to the
// result in 64 bits is 1.25 (333 tokens) to 1.4 times (2K chunk, five tokens) that of fp32 sums
// rounded once.
//
// What bounds it: the chain softmax -> P V -> Q K^T -> softmax of a tile.  A tile pair is 4
// products of 128 x 128 x 128 (2048 cycles at the dense rate) and 2 * 128 * 128 exponentials
// (1024 cycles); a tile's softmax takes 1100 cycles, its two products 1024, and each of the two
// hand-overs through a barrier some 300, so a pair takes about 2700; over a whole 8K prompt the
// tensor core is busy for 63 % of the time.  Measured: an 8K prompt of 32 heads with a 4K window
// 345-349 us (1.19 PFLOP/s of visible pairs), a 2K chunk of 32 / 8 heads 110 us (1.25), five tokens
// over a 32K window 33 us (4.0 TB/s: 19 us of them the stream of K and V at the copy rate, the
// rest its start and the join).
#include <cuda.h>
#include <math_constants.h>

#include <algorithm>
#include <cfloat>
#include <mutex>

#include "quest_device.cuh"
#include "quest_tc.cuh"

namespace quest {

namespace {

// Three warpgroups: the softmax of either tile, and the fetch warps (8: Q and K, 10: V) with the
// issue warps (9 and 11, a query tile each).  168 registers a thread hold a softmax row's 128
// scores half by half without a spill; moving registers from the third warpgroup to the others
// made the compiler spill in all of them (a few bytes cost 4 %: local memory waits behind the
// tensor core's reads of shared memory).
constexpr int kPromptThreads = 384;
constexpr int kTileRows = 128;       // query rows of a tile; two tiles a CTA
constexpr int kTileTokens = 128;     // tokens of a K / V tile
constexpr int kTileBytes = kTileTokens * kHeadDim * 2;  // 32 KiB
constexpr int kKvStages = 5;         // K and V tiles in flight, alternating
constexpr int kScores = 3;           // barriers of a query tile's scores, in turn
constexpr int kHalfBytes = kTileBytes / 2;  // 64 dims of every row: one 128-byte swizzle span
constexpr float kBias = 8.f;
constexpr float kLazy = 6.f;

struct PromptSmem {
  static constexpr int q = 0;                             // [2][32 KiB]
  static constexpr int kv = 2 * kTileBytes;               // [kKvStages][32 KiB]
  static constexpr int bars = kv + kKvStages * kTileBytes;
  static constexpr int total = bars + 256;
};
static_assert(PromptSmem::total + 1024 <= (int)kMaxSmem, "shared memory of a CTA");

struct PromptParams {
  Params p;
  int n_tokens, sink, window;
  int log_g;     // log2 of the group size
  int part_rows; // rows of a work item that partials have room for
};

// Shared-memory operand descriptors, 128-byte swizzle: atoms of 8 rows x 64 dims (1 KiB).
// Q tile: the atoms of dims 0-63 of all rows, then those of dims 64-127, kHalfBytes apart.
// K and V tiles: per 8 tokens the atoms of both halves of the dims side by side, so that a
// whole page is one TMA box (two boxes a page took the fetch warp 3200 cycles per tile pair,
// more than the products); 8-token groups are kGroupBytes apart.
constexpr int kAtomBytes = 1024, kGroupBytes = 2 * kAtomBytes;
// fp16 x fp16 -> fp32, 128 x 128 x 16; bit 16: B is MN-major.
constexpr uint32_t kIdescQK = 1u << 4 | (kTileTokens >> 3) << 17 | (kTileRows >> 4) << 24;
constexpr uint32_t kIdescPV = 1u << 4 | 1u << 16 | (kHeadDim >> 3) << 17 | (kTileRows >> 4) << 24;

__device__ __forceinline__ void record(const Params& p, int code, int b, int page) {
  record_at<kSitePrompt>(p, code, b, page);
}
__device__ __forceinline__ bool prompt_wait(const Params& p, uint64_t* bar, uint32_t parity,
                                            volatile int* give_up) {
  return wait_at<kSitePrompt>(p, bar, parity, give_up);
}

struct Bars {
  uint64_t q_full;
  uint64_t kv_full[kKvStages];
  // S of query tile t and K / V tile j is in s_full[t][j % 3]; its completion also says that
  // Q K^T (t, j) and P V (t, j - 1) have read their K and V tiles.  Three of them, so that none
  // completes a further phase while someone still has to ask for the one before: the fetch of
  // tile j waits for the scores of tile j - 2, and the next phase there, tile j + 1's, comes
  // after P V (j) and so after the fetch of both its tiles (with two, tile j's scores, which V (j)
  // has no part in, could overtake a V warp that was late, whose wait then never ended).
  uint64_t s_full[2][kScores], p_full[2], o_full[2], drain[2];
  uint32_t tmem;
  int give_up;
  int fetched[2];  // K and V tiles whose copies have been issued
};
static_assert(sizeof(Bars) <= 256, "barrier area");

// The CTA's list of pages: the sinks', then those from the first token any row's window
// holds to the last row's own.
struct PageList {
  int n_sink, first, count, lo;  // lo: the first position in some row's window
  __device__ __forceinline__ int page(int i) const { return i < n_sink ? i : first + i - n_sink; }
};

// Where split s of this CTA's work item keeps its rows' shares.
__device__ __forceinline__ size_t part_slot(const PromptParams& pp, int s) {
  const unsigned blocks = gridDim.x / (unsigned)pp.p.n_splits;
  const unsigned blk = (gridDim.x - 1 - blockIdx.x) / (unsigned)pp.p.n_splits;
  const size_t item = ((size_t)blockIdx.z * pp.p.Hkv + blockIdx.y) * blocks + blk;
  return (item * pp.p.n_splits + s) * pp.part_rows;
}

template <int P>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(PromptParams pp, const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ unsigned char smem_raw[];
  constexpr int PPT = kTileTokens / P;  // pages of a K / V tile
  const Params& p = pp.p;
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Bars& bars = *reinterpret_cast<Bars*>(smem + PromptSmem::bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lg = pp.log_g, G = 1 << lg, TT = kTileRows >> lg;  // tokens of a query tile

  const int blk = (int)(gridDim.x - 1 - blockIdx.x) / p.n_splits;  // the longest rows first
  const int n = pp.n_tokens, tok0 = blk * 2 * TT;
  const int tok1 = min(n, tok0 + 2 * TT);
  const bool two = tok1 - tok0 > TT;
  const int n_q = two ? 2 : 1;  // query tiles with rows

  if (threadIdx.x == 0) {
    mbar_init(&bars.q_full, 1);
    for (int i = 0; i < kKvStages; ++i) {
      mbar_init(&bars.kv_full[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < kScores; ++i) mbar_init(&bars.s_full[t][i], 1);
      mbar_init(&bars.drain[t], 1);
      mbar_init(&bars.p_full[t], two ? 5 : 4);
      mbar_init(&bars.o_full[t], 1);
    }
    bars.give_up = bars.fetched[0] = bars.fetched[1] = 0;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(&bars.tmem);
  if (warp == 8 && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v)
                 : "memory");
  pdl_wait();
  pdl_trigger();

  // ---- the CTA's work (its length and first pages are looked up while the barriers and TMEM
  // are set up)
  const int split = (int)blockIdx.x % p.n_splits;
  const int g = (int)blockIdx.y, b = (int)blockIdx.z;
  int L = p.seq_lens[b];
  if (L < 0 || (long long)L > (long long)p.max_pages * P) {
    if (threadIdx.x == 0) record(p, QUEST_ERR_BAD_LENGTH, b, -1);
    L = 0;
  }
  const int pos0 = L - n;  // position of query token 0 (may be negative)
  const int end = pos0 + tok1;
  PageList list{0, 0, 0, 0};
  if (end > 0) {
    list.lo = max(0, max(0, pos0 + tok0) - pp.window + 1);
    list.first = list.lo / P;
    list.n_sink = min((min(pp.sink, list.lo) + P - 1) / P, list.first);
    list.count = list.n_sink + (end + P - 1) / P - list.first;
  }
  const int tiles = (list.count + PPT - 1) / PPT;
  const int j0 = tiles * split / p.n_splits, j1 = tiles * (split + 1) / p.n_splits;

  // Pages of the list, for the fetch warps: 32 at a time, a page per lane, the next 32 on their
  // way; entries behind the list's end repeat its last page (their tokens are hidden).
  auto entry = [&](int i) {
    return p.block_table[(size_t)b * p.max_pages + list.page(min(i, list.count - 1))];
  };
  int now = 0, next = 0;
  if ((warp == 8 || warp == 10) && j1 > j0) {
    now = entry(j0 * PPT + lane);
    next = entry(j0 * PPT + 32 + lane);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&bars.tmem);
  volatile int* give_up = &bars.give_up;
  if (warp == 8 && elect_lane()) {
    mbar_arrive_expect_tx(&bars.q_full, n_q * kTileBytes);
    for (int i = 0; i < 2 * n_q; ++i)
      tma_3d(smem + PromptSmem::q + (i >> 1) * kTileBytes + (i & 1) * kHalfBytes, &map_q,
             64 * (i & 1), g * G, b * n + tok0 + (i >> 1) * TT, &bars.q_full);
  }
  __syncwarp();

  // A place per row that nothing else uses once the last product of the row's tile is done (the
  // other tile may still be at work on the K / V tiles): the row's start in the tile's queries.
  auto stash = [&](int t, int row) {
    return reinterpret_cast<float2*>(smem + PromptSmem::q + t * kTileBytes + 256 * row);
  };
  bool again = false;
  if (warp >= 8) {
    if (warp == 8 || warp == 10) {
      // ---- fetch: warp 8 the K tiles (the queries are on their way), warp 10 the V tiles
      const int kv = warp == 10;
      if (j1 > j0) {
        auto checked = [&](int phys, int i) {
          if (phys >= 0 && phys < p.num_phys) return phys;
          record(p, QUEST_ERR_BAD_PAGE, b, list.page(min(i, list.count - 1)));
          return 0;
        };
        now = checked(now, j0 * PPT + lane);
        int st = kv, sc = 0;  // the stage; the barrier and phase of the scores of tile j - 2
        uint32_t ph = 0;
        int j = j0;
        for (; j < j1; ++j) {
          // (a test of the waits: the last V tile of a work item never comes)
          if (kv && j == j1 - 1 && (p.debug_flags & QUEST_DEBUG_WITHHOLD_VALUES)) break;
          const int at = (j - j0) * PPT & 31;
          if (at == 0 && j > j0) {
            now = checked(next, j * PPT + lane);
            next = entry(j * PPT + 32 + lane);
          }
          // K (j) takes the stage of V (j - 3), V (j) that of K (j - 2): both are free once
          // the scores of tile j - 2 are there
          if (j - j0 >= 2) {
            bool free = prompt_wait(p, &bars.s_full[0][sc], ph, give_up);
            if (n_q > 1) free = free && prompt_wait(p, &bars.s_full[1][sc], ph, give_up);
            if (++sc == kScores) {
              sc = 0;
              ph ^= 1u;
            }
            if (!__all_sync(0xffffffffu, free)) break;
          }
          const bool leader = elect_lane();
          if (leader) mbar_arrive_expect_tx(&bars.kv_full[st], kTileBytes);
#pragma unroll
          for (int e = 0; e < PPT; ++e) {
            const int phys = __shfl_sync(0xffffffffu, now, at + e);
            if (leader)
              tma_page(smem + PromptSmem::kv + st * kTileBytes + e * P * kHeadDim * 2,
                       kv ? &map_v : &map_k, (phys * p.Hkv + g) * (P / 8), &bars.kv_full[st]);
          }
          __syncwarp();
          if ((st += 2) >= kKvStages) st -= kKvStages;
        }
        if (lane == 0) bars.fetched[kv] = j - j0;
      }
    } else if (warp - 9 < 2 * n_q - 1 && j1 > j0) {
      // ---- issue: warp 9 the products of query tile 0, warp 11 those of tile 1.  (One warp for
      // both spent 1000 cycles of every 3270 between its products, on waits and commits; the
      // other tile's products fill those.)
      const int t = warp == 11;
      // Q and K are K-major: the stride is that of 8-row groups.  V is MN-major: the lead is
      // that of its 64-dim spans, the stride that of 8-token groups.  Address fields count
      // 16 bytes.
      const uint64_t q_desc =
          smem_desc(smem_u32(smem + PromptSmem::q) + t * kTileBytes, 16, kAtomBytes);
      const uint64_t k_desc = smem_desc(smem_u32(smem + PromptSmem::kv), 16, kGroupBytes);
      const uint64_t v_desc = smem_desc(smem_u32(smem + PromptSmem::kv), kAtomBytes, kGroupBytes);
      const uint32_t s_mem = tmem + t * 128, o_mem = tmem + 256 + t * 128;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, prompt_wait(p, bar, parity, give_up)) != 0;
      };
      auto qk = [&](int st, uint64_t* done) {
        if (elect_lane()) {
#pragma unroll
          for (int k = 0; k < kHeadDim / 16; ++k) {
            const uint32_t oq = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
            const uint32_t ok = ((k >> 2) * kAtomBytes + (k & 3) * 32) >> 4;
            mma_ss(s_mem, q_desc + oq, k_desc + (uint32_t)(st * (kTileBytes >> 4)) + ok, kIdescQK,
                   k > 0);
          }
          commit(done);
        }
        __syncwarp();
      };
      bool ok = wait(&bars.q_full, 0) && wait(&bars.kv_full[0], 0);
      fence_after();
      // The two tiles' groups of products, P V (j) with Q K^T (j + 1), take turns: side by side
      // they end together, the two softmaxes then run together too, and nothing overlaps (a
      // tile pair took 4200 cycles so, against 3100 in turns).  The turn is the fifth arrival on
      // p_full, beside the softmax warps': one wait for both.
      if (two && t == 0 && lane == 0) mbar_arrive(&bars.p_full[0]);
      if (ok) qk(0, &bars.s_full[t][0]);
      int sv = 1, sk = 2, sc = 1;  // stages of the V and the next K tile, the next scores' barrier
      uint32_t round_v = 0, round_k = 0;
      for (int j = j0; j < j1 && ok; ++j) {
        const bool more = j + 1 < j1;
        ok = wait(&bars.kv_full[sv], round_v & 1) &&
             (!more || wait(&bars.kv_full[sk], round_k & 1));
        if (!ok) break;
        // Values that no row of the CTA sees (slots behind the last token, tokens between
        // the sinks and the first window) may be anything: 0 * NaN is not 0.  (Both issue
        // warps store these zeros, each before its own products.)
        const int i0 = j * PPT;
        if (i0 <= list.n_sink || (j + 1) * PPT >= list.count) {
          bool touched = false;
          for (int c = lane; c < kTileTokens; c += 32) {
            const int i = i0 + c / P;
            const int pos = list.page(min(i, list.count - 1)) * P + c % P;
            if (i >= list.count || pos >= end || (pos >= pp.sink && pos < list.lo)) {
              touched = true;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                *reinterpret_cast<uint4*>(smem + PromptSmem::kv + sv * kTileBytes +
                                          (c >> 3) * kGroupBytes + (e >> 3) * kAtomBytes +
                                          (c & 7) * 128 + (e & 7) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
          }
          if (touched) fence_proxy_async_smem();
          __syncwarp();
        }
        if (!(ok = wait(&bars.p_full[t], (j - j0) & 1))) break;
        fence_after();
        if (elect_lane()) {
#pragma unroll
          for (int k = 0; k < kTileTokens / 16; ++k)
            mma_ts(o_mem, s_mem + 8 * k,
                   v_desc + (uint32_t)(sv * (kTileBytes >> 4) + k * (2 * kGroupBytes >> 4)),
                   kIdescPV, j > j0 || k > 0);
          if (!more) commit(&bars.o_full[t]);
        }
        __syncwarp();
        if (more) qk(sk, &bars.s_full[t][sc]);
        if (++sc == kScores) sc = 0;
        if (two && lane == 0) mbar_arrive(&bars.p_full[t ^ 1]);
        __syncwarp();
        if ((sv += 2) >= kKvStages) {
          sv -= kKvStages;
          ++round_v;
        }
        if ((sk += 2) >= kKvStages) {
          sk -= kKvStages;
          ++round_k;
        }
      }
    }
  } else {
    // ---- softmax: a thread a row
    const int t = warp >> 2, row = threadIdx.x & 127;
    const int tok = tok0 + t * TT + (row >> lg);
    const int pr = pos0 + tok;  // the row's position
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lanes + t * 128, o_col = tmem + lanes + 256 + t * 128;
    float m = -CUDART_INF_F, l = 0.f;
    bool ok = true;
    if (t < n_q) {
      const int r0 = pos0 + tok0 + t * TT;
      const int r1 = min(r0 + TT, end) - 1;
      for (int j = j0; j < j1; ++j) {
        const uint32_t turn = (uint32_t)(j - j0) / kScores;  // (counters would spill here)
        ok = __all_sync(0xffffffffu, prompt_wait(p, &bars.s_full[t][(uint32_t)(j - j0) - turn * kScores],
                                                 turn & 1, give_up));
        if (!ok) break;
        const int i0 = j * PPT;
        fence_after();
        const int base = (list.first + i0 - list.n_sink) * P;
        const bool whole = i0 >= list.n_sink && i0 + PPT <= list.count &&
                           base + kTileTokens - 1 <= r0 &&
                           (base > r1 - pp.window || base + kTileTokens <= pp.sink);
        if (!whole) {
          // Hidden tokens' scores become -inf in TMEM before the common path (a mask inside
          // it costs every tile the registers and the order of its instructions).  32
          // tokens at a time as bits: page by page those up to the row's own position that
          // are in its window or among the sinks.
#pragma unroll 1
          for (int u = 0; u < 4; ++u) {
            uint32_t x[32], bits = 0;
            tmem_ld32(s_col + 32 * u, x);
#pragma unroll
            for (int e = 0; e < 32 / P; ++e) {
              const int i = i0 + u * (32 / P) + e, at = list.page(i) * P;
              const int hi = min(max(pr + 1 - at, 0), P);
              const int lo = min(max(pr + 1 - pp.window - at, 0), P);
              const int sk = min(max(pp.sink - at, 0), P);
              const uint32_t b32 = low_bits(hi) & (~low_bits(lo) | low_bits(sk));
              bits |= (i < list.count ? b32 : 0u) << (P * e & 31);
            }
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(bits & 1u << k)) x[k] = 0xff800000u;
            tmem_st32(s_col + 32 * u, x);
          }
          tmem_wait_st();
        }
        // 32 scores at s + 32 u: their weights against the reference m
        uint32_t w[kTileTokens / 2];
        uint64_t sum[2] = {0, 0};
        auto weigh = [&](const float* s, int u) {
          const float shift = kBias - (m == -CUDART_INF_F ? 0.f : m);
          const uint64_t shift2 = pair(shift, shift), scale2 = pair(p.qscale, p.qscale);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float a, c;
            unpair(fma2(pair(s[2 * k], s[2 * k + 1]), scale2, shift2), a, c);
            a = ex2(a);
            c = ex2(c);
            sum[k & 1] = add2(sum[k & 1], pair(a, c));
            w[16 * u + k] = pack2(a, c);
          }
        };
        // The weights are taken against the reference as it is, the maximum beside them (the two
        // use different pipes).  Where a row exceeds the reference by 2^kLazy the warp's rows
        // move theirs, l and O with them, and take the weights again from S, which P has not
        // replaced yet.
        float top;
        {
          float best[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float s[64];
            tmem_ld32(s_col + 64 * h, reinterpret_cast<uint32_t*>(s));
            tmem_ld32(s_col + 64 * h + 32, reinterpret_cast<uint32_t*>(s) + 32);
            tmem_wait_ld();
            // two chains of three-input maxima and two of sums: four of each spill, one waits on
            // itself
#pragma unroll
            for (int k = 0; k < 64; k += 4)
#pragma unroll
              for (int e = 0; e < 2; ++e) best[e] = max3(best[e], s[k + e], s[k + 2 + e]);
            weigh(s, 2 * h);
            weigh(s + 32, 2 * h + 1);
          }
          top = fmaxf(best[0], best[1]) * p.qscale;
        }
        if (__any_sync(0xffffffffu, top > m + kLazy)) {
          const float mn = fmaxf(m, top);
          const float f = mn == -CUDART_INF_F ? 1.f : ex2(m - mn);
          m = mn;
          l *= f;
          if (j > j0) {
#pragma unroll 1
            for (int u = 0; u < 8; ++u) {
              uint32_t o[16];
              tmem_ld16(o_col + 16 * u, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(o_col + 16 * u, o);
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) sum[k] = 0;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float s[32];
            tmem_ld32(s_col + 32 * u, reinterpret_cast<uint32_t*>(s));
            tmem_wait_ld();
            weigh(s, u);
          }
        }
        tmem_st32(s_col, w);
        tmem_st32(s_col + 32, w + 32);
        {
          float a, c;
          unpair(add2(sum[0], sum[1]), a, c);
          l += a + c;
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[t]);
      }
      // (where no product ran, the queries have to land before their space is used again)
      if (ok)
        ok = __all_sync(0xffffffffu, prompt_wait(p, j1 > j0 ? &bars.o_full[t] : &bars.q_full, 0,
                                                 give_up));
      fence_after();
      const bool none = l == 0.f;  // (a NaN sum is not: its NaN goes out)
      const bool mine = tok < tok1;
      bool odd = false;  // some of the row's O is not finite
      if (ok && p.n_splits == 1) {
        // ---- out = O / l, through the tile's own query space (its products are done): a row
        // of 256 B per thread goes to shared memory, two rows at a time leave as whole lines
        const size_t row0 = ((size_t)b * n + tok0 + t * TT) * p.Hq + ((size_t)g << lg);
        unsigned char* stage = smem + PromptSmem::q + t * kTileBytes;
        const float inv = none ? 0.f : 1.f / l;
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
          uint32_t o[32];
          if (j1 > j0) {
            tmem_ld32(o_col + 32 * u, o);
            tmem_wait_ld();
            odd |= not_finite(o);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = none ? 0u
                          : pack2(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                  __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
            *reinterpret_cast<uint4*>(stage + row * 256 + (((4 * u + e) ^ (row & 15)) << 4)) =
                make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
        if (mine && p.lse)
          p.lse[row0 + (size_t)(row >> lg) * p.Hq + (row & (G - 1))] =
              none ? -CUDART_INF_F : (m - kBias + log2f(l)) * 0.6931471805599453f;
        __syncwarp();
        const int c = lane & 15;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const int r = (row & ~31) + 2 * i + (lane >> 4);
          if (tok0 + t * TT + (r >> lg) < tok1)
            *reinterpret_cast<uint4*>(
                p.out + (row0 + (size_t)(r >> lg) * p.Hq + (r & (G - 1))) * kHeadDim + 8 * c) =
                *reinterpret_cast<const uint4*>(stage + r * 256 + ((c ^ (r & 15)) << 4));
        }
      } else if (ok) {
        // ---- a split's share: O, m and l as they are (the loads are the whole warp's)
        const size_t slot = part_slot(pp, split) + t * kTileRows + row;
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
          uint32_t o[32];
          if (j1 > j0) {
            tmem_ld32(o_col + 32 * u, o);
            tmem_wait_ld();
            odd |= not_finite(o);
          }
          if (none) {  // (its O may be 0 * NaN)
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (mine) {  // whole sectors: a lane's row is 512 B from its neighbour's
#pragma unroll
            for (int e = 0; e < 4; ++e)
              store8(p.part_acc + slot * kHeadDim + 32 * u + 8 * e, o + 8 * e);
          }
        }
        if (mine) {
          p.part_ml[2 * slot] = m;
          p.part_ml[2 * slot + 1] = l;
        }
      }
      // (m and l of a row that has to be taken again, below; l < 0: it has not)
      again = ok && mine && j1 > j0 && odd && !none && l <= FLT_MAX;
      __syncwarp();
      *stash(t, row) = again ? make_float2(m, l) : make_float2(0.f, -1.f);
    }
  }
  fence_before();
  bool any_again = __syncthreads_or(again);
  fence_after();
  if (*give_up) {  // (nobody sets it any more)
    // A wait ran out: copies and products in flight end before their memory goes.  (Otherwise the
    // results were waited for, and with them everything that went into them.)
    any_again = false;
    if (warp == 9 || warp == 11) {
      if (elect_lane()) commit(&bars.drain[warp == 11]);  // the products that this thread issued
      __syncwarp();
      settle(&bars.drain[warp == 11], 0);
    } else if (warp == 8 && lane < kKvStages) {
      // copies into stage `lane`: K tile j is number 2 j of all, V tile j number 2 j + 1, number u
      // goes to stage u % kKvStages, and as u and u + kKvStages are a K and a V tile, the later of
      // them only once the earlier has been used: phase after phase
      int phases = 0;
      for (int kv = 0; kv < 2; ++kv)
        for (int u = kv; u < 2 * bars.fetched[kv]; u += 2) phases += u % kKvStages == lane;
      if (phases > 0) settle(&bars.kv_full[lane], (uint32_t)(phases - 1) & 1);
    } else if (warp == 10 && lane == 0) {
      settle(&bars.q_full, 0);
    }
    __syncthreads();
  }
  if (warp == 9) tmem_free(tmem);

  // An infinity or NaN among the values of a tile reaches all of its rows, as 0 * NaN, those too
  // that do not see its token.  Such a row (its scores are finite, its O is not) is taken again
  // from what it sees, by a warp, a token at a time.
  if (any_again) {
    for (int r = warp; r < (tok1 - tok0) * G; r += kPromptThreads / 32) {
      const float2 ml = *stash(r / kTileRows, r % kTileRows);
      const float m_r = ml.x, l_r = ml.y;
      if (l_r < 0.f) continue;  // warp-uniform
      const int pos_r = pos0 + tok0 + (r >> lg);
      const size_t at = (((size_t)b * n + tok0 + (r >> lg)) * p.Hq + ((size_t)g << lg) +
                         (r & (G - 1))) * kHeadDim + 4 * lane;
      const uint2 qw = *reinterpret_cast<const uint2*>(p.q + at);
      const float2 qa = h2f(qw.x), qb = h2f(qw.y);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      const int last = min(j1 * PPT, list.count);
#pragma unroll 1
      for (int e = j0 * PPT; e < last; ++e) {
        const int lp = list.page(e);
        const int phys = p.block_table[(size_t)b * p.max_pages + lp];
        if (phys < 0 || phys >= p.num_phys) continue;
        const size_t from = ((size_t)phys * p.Hkv + g) * P * kHeadDim + 4 * lane;
#pragma unroll 4
        for (int k = 0; k < P; ++k) {
          const int pos = lp * P + k;
          if (pos > pos_r || (pos >= pp.sink && pos <= pos_r - pp.window)) continue;
          const uint2 kw = *reinterpret_cast<const uint2*>(p.k_pool + from + k * kHeadDim);
          const uint2 vw = *reinterpret_cast<const uint2*>(p.v_pool + from + k * kHeadDim);
          const float2 ka = h2f(kw.x), kb = h2f(kw.y), va = h2f(vw.x), vb = h2f(vw.y);
          const float x = warp_sum(fmaf(qa.x, ka.x, qa.y * ka.y) + fmaf(qb.x, kb.x, qb.y * kb.y));
          // (a visible infinity counts however small its weight: 0 * inf is not it)
          const float w =
              x == -CUDART_INF_F ? 0.f : fmaxf(ex2(fmaf(x, p.qscale, kBias - m_r)), FLT_MIN);
          acc[0] = fmaf(w, va.x, acc[0]);
          acc[1] = fmaf(w, va.y, acc[1]);
          acc[2] = fmaf(w, vb.x, acc[2]);
          acc[3] = fmaf(w, vb.y, acc[3]);
        }
      }
      if (p.n_splits == 1)
        *reinterpret_cast<uint2*>(p.out + at) =
            make_uint2(pack2(acc[0] / l_r, acc[1] / l_r), pack2(acc[2] / l_r, acc[3] / l_r));
      else
        *reinterpret_cast<float4*>(p.part_acc + (part_slot(pp, split) + r) * kHeadDim + 4 * lane) =
            make_float4(acc[0], acc[1], acc[2], acc[3]);
    }
  }
}

// The shares of the rows' splits into out and lse: a warp a row, lane l the dims 4 l .. 4 l + 3
// and the maxima and sums of splits l and l + 32, kTogether shares on their way together.  A
// kernel of its own because the work items are few: joined by the last CTA of each, 20 rows of
// 19 splits took 6 us and 256 rows of 5 splits 27 us, more than the products.
constexpr int kJoinThreads = 128;
template <int kTogether>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(PromptParams pp, int rows,
                                                                   int blocks) {
  pdl_wait();
  pdl_trigger();
  const Params& p = pp.p;
  const int lane = threadIdx.x & 31, lg = pp.log_g, G = 1 << lg, n = p.n_splits;
  const int at = (int)blockIdx.x * (kJoinThreads / 32) + (int)(threadIdx.x >> 5);
  if (at >= rows) return;  // (row of q, out and lse; the warp's)
  const int h = at % p.Hq, tok = at / p.Hq % pp.n_tokens, b = at / p.Hq / pp.n_tokens;
  const int per = 2 * kTileRows >> lg;  // tokens of a work item
  const size_t item = ((size_t)b * p.Hkv + (h >> lg)) * blocks + tok / per;
  const size_t slot = item * n * pp.part_rows + (tok % per) * G + (h & (G - 1));
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + slot;
  const float4* acc = reinterpret_cast<const float4*>(p.part_acc + slot * kHeadDim) + lane;
  const float2 nothing = make_float2(-CUDART_INF_F, 0.f);
  const float2 x = lane < n ? __ldcg(ml + (size_t)lane * pp.part_rows) : nothing;
  const float2 y = lane + 32 < n ? __ldcg(ml + (size_t)(lane + 32) * pp.part_rows) : nothing;
  float fx = 0.f, fy = 0.f, M = 0.f, Z = 0.f;
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += kTogether) {
    float4 a[kTogether];
#pragma unroll
    for (int e = 0; e < kTogether; ++e)
      a[e] = s0 + e < n ? __ldcg(acc + (size_t)(s0 + e) * pp.part_rows * (kHeadDim / 4))
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    if (s0 == 0) {
      M = warp_max(fmaxf(x.x, y.x));
      // an empty split has m = -inf, l and O 0; with NaN scores alone m = -inf too, and l and O NaN;
      // an infinite O stays one under any factor
      fx = x.x == -CUDART_INF_F ? (x.y == 0.f ? 0.f : 1.f) : fmaxf(ex2(x.x - M), FLT_MIN);
      fy = y.x == -CUDART_INF_F ? (y.y == 0.f ? 0.f : 1.f) : fmaxf(ex2(y.x - M), FLT_MIN);
      Z = warp_sum(fmaf(x.y, fx, y.y * fy));
    }
#pragma unroll
    for (int e = 0; e < kTogether; ++e) {
      const int s = s0 + e;
      const float f = __shfl_sync(0xffffffffu, s < 32 ? fx : fy, s & 31);
      A.x = fmaf(a[e].x, f, A.x);
      A.y = fmaf(a[e].y, f, A.y);
      A.z = fmaf(a[e].z, f, A.z);
      A.w = fmaf(a[e].w, f, A.w);
    }
  }
  const bool none = Z == 0.f;
  const float inv = none ? 0.f : 1.f / Z;
  reinterpret_cast<uint2*>(p.out + (size_t)at * kHeadDim)[lane] =
      none ? make_uint2(0u, 0u) : make_uint2(pack2(A.x * inv, A.y * inv), pack2(A.z * inv, A.w * inv));
  if (lane == 0 && p.lse)
    p.lse[at] = none ? -CUDART_INF_F : (M - kBias + log2f(Z)) * 0.6931471805599453f;
}

}  // namespace

static int prompt_blocks(int G, int n_tokens) {
  const int tokens = 2 * kTileRows / G;
  return (n_tokens + tokens - 1) / tokens;
}

int prompt_part_rows(int G, int n_tokens) {
  return (int)std::min<long long>(2 * kTileRows, (long long)n_tokens * G);
}

// Few work items share their K / V tiles with as many CTAs as fill the GPU once, at least two
// tiles each.
int prompt_splits(const Params& p, int n_tokens, int pages, int user_pps) {
  const long long items = (long long)p.B * p.Hkv * prompt_blocks(p.Hq / p.Hkv, n_tokens);
  const int tiles = (pages * p.P + kTileTokens - 1) / kTileTokens;
  long long s = user_pps > 0 ? (pages + user_pps - 1) / user_pps : std::max(1, tiles / 2);
  s = std::min<long long>(s, (user_pps > 0 ? kPromptParts : kPromptParts / 2) / items);
  return (int)std::max<long long>(1, std::min<long long>(s, std::min(tiles, 64)));
}

cudaError_t launch_prompt(const Params& p, int n_tokens, int sink, int window, cudaStream_t s) {
  PromptParams pp{};
  pp.p = p;
  pp.n_tokens = n_tokens;
  pp.sink = std::min(sink, 1 << 30);  // positions stay far below, so sums with these do too
  pp.window = std::min(window, 1 << 30);
  const int G = p.Hq / p.Hkv;
  pp.log_g = G == 8 ? 3 : G / 2;
  pp.part_rows = prompt_part_rows(G, n_tokens);
  CUtensorMap mq, mk, mv;
  const cuuint64_t qd[3] = {kHeadDim, (cuuint64_t)p.Hq, (cuuint64_t)p.B * n_tokens};
  const cuuint64_t qs[2] = {kHeadDim * 2, (cuuint64_t)p.Hq * kHeadDim * 2};
  const cuuint32_t qb[3] = {64, (cuuint32_t)G, (cuuint32_t)(kTileRows / G)};
  cudaError_t e = make_map(&mq, p.q, 3, qd, qs, qb);
  if (e != cudaSuccess) return e;
  // a pool as [8-row group][half of the dims][row][64 dims]
  const cuuint64_t kd[4] = {64, 8, 2, (cuuint64_t)p.num_phys * p.Hkv * (p.P / 8)};
  const cuuint64_t ks[3] = {kHeadDim * 2, kHeadDim, 8 * kHeadDim * 2};
  const cuuint32_t kb[4] = {64, 8, 2, (cuuint32_t)(p.P / 8)};
  if ((e = make_map(&mk, p.k_pool, 4, kd, ks, kb)) != cudaSuccess) return e;
  if ((e = make_map(&mv, p.v_pool, 4, kd, ks, kb)) != cudaSuccess) return e;
  const void* fn = p.P == 16 ? (const void*)prompt_kernel<16> : (const void*)prompt_kernel<32>;
  const size_t smem = PromptSmem::total + 1024;
  if ((e = ensure_smem(fn, smem)) != cudaSuccess) return e;
  void* args[] = {&pp, &mq, &mk, &mv};
  int blocks = prompt_blocks(G, n_tokens);
  e = launch_pdl(fn, dim3((unsigned)(blocks * p.n_splits), p.Hkv, p.B), dim3(kPromptThreads), smem,
                 s, args);
  if (e != cudaSuccess || p.n_splits == 1) return e;
  int rows = p.B * n_tokens * p.Hq;  // at most kPromptParts work items of 256
  void* join_args[] = {&pp, &rows, &blocks};
  constexpr int per = kJoinThreads / 32;
  // (333 tokens of 4 kv heads, 5 splits: 16.2 us in all with eight shares together, 17.5 with
  // sixteen; five tokens over a 32K window, 19 splits: 34.5 and 32.9)
  const void* join = p.n_splits <= 8 ? (const void*)prompt_join_kernel<8>
                                     : (const void*)prompt_join_kernel<16>;
  return launch_pdl(join, dim3((unsigned)((rows + per - 1) / per)),
                    dim3(kJoinThreads), 0, s, join_args);
}

}  // namespace quest
