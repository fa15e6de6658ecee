// quest_prefix_kernel.cu - attention of the last token or tokens of every sequence where groups of
// sequences share a prefix, on the fifth-generation tensor cores (tcgen05, accumulators in TMEM,
// operands by TMA).
//
// The work is a queue of jobs, each a run of pages that up to 128 rows attend over, a row being
// (query token, query head): first the cuts of the prefixes, whose rows are a group's query tokens
// with the G heads of a kv head (so that a prefix is read once for all of them), then every
// sequence's own tokens behind its prefix (G rows a query token).  A CTA an SM takes jobs in turn;
// the lengths are on the device only, so nobody could deal them out evenly beforehand.  Per 128
// tokens of a job:
//   S = Q K^T,   P = 2^(S c - m + 8),   O += P V
// with a running maximum m and sum of weights per row, which sees the tokens up to its own position:
// of a prefix all of them but where its sequence is shorter.  P is one fp16 number a weight, off by
// 2^-11 of it at most, sums and O are fp32: outputs are 2.8e-4 from 64 bits (rms, relative) where
// fp16's own rounding makes 2.1e-4.  (The single-token decode has 22 bits a weight.  Here a second
// fp16 number and product took 42.3 us for 40.0, 87.3 for 80.6 and 31.8 for 29.3: a 32K document, an 8K
// prompt with 2K answers, four groups; low parts in other lanes of the same product, for up to 64
// rows, 42.6, 85.8 and 32.1.)  What a job leaves is a share (m, sum, O) per row; prefix_join_kernel
// joins a row's shares.
//
// Eight softmax warps share a tile: warps 0-3 its first 64 tokens, warps 4-7 the other 64, a thread
// a row of 64 scores in registers.  Either half has a maximum, a sum and an O of its own (two O in
// TMEM), so that the halves never wait for one another; they are added at a job's end, in registers.
// Scores have two buffers in TMEM: Q K^T of tile t + 1 runs while tile t is in its softmax, P V
// while tile t + 1 is.  Warps 8 and 9 fetch K and V (a page a TMA box, three tiles of each in
// flight, over the ends of jobs), warp 10 issues the products, warp 11 takes jobs from the queue, one
// ahead of the fetches, warp 12 fetches their queries.
//
// What bounds it: DRAM where there is enough to read.  A tile takes a CTA 0.85 us when nothing waits
// for memory (Q K^T, softmax and P V hand over to one another four times; the tensor core has 1024 of
// these 1650 cycles), which is 64 KiB, so 152 CTAs could take 11.7 TB/s; a job's start and end cost
// 2.2 us with its last tile, of which 0.8 are the share on its way out, and its loads go on
// meanwhile.  Measured: 16 sequences of 32 MHA heads with 2K tokens of their own behind 8K shared ones
// 80 us (483 MB: 6.0 TB/s, 6.7 in the jobs' launch), 32 sequences of 32 / 8 heads with 512 behind
// 32K 40 us (177 MB), of which 3 are the first lengths, pages and tiles, some 4 the last jobs, which
// not every CTA has, and 5 the join with its launch.
//
// (Two chains a CTA, which took whole tiles in turn with an issue warp each, faulted on long runs of
// full row blocks for a reason that was not found, and are not here; tails on the span decode, in a
// launch that starts with the prefixes', took 93 us for the 80 and 45 for the 41: its CTAs do not fit
// beside these, and each begins with its own look-ups.)
#include <math_constants.h>

#include <algorithm>
#include <cfloat>

#include "quest_device.cuh"
#include "quest_tc.cuh"

namespace quest {

namespace {

constexpr int kPrefixThreads = 416;
constexpr int kRows = kPrefixRows, kTokens = kPrefixTokens;
constexpr int kTile = kTokens * kHeadDim * 2;  // 32 KiB
constexpr int kHalf = kTile / 2;  // 64 dims of every row: one 128-byte swizzle span
constexpr int kSlots = 3;         // K tiles, and V tiles, in flight
constexpr float kBias = 8.f;      // as the tail's: shares of both are joined
constexpr float kLazy = 6.f;      // the maximum moves when a row exceeds it by 2^6

// A run of pages that a row block attends over.
struct Job {
  int n;       // tiles, of 128 tokens from page0's first on; 0: its rows see nothing; -1: no more jobs
  int ragged;  // its rows may see different tokens (of a prefix, or of several query tokens)
  int shared;  // of a prefix
  int seq;     // the row of the block table
  int g;       // the kv head
  int page0, end;   // the first page; the position behind the last token
  int q_tok, rows;  // the first query token (of all sequences' counted through); rows in use
  int share;        // the first row's place in part_ml / part_acc
};

struct Bars {
  uint64_t q_full, q_free;                        // a job's queries: fetched; last read
  uint64_t full[kSlots][2], free[kSlots][2];      // of a slot's K and V: fetched; read
  // Scores and weights of a buffer: tile t (of all jobs, counted through) is in buffer t % 2.  Nobody
  // is late by a phase: Q K^T of tile t + 2 is issued after the weights of tile t have been waited
  // for, which every softmax warp gave after it had seen the scores of tile t.
  uint64_t s_full[2], p_full[2];
  // P V of a tile is done.  Who asks for tile t - 1 has seen the scores of tile t, whose barrier
  // also says that P V of tile t - 2 is done.
  uint64_t pv_done;
  uint64_t o_full, o_free;             // a job's O: complete; read
  uint64_t job_full[2], job_free[2];   // a job's description: written; read by every warp
  uint64_t want;                       // a job's K tiles have been asked for: the next may be taken
  uint64_t pair[4];                    // a row's halves have left their maxima and sums
  uint64_t drain;
  Job job[2];
  uint32_t tmem;
  int give_up;
  unsigned moves;             // pages that warps have been through, taking rows again
  int fetched[2], q_fetched;  // K and V tiles, and queries, whose copies have been issued
};

// The queries, then K and V of each slot side by side.  (There is no room to align the start: the
// kernel checks it.)
struct Smem {
  static constexpr int q = 0;
  static constexpr int kv = kTile;  // [kSlots][K, V]
  static constexpr int stash = kv + 2 * kSlots * kTile;  // [2][128] a half's maximum and sum
  static constexpr int bars = stash + 2 * kRows * 8;
  static constexpr int total = bars + 512;
};
static_assert(sizeof(Bars) <= 512, "barrier area");
static_assert(Smem::total <= (int)kMaxSmem, "shared memory of a CTA");

// Operands as in the prompt kernel: Q as the atoms of dims 0-63 of all rows, then those of dims
// 64-127; K and V per 8 tokens the atoms of both halves side by side, so that a page is one box.
constexpr int kAtomBytes = 1024, kGroupBytes = 2 * kAtomBytes;
// fp16 x fp16 -> fp32, 128 x 128 x 16; bit 16: B is MN-major.
constexpr uint32_t kIdescQK = 1u << 4 | (kTokens >> 3) << 17 | (kRows >> 4) << 24;
constexpr uint32_t kIdescPV = 1u << 4 | 1u << 16 | (kHeadDim >> 3) << 17 | (kRows >> 4) << 24;

struct PrefixParams {
  Params p;      // exited: the queue's counter
  int log_g;
  int n;            // query tokens of a sequence
  int splits;       // jobs of a tail, at most
  int piece_pages;  // pages of such a job, where splits allow it
};

// What a sequence of length L has behind its group's prefix: pages, and the jobs they are cut into.
struct Tail {
  int pages, jobs;
};
__device__ __forceinline__ Tail tail_of(const PrefixParams& pp, int first, int L) {
  Tail t;
  t.pages = max(0, (L + pp.p.P - 1) / pp.p.P - first);
  t.jobs = min(pp.splits, max(1, (t.pages + pp.piece_pages - 1) / pp.piece_pages));
  return t;
}

// Job c of the prefixes: of a group's jobs the row blocks vary fastest (those that read the same
// tiles run side by side), then the splits, then the kv heads.
struct Cut {
  int group, at, blk, page0, page1;
};
template <int PPT>
__device__ __forceinline__ Cut cut_of(const PrefixTable& t, int n, int lg, int c) {
  Cut x;
  x.group = t.group_of_cta(c);
  const PrefixTable::Group& q = t.group[x.group];
  const int blocks = ((q.count * n << lg) + kRows - 1) / kRows;
  x.at = c - q.cta0;
  x.blk = x.at % blocks;
  const int split = x.at / blocks % q.splits, tiles = (q.pages + PPT - 1) / PPT;
  x.page0 = tiles * split / q.splits * PPT;
  x.page1 = min(tiles * (split + 1) / q.splits * PPT, q.pages);
  return x;
}

// A wait for the next job, or for what other warps do with this one, which may be a whole job long:
// its limit is a second at least, however short the waits for copies and products may be (one of
// those that runs out ends this one too).  While a warp takes rows of a job again (32 rows of 512K
// tokens take it 3 s) the limit starts anew with every page that it is through.
__device__ __forceinline__ bool idle_wait(const Params& p, uint64_t* bar, uint32_t parity,
                                          volatile int* give_up, const volatile unsigned* moves) {
  if (mbar_try_wait(bar, parity)) return true;
  long long t0 = 0;
  unsigned seen = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 1024; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*give_up) return false;
    const long long now = global_ns();
    const unsigned at = *moves;
    if (t0 == 0 || at != seen) {
      t0 = now;
      seen = at;
    }
    if (now - t0 > max(p.wait_limit_ns, kDefaultWaitNs)) {
      *give_up = 1;
      record_at<kSitePrefix>(p, QUEST_ERR_TIMEOUT, -1, -1);
      return false;
    }
  }
}

// What brings a half's part of a softmax to the maximum M of both (as part_factor of the span
// decode: a part without a weight is 0, one of NaN scores goes on, an infinite O stays one).
__device__ __forceinline__ float half_factor(float m, float l, float M) {
  return m == -CUDART_INF_F ? (l == 0.f ? 0.f : 1.f) : fmaxf(ex2(m - M), FLT_MIN);
}

template <int P>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ PrefixParams pp, const __grid_constant__ PrefixTable table,
                  const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_1,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ __align__(1024) unsigned char smem[];
  constexpr int PPT = kTokens / P;  // pages of a tile
  const Params& p = pp.p;
  if (smem_u32(smem) & 1023) {  // (the swizzle's atoms; no compiler has placed it elsewhere)
    if (threadIdx.x == 0) record_at<kSitePrefix>(p, QUEST_ERR_UNSUPPORTED, -1, -1);
    return;
  }
  Bars& bars = *reinterpret_cast<Bars*>(smem + Smem::bars);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);  // (uniform to the compiler)
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars.q_full, 1);
    mbar_init(&bars.q_free, 1);
    for (int i = 0; i < kSlots; ++i)
      for (int kv = 0; kv < 2; ++kv) {
        mbar_init(&bars.full[i][kv], 1);
        mbar_init(&bars.free[i][kv], 1);
      }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 8);
      mbar_init(&bars.job_full[i], 1);
      mbar_init(&bars.job_free[i], 12);
    }
    mbar_init(&bars.want, 1);
    mbar_init(&bars.pv_done, 1);
    mbar_init(&bars.o_full, 1);
    mbar_init(&bars.o_free, 8);
    for (int i = 0; i < 4; ++i) mbar_init(&bars.pair[i], 2);
    mbar_init(&bars.drain, 1);
    bars.give_up = bars.fetched[0] = bars.fetched[1] = bars.q_fetched = 0;
    bars.moves = 0u;
    fence_mbar_init();
  }
  if (warp == 10) tmem_alloc(&bars.tmem);
  if (warp == 8 && lane < 4)
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0   ? &map_q
                                                  : lane == 1 ? &map_k
                                                  : lane == 2 ? &map_v
                                                              : &map_1)
                 : "memory");
  fence_before();
  __syncthreads();
  fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&bars.tmem);
  volatile int* give_up = &bars.give_up;
  const int lg = pp.log_g, nq = pp.n;

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_at<kSitePrefix>(p, bar, parity, give_up)) != 0;
  };
  auto idle = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, idle_wait(p, bar, parity, give_up, &bars.moves)) != 0;
  };
  auto length = [&](int seq) {
    const int L = p.seq_lens[seq];
    if (L >= 0 && (long long)L <= (long long)p.max_pages * P) return L;
    record_at<kSitePrefix>(p, QUEST_ERR_BAD_LENGTH, seq, -1);
    return 0;
  };
  // The k-th job of the CTA, for every warp but the one that writes them; false: there is none.
  auto take = [&](int k, Job& job) {
    if (!idle(&bars.job_full[k & 1], (uint32_t)(k >> 1) & 1)) return false;
    job = bars.job[k & 1];
    __syncwarp();
    return job.n >= 0;
  };
  // The softmax warps give a job's description back when they are done with the job, the others once
  // they have read it.
  auto give_back = [&](int k) {
    if (lane == 0) mbar_arrive(&bars.job_free[k & 1]);
  };

  if (warp == 11) {
    // ---- jobs
    const int sequences = p.B;
    int index = (int)blockIdx.x;
    // 32 sequences at a time, a sequence a lane: its tail's jobs (of all kv heads), the sum up to it;
    // `base`: the index of the first one's first job
    int b0 = -32, base = table.ctas, chunk = 0, sum = 0, first = 0;
    Tail tail{0, 0};
    int L = 0;
    for (int k = 0;; ++k) {
      Job job{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0};
      if (k > 0) {
        // not before this CTA's fetches are through with the job before: taken any earlier (all
        // CTAs took their first three at the start) the jobs were dealt out, not queued for
        if (!idle(&bars.want, (uint32_t)(k - 1) & 1)) break;
        if (lane == 0) index = (int)(gridDim.x + atomicAdd(p.exited, 1u));
        index = __shfl_sync(0xffffffffu, index, 0);
      }
      if (index < table.ctas) {
        const Cut x = cut_of<PPT>(table, nq, lg, index);
        const PrefixTable::Group& q = table.group[x.group];
        const int tokens = q.count * nq;
        const int tok0 = x.blk * (kRows >> lg), tok1 = min(tokens, tok0 + (kRows >> lg));
        int most = 0;  // the longest of the rows' sequences
        for (int i = tok0 / nq + lane; i * nq < tok1; i += 32) most = max(most, length(q.first + i));
        job.ragged = job.shared = 1;
        job.seq = q.first;
        job.g = x.at / (((tokens << lg) + kRows - 1) / kRows) / q.splits;
        job.page0 = x.page0;
        job.end = min(__reduce_max_sync(0xffffffffu, most), x.page1 * P);
        job.q_tok = q.first * nq + tok0;
        job.rows = (tok1 - tok0) << lg;
        job.share = q.part0 + x.at * min(tokens << lg, kRows);
        job.n = 0;
      } else {
        while (index >= base + chunk && b0 + 32 < sequences) {
          base += chunk;
          b0 += 32;
          const int b = b0 + lane;
          int mine = 0;
          if (b < sequences) {
            L = length(b);
            first = table.group[table.group_of_seq(b)].pages;
            tail = tail_of(pp, first, L);
            mine = tail.jobs * p.Hkv;
          }
          sum = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
          }
          chunk = __shfl_sync(0xffffffffu, sum, 31);
        }
        if (index < base + chunk) {
          const int at = __ffs(__ballot_sync(0xffffffffu, index - base < sum)) - 1;
          const int jobs = __shfl_sync(0xffffffffu, tail.jobs, at);
          const int pages = __shfl_sync(0xffffffffu, tail.pages, at);
          const int start = __shfl_sync(0xffffffffu, first, at);
          const int local = index - base - __shfl_sync(0xffffffffu, sum, at) + jobs * p.Hkv;
          const int split = local / p.Hkv;
          job.ragged = nq > 1;
          job.seq = b0 + at;
          job.q_tok = job.seq * nq;
          job.g = local % p.Hkv;
          job.page0 = start + pages * split / jobs;
          job.end = min(__shfl_sync(0xffffffffu, L, at), (start + pages * (split + 1) / jobs) * P);
          job.rows = nq << lg;
          job.share = table.parts + ((job.seq * p.Hkv + job.g) * pp.splits + split) * job.rows;
          job.n = 0;
        }
      }
      if (job.n == 0) job.n = max(0, job.end - job.page0 * P + kTokens - 1) / kTokens;
      if (k >= 2 && !idle(&bars.job_free[k & 1], (uint32_t)((k >> 1) - 1) & 1)) break;
      if (lane == 0) {
        bars.job[k & 1] = job;
        mbar_arrive(&bars.job_full[k & 1]);
      }
      __syncwarp();
      if (job.n < 0) break;
    }
  } else if (warp == 12) {
    // ---- queries
    Job job;
    int loads = 0;
    for (int k = 0; take(k, job); ++k) {
      give_back(k);
      if (job.n == 0) continue;
      if (loads > 0 && !idle(&bars.q_free, (uint32_t)(loads - 1) & 1)) break;
      if (elect_lane()) {
        // of a tail only its own rows: the others' scores may be anything
        mbar_arrive_expect_tx(&bars.q_full, job.shared ? kTile : kHeadDim * 2 * job.rows);
        for (int i = 0; i < 2; ++i)
          tma_3d(smem + Smem::q + i * kHalf, job.shared ? &map_q : &map_1, 64 * i, job.g << lg,
                 job.q_tok, &bars.q_full);
      }
      __syncwarp();
      ++loads;
    }
    if (lane == 0) bars.q_fetched = loads;
  } else if (warp >= 8 && warp < 10) {
    // ---- fetch: warp 8 the K tiles, warp 9 the V tiles
    const int kv = warp - 8;
    Job job;
    int slot = 0, total = 0;
    uint32_t ph = 1;  // (of the phase before a slot's first: over)
    bool ok = true;
    // the first job's pages are looked up beside its lengths
    int early = 0;
    if ((int)blockIdx.x < table.ctas) {
      const Cut x = cut_of<PPT>(table, nq, lg, (int)blockIdx.x);
      early = p.block_table[(size_t)table.group[x.group].first * p.max_pages +
                            min(x.page0 + lane, table.group[x.group].pages - 1)];
    }
    for (int k = 0; ok && take(k, job); ++k) {
      give_back(k);
      // Pages, 32 at a time, a page per lane, the next 32 on their way; entries behind the job's
      // end repeat its last page (its tokens are hidden there).
      const int pages = (job.end + P - 1) / P - job.page0;
      auto entry = [&](int i) {
        return p.block_table[(size_t)job.seq * p.max_pages + job.page0 + min(i, pages - 1)];
      };
      auto checked = [&](int phys, int i) {
        if (phys >= 0 && phys < p.num_phys) return phys;
        if (i < pages) record_at<kSitePrefix>(p, QUEST_ERR_BAD_PAGE, job.seq, job.page0 + i);
        return 0;
      };
      int now = 0, next = 0;
      if (job.n > 0) {
        now = checked(k == 0 && job.shared ? early : entry(lane), lane);
        if (pages > 32) next = entry(32 + lane);
      }
      for (int i = 0; i < job.n; ++i) {
        // (a test of the waits: the last V tile of a job never comes)
        if (kv && i == job.n - 1 && (p.debug_flags & QUEST_DEBUG_WITHHOLD_VALUES)) {
          ok = false;
          break;
        }
        const int at = i * PPT & 31;
        if (at == 0 && i > 0) {
          now = checked(next, i * PPT + lane);
          next = entry(i * PPT + 32 + lane);
        }
        if (total >= kSlots && !(ok = idle(&bars.free[slot][kv], ph))) break;
        const bool leader = elect_lane();
        if (leader) mbar_arrive_expect_tx(&bars.full[slot][kv], kTile);
#pragma unroll
        for (int e = 0; e < PPT; ++e) {
          const int phys = __shfl_sync(0xffffffffu, now, at + e);
          if (leader)
            tma_page(smem + Smem::kv + (2 * slot + kv) * kTile + e * P * kHeadDim * 2,
                     kv ? &map_v : &map_k, (phys * p.Hkv + job.g) * (P / 8), &bars.full[slot][kv]);
        }
        __syncwarp();
        ++total;
        if (++slot == kSlots) {
          slot = 0;
          ph ^= 1u;
        }
      }
      if (kv == 0 && lane == 0) mbar_arrive(&bars.want);
    }
    if (lane == 0) bars.fetched[kv] = total;
  } else if (warp == 10) {
    // ---- issue
    const uint64_t q_desc = smem_desc(smem_u32(smem + Smem::q), 16, kAtomBytes);
    const uint64_t k_desc = smem_desc(smem_u32(smem + Smem::kv), 16, kGroupBytes);
    const uint64_t v_desc = smem_desc(smem_u32(smem + Smem::kv + kTile), kAtomBytes, kGroupBytes);
    constexpr uint32_t kSlotStep = 2 * kTile >> 4;
    int ks = 0, vs = 0;  // slots of the next K and of the next V tile
    uint32_t kph = 0, vph = 0;
    // Q K^T of the next K tile into a buffer (whose weights P V has been given before); `last` of
    // its job.
    auto qk = [&](int buffer, bool last) {
      if (!wait(&bars.full[ks][0], kph)) return false;
      fence_after();
      if (elect_lane()) {
#pragma unroll
        for (int k = 0; k < kHeadDim / 16; ++k) {
          const uint32_t oq = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
          const uint32_t ok = ((k >> 2) * kAtomBytes + (k & 3) * 32) >> 4;
          mma_ss(tmem + buffer * kTokens, q_desc + oq, k_desc + ks * kSlotStep + ok, kIdescQK, k > 0);
        }
        commit(&bars.s_full[buffer]);
        commit(&bars.free[ks][0]);
        if (last) commit(&bars.q_free);
      }
      __syncwarp();
      if (++ks == kSlots) {
        ks = 0;
        kph ^= 1u;
      }
      return true;
    };
    Job job;
    int t = 0, done = 0;  // tiles and jobs (with tiles) before this one
    bool ok = true;
    for (int k = 0; ok && take(k, job); ++k) {
      give_back(k);
      if (job.n == 0) continue;
      ok = wait(&bars.q_full, (uint32_t)done & 1) && qk(t & 1, job.n == 1);
      for (int i = 0; ok && i < job.n; ++i, ++t) {
        if (i + 1 < job.n && !(ok = qk((t + 1) & 1, i + 2 == job.n))) break;
        if (!(ok = wait(&bars.full[vs][1], vph))) break;
        // values that no row of the job sees may be anything: 0 * NaN is not 0
        const int behind = job.end - job.page0 * P - i * kTokens;
        if (behind < kTokens) {
          for (int c = behind + lane; c < kTokens; c += 32)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              *reinterpret_cast<uint4*>(smem + Smem::kv + (2 * vs + 1) * kTile +
                                        (c >> 3) * kGroupBytes + (e >> 3) * kAtomBytes +
                                        (c & 7) * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!(ok = idle(&bars.p_full[t & 1], (uint32_t)(t >> 1) & 1))) break;
        if (i == 0 && done > 0 && !(ok = idle(&bars.o_free, (uint32_t)(done - 1) & 1))) break;
        fence_after();
        if (elect_lane()) {
#pragma unroll
          for (int k = 0; k < kTokens / 16; ++k)  // the first half's four, then the other's
            mma_ts(tmem + 256 + (k >> 2) * kHeadDim,
                   tmem + (t & 1) * kTokens + (k >> 2) * 64 + 8 * (k & 3),
                   v_desc + (uint32_t)(vs * kSlotStep + k * (2 * kGroupBytes >> 4)), kIdescPV,
                   i > 0 || (k & 3) > 0);
          commit(&bars.free[vs][1]);
          commit(&bars.pv_done);
          if (i + 1 == job.n) commit(&bars.o_full);
        }
        __syncwarp();
        if (++vs == kSlots) {
          vs = 0;
          vph ^= 1u;
        }
      }
      ++done;
    }
  } else {
    // ---- softmax: a thread a row's 64 tokens
    const int half = warp >> 2, row = threadIdx.x & 127, G = 1 << lg;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lanes + 64 * half, o_col = tmem + lanes + 256 + 128 * half;
    float2* stash = reinterpret_cast<float2*>(smem + Smem::stash);  // [half][row]
    Job job;
    int t = 0, done = 0;
    uint32_t pairs = 0;
    bool ok = true;
    for (int k = 0; ok && take(k, job); ++k) {
      const bool mine = row < job.rows;
      const bool some = (row & ~31) < job.rows;  // (the warp's)
      const int pos0 = job.page0 * P;
      // the last position that the row sees; the least of the warp's rows, which go together
      int pr = job.end - 1;
      if (job.ragged && mine) {
        const int tok = job.q_tok + (row >> lg);
        pr = min(pr, length(tok / nq) - nq + tok % nq);
      }
      const int least = __reduce_min_sync(0xffffffffu, pr);
      float m = -CUDART_INF_F, l = 0.f;
      for (int i = 0; i < job.n; ++i, ++t) {
        if (!(ok = idle(&bars.s_full[t & 1], (uint32_t)(t >> 1) & 1))) break;
        if (some) {  // (without a query in the warp's rows their weights may be anything)
          fence_after();
          const uint32_t s_now = s_col + (t & 1) * kTokens;
          float s[64];
          tmem_ld32(s_now, reinterpret_cast<uint32_t*>(s));
          tmem_ld32(s_now + 32, reinterpret_cast<uint32_t*>(s) + 32);
          tmem_wait_ld();
          const int base = pos0 + i * kTokens + 64 * half;
          if (base + 63 > least) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (base + e > pr) s[e] = -CUDART_INF_F;
          }
          float best[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int e = 0; e < 64; e += 4)
#pragma unroll
            for (int u = 0; u < 2; ++u) best[u] = max3(best[u], s[e + u], s[e + 2 + u]);
          const float top = fmaxf(best[0], best[1]) * p.qscale;
          // The reference moves only when a row exceeds it by 2^kLazy; the warp's rows move theirs
          // together, l and O with them.  Lanes without a query have no say: of a tail only its own
          // rows were fetched, the others hold what the CTA's last job left there, which the order
          // that the jobs were taken in decides.
          if (__any_sync(0xffffffffu, mine && top > m + kLazy)) {
            const float mn = fmaxf(m, top);
            const float f = mn == -CUDART_INF_F ? 1.f : ex2(m - mn);
            m = mn;
            l *= f;
            if (i > 0) {
              // (a product that the slowest warp's weights hold up: it may be taking rows again)
              if (!(ok = idle(&bars.pv_done, (uint32_t)(t - 1) & 1))) break;
              fence_after();
#pragma unroll 1
              for (int u = 0; u < 8; ++u) {
                uint32_t o[16];
                tmem_ld16(o_col + 16 * u, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(o_col + 16 * u, o);
              }
            }
          }
          uint32_t w[32];
          uint64_t sum[2] = {0, 0};
          const float shift = kBias - (m == -CUDART_INF_F ? 0.f : m);
          const uint64_t shift2 = pair(shift, shift), scale2 = pair(p.qscale, p.qscale);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float a, c;
            unpair(fma2(pair(s[2 * e], s[2 * e + 1]), scale2, shift2), a, c);
            a = ex2(a);
            c = ex2(c);
            sum[e & 1] = add2(sum[e & 1], pair(a, c));
            w[e] = pack2(a, c);
          }
          tmem_st32(s_now, w);
          float a, c;
          unpair(add2(sum[0], sum[1]), a, c);
          l += a + c;
          tmem_wait_st();
          fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[t & 1]);
      }
      if (!ok) break;
      // ---- the rows' shares: warps 0-3 the dims 0-63, warps 4-7 the others
      const int dim0 = 64 * half;
      float M = -CUDART_INF_F, Z = 0.f, f0 = 0.f, f1 = 0.f;
      if (job.n > 0) {
        if (!(ok = idle(&bars.o_full, (uint32_t)done & 1))) break;
        ++done;
        fence_after();
        if (some) {
          // a row's halves are in warps w and w + 4
          stash[half * kRows + row] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.pair[warp & 3]);
          if (!(ok = idle(&bars.pair[warp & 3], pairs & 1))) break;
          ++pairs;
          const float2 other = stash[(half ^ 1) * kRows + row];
          M = fmaxf(m, other.x);
          const float fm = half_factor(m, l, M), fo = half_factor(other.x, other.y, M);
          Z = fmaf(l, fm, other.y * fo);
          f0 = half ? fo : fm;
          f1 = half ? fm : fo;
        }
      }
      const bool none = Z == 0.f;  // (a NaN sum is not: its NaN goes out)
      bool odd = false;            // some of the row's O is not finite
      const size_t slot = (size_t)job.share + row;
      if (some) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t o[32], x[32];
          tmem_ld32(tmem + lanes + 256 + dim0 + 32 * u, o);  // (without a tile anything: not used)
          tmem_ld32(tmem + lanes + 384 + dim0 + 32 * u, x);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            o[e] = __float_as_uint(fmaf(__uint_as_float(x[e]), f1, __uint_as_float(o[e]) * f0));
            odd |= (o[e] & 0x7f800000u) == 0x7f800000u;
            if (none) o[e] = 0u;  // (it may be 0 * NaN)
          }
          if (mine) {  // whole sectors: a lane's row is 512 B from its neighbour's
#pragma unroll
            for (int e = 0; e < 4; ++e)
              store8(p.part_acc + slot * kHeadDim + dim0 + 32 * u + 8 * e, o + 8 * e);
          }
          __syncwarp();
        }
        if (mine && half == 0) {
          p.part_ml[2 * slot] = M;
          p.part_ml[2 * slot + 1] = Z;
        }
      }
      fence_before();
      __syncwarp();
      if (job.n > 0 && lane == 0) mbar_arrive(&bars.o_free);
      // An infinity or NaN among the values of a tile reaches all of its rows, as 0 * NaN, those too
      // that do not see its token.  Such a row (its scores are finite, its O is not) is taken again
      // from what it sees, by its warp, a token at a time.
      unsigned todo = __ballot_sync(0xffffffffu, mine && odd && !none && Z <= FLT_MAX);
      while (todo) {  // (the warp's)
        const int from = __ffs(todo) - 1, r = (row & ~31) + from;
        todo &= todo - 1u;
        const float m_r = __shfl_sync(0xffffffffu, M, from);
        const int last = __shfl_sync(0xffffffffu, pr, from) + 1;
        const int tok = job.q_tok + (r >> lg);
        const uint2 qw = *reinterpret_cast<const uint2*>(
            p.q + ((size_t)tok * p.Hq + ((size_t)job.g << lg) + (r & (G - 1))) * kHeadDim + 4 * lane);
        const float2 qa = h2f(qw.x), qb = h2f(qw.y);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int page = job.page0; page * P < last; ++page) {
          if (lane == 0) atomicAdd(&bars.moves, 1u);
          const int phys = p.block_table[(size_t)job.seq * p.max_pages + page];
          if (phys < 0 || phys >= p.num_phys) continue;
          const size_t at = ((size_t)phys * p.Hkv + job.g) * P * kHeadDim + 4 * lane;
#pragma unroll 4
          for (int e = 0; e < min(P, last - page * P); ++e) {
            const uint2 kw = *reinterpret_cast<const uint2*>(p.k_pool + at + e * kHeadDim);
            const uint2 vw = *reinterpret_cast<const uint2*>(p.v_pool + at + e * kHeadDim);
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
        if (lane >> 4 == half)  // (the other half's warp does its dims)
          *reinterpret_cast<float4*>(p.part_acc + ((size_t)job.share + r) * kHeadDim + 4 * lane) =
              make_float4(acc[0], acc[1], acc[2], acc[3]);
      }
      give_back(k);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (*give_up) {  // (nobody sets it any more)
    // A wait ran out: copies and products in flight end before their memory goes.  (Otherwise the
    // results were waited for, and with them everything that went into them.)
    if (warp == 10) {
      if (elect_lane()) commit(&bars.drain);  // the products that this thread issued
      __syncwarp();
      settle(&bars.drain, 0);
    } else if ((warp == 8 || warp == 9) && lane < kSlots) {
      // copies into slot `lane`: its phases so far
      const int phases = (bars.fetched[warp - 8] + kSlots - 1 - lane) / kSlots;
      if (phases > 0) settle(&bars.full[lane][warp - 8], (uint32_t)(phases - 1) & 1);
    } else if (warp == 12 && lane == 0 && bars.q_fetched > 0) {
      settle(&bars.q_full, (uint32_t)(bars.q_fetched - 1) & 1);
    }
    __syncthreads();
  }
  if (warp == 10) tmem_free(tmem);
}

// The shares of a prefix and of a tail into out and lse: a block of one warp a row (query token, query
// head), lane l the dims 4 l .. 4 l + 3.  Such blocks wait beside the jobs' CTA, seven an SM: 0.9 us
// less than blocks of four, of which one fits (40.4 and 41.4 us at 32 tails behind 32K).  First come
// the prefix's splits (of the row's work item, part_rows rows apart), then the tail's (of the row's kv
// head, a job's rows apart).
__global__ void __launch_bounds__(32) prefix_join_kernel(
    const __grid_constant__ PrefixParams pp, const __grid_constant__ PrefixTable t) {
  const Params& p = pp.p;
  const int lane = threadIdx.x, G = p.Hq / p.Hkv, at = (int)blockIdx.x;
  const int h = at % p.Hq, tok = at / p.Hq, b = tok / pp.n, g = h / G;
  const PrefixTable::Group& q = t.group[t.group_of_seq(b)];
  const int shared = q.pages > 0 ? q.splits : 0;
  size_t slot0 = 0, step = 0;  // of the prefix's
  if (shared) {
    const int rows = q.count * pp.n * G, part_rows = min(rows, kPrefixRows);
    const int blocks = (rows + kPrefixRows - 1) / kPrefixRows;
    const int r = (tok - q.first * pp.n) * G + h % G;
    slot0 = q.part0 + ((size_t)g * shared * blocks + r / kPrefixRows) * part_rows + r % kPrefixRows;
    step = (size_t)blocks * part_rows;
  }
  const int tail_rows = pp.n * G;
  const size_t tail0 =
      t.parts + ((size_t)b * p.Hkv + g) * pp.splits * tail_rows + tok % pp.n * G + h % G;
  auto slot = [&](int s) {
    return s < shared ? slot0 + s * step : tail0 + (size_t)(s - shared) * tail_rows;
  };
  pdl_wait();
  pdl_trigger();
  if (at == 0 && lane == 0) *p.exited = 0u;  // the queue, for the next call
  const int L = __ldcg(p.seq_lens + b);
  const bool known = L >= 0 && (long long)L <= (long long)p.max_pages * p.P;
  constexpr int kOf = 2 * kPrefixSplits / 32;  // shares of a lane
  constexpr int kTogether = 8;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  auto load = [&](int s) {
    return __ldcg(reinterpret_cast<const float4*>(p.part_acc + slot(s) * kHeadDim) + lane);
  };
  auto load_ml = [&](int s) { return __ldcg(reinterpret_cast<const float2*>(p.part_ml) + slot(s)); };
  // The prefix's shares and the tail's first, which every row has, are on their way beside the
  // length, which says how many more the tail has.
  float2 ml[kOf];
#pragma unroll
  for (int e = 0; e < kOf; ++e)
    ml[e] = lane + 32 * e <= shared ? load_ml(lane + 32 * e) : make_float2(-CUDART_INF_F, 0.f);
  float4 a[kTogether];
#pragma unroll
  for (int i = 0; i < kTogether; ++i) a[i] = i <= shared ? load(i) : zero;
  const int n = shared + tail_of(pp, q.pages, known ? L : 0).jobs;
  auto share = [&](int s) { return s < n ? load(s) : zero; };
  if (n > shared + 1) {
#pragma unroll
    for (int e = 0; e < kOf; ++e)
      if (lane + 32 * e > shared && lane + 32 * e < n) ml[e] = load_ml(lane + 32 * e);
#pragma unroll
    for (int i = 0; i < kTogether; ++i)
      if (i > shared) a[i] = share(i);
  }
  float f[kOf], Z = 0.f, M = -CUDART_INF_F;
#pragma unroll
  for (int e = 0; e < kOf; ++e) M = fmaxf(M, ml[e].x);
  M = warp_max(M);
#pragma unroll
  for (int e = 0; e < kOf; ++e) {
    f[e] = half_factor(ml[e].x, ml[e].y, M);
    Z = fmaf(ml[e].y, f[e], Z);
  }
  Z = warp_sum(Z);
  float4 A = zero;
#pragma unroll
  for (int e = 0; e < kOf; ++e) {  // (share s has its factor in lane s % 32's f[s / 32])
#pragma unroll 1
    for (int s0 = 32 * e; s0 < min(n, 32 * e + 32); s0 += kTogether) {
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        const float w = __shfl_sync(0xffffffffu, f[e], (s0 + i) & 31);
        A.x = fmaf(a[i].x, w, A.x);
        A.y = fmaf(a[i].y, w, A.y);
        A.z = fmaf(a[i].z, w, A.z);
        A.w = fmaf(a[i].w, w, A.w);
        a[i] = share(s0 + kTogether + i);
      }
    }
  }
  const bool none = Z == 0.f;
  const float inv = none ? 0.f : 1.f / Z;
  reinterpret_cast<uint2*>(p.out + (size_t)at * kHeadDim)[lane] =
      none ? make_uint2(0u, 0u)
           : make_uint2(pack2(A.x * inv, A.y * inv), pack2(A.z * inv, A.w * inv));
  if (lane == 0 && p.lse)
    p.lse[at] = none ? -CUDART_INF_F : (M - kBias + log2f(Z)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_prefix(const Params& p, const PrefixTable& t, int n_tokens, int splits,
                          int piece_pages, cudaStream_t s) {
  PrefixParams pp{};
  pp.p = p;
  const int G = p.Hq / p.Hkv;
  pp.log_g = G == 8 ? 3 : G / 2;
  pp.n = n_tokens;
  pp.splits = splits;
  pp.piece_pages = piece_pages;
  CUtensorMap mq, m1, mk, mv;
  const cuuint64_t qd[3] = {kHeadDim, (cuuint64_t)p.Hq, (cuuint64_t)p.B * n_tokens};
  const cuuint64_t qs[2] = {kHeadDim * 2, (cuuint64_t)p.Hq * kHeadDim * 2};
  const cuuint32_t qb[3] = {64, (cuuint32_t)G, (cuuint32_t)(kRows / G)};
  const cuuint32_t q1[3] = {64, (cuuint32_t)G, (cuuint32_t)n_tokens};
  cudaError_t e = make_map(&mq, p.q, 3, qd, qs, qb);
  if (e != cudaSuccess) return e;
  if ((e = make_map(&m1, p.q, 3, qd, qs, q1)) != cudaSuccess) return e;
  // a pool as [8-row group][half of the dims][row][64 dims]
  const cuuint64_t kd[4] = {64, 8, 2, (cuuint64_t)p.num_phys * p.Hkv * (p.P / 8)};
  const cuuint64_t ks[3] = {kHeadDim * 2, kHeadDim, 8 * kHeadDim * 2};
  const cuuint32_t kb[4] = {64, 8, 2, (cuuint32_t)(p.P / 8)};
  if ((e = make_map(&mk, p.k_pool, 4, kd, ks, kb)) != cudaSuccess) return e;
  if ((e = make_map(&mv, p.v_pool, 4, kd, ks, kb)) != cudaSuccess) return e;
  const void* fn = p.P == 16 ? (const void*)prefix_kernel<16> : (const void*)prefix_kernel<32>;
  if ((e = ensure_smem(fn, Smem::total)) != cudaSuccess) return e;
  void* args[] = {&pp, const_cast<PrefixTable*>(&t), &mq, &m1, &mk, &mv};
  const long long jobs = t.ctas + (long long)p.B * p.Hkv * splits;  // at most
  e = launch_pdl(fn, dim3((unsigned)std::min<long long>(jobs, kPrefixSms)), dim3(kPrefixThreads),
                 Smem::total, s, args);
  if (e != cudaSuccess) return e;
  void* join_args[] = {&pp, const_cast<PrefixTable*>(&t)};
  const long long rows = (long long)p.B * n_tokens * p.Hq;
  return launch_pdl((const void*)prefix_join_kernel, dim3((unsigned)rows), dim3(32), 0, s, join_args);
}

}  // namespace quest
