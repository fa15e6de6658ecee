// quest_prefix_kernel.cu - attention of a group's query tokens over the prefix that their
// sequences share, on the fifth-generation tensor cores (tcgen05, accumulators in TMEM, operands
// by TMA).
//
// A row is (sequence of the group, query head of a kv head's group); a CTA takes 128 rows and a
// run of the prefix's tokens, 128 to a K / V tile, so that a tile is read once for up to 128 rows:
//   S = Q K^T,   P = 2^(S c - m + 8),   O += P V
// with a running maximum m and sum of weights per row.  There is no causal mask (queries come
// after the prefix); a row ends with its own sequence where that is shorter.  What leaves is a
// share (m, sum, O) per row, which prefix_join_kernel joins with the other shares and the tail's.
//
// Eight softmax warps share a tile: warps 0-3 its first 64 tokens, warps 4-7 the other 64, a thread
// a row of 64 scores in registers.  Either half has a maximum, a sum and an O of its own (two O in
// TMEM), so that the halves never wait for one another; they are added at the end, in registers.
// Scores have two buffers in TMEM: Q K^T of tile j + 1 runs while tile j is in its softmax, P V
// while tile j + 1 is.  Warps 8 and 9 fetch K and V (a page a TMA box, three tiles of each in
// flight), warp 10 issues the products.
#include <math_constants.h>

#include <algorithm>
#include <cfloat>

#include "quest_device.cuh"
#include "quest_tc.cuh"

namespace quest {

namespace {

constexpr int kPrefixThreads = 352;
constexpr int kRows = kPrefixRows, kTokens = kPrefixTokens;
constexpr int kTile = kTokens * kHeadDim * 2;  // 32 KiB
constexpr int kHalf = kTile / 2;  // 64 dims of every row: one 128-byte swizzle span
constexpr int kSlots = 3;         // K tiles, and V tiles, in flight
constexpr float kBias = 8.f;      // as the tail's: shares of both are joined
constexpr float kLazy = 6.f;      // the maximum moves when a row exceeds it by 2^6

// The queries, then K and V of each slot side by side.
struct Smem {
  static constexpr int q = 0;
  static constexpr int kv = kTile;  // [kSlots][K, V]
  static constexpr int bars = kv + 2 * kSlots * kTile;
  static constexpr int total = bars + 256;
};
static_assert(Smem::total + 1024 <= (int)kMaxSmem, "shared memory of a CTA");

// Operands as in the prompt kernel: Q as the atoms of dims 0-63 of all rows, then those of dims
// 64-127; K and V per 8 tokens the atoms of both halves side by side, so that a page is one box.
constexpr int kAtomBytes = 1024, kGroupBytes = 2 * kAtomBytes;
// fp16 x fp16 -> fp32, 128 x 128 x 16; bit 16: B is MN-major.
constexpr uint32_t kIdescQK = 1u << 4 | (kTokens >> 3) << 17 | (kRows >> 4) << 24;
constexpr uint32_t kIdescPV = 1u << 4 | 1u << 16 | (kHeadDim >> 3) << 17 | (kRows >> 4) << 24;

struct Bars {
  uint64_t q_full;
  uint64_t full[kSlots][2], free[kSlots][2];  // of a slot's K and V: fetched; read by its product
  // Scores and weights of a buffer: tile i (from the CTA's first) is in buffer i % 2.  Nobody is
  // late by a phase: Q K^T of tile i + 2 is issued after the weights of tile i have been waited for,
  // which every softmax warp gave after it had seen the scores of tile i.
  uint64_t s_full[2], p_full[2];
  // P V of a tile is done.  Who asks for tile i - 1 has seen the scores of tile i, whose barrier
  // also says that P V of tile i - 2 is done.
  uint64_t pv_done, o_full, drain;
  uint32_t tmem;
  int give_up;
  int fetched[2];  // K and V tiles whose copies have been issued
};
static_assert(sizeof(Bars) <= 256, "barrier area");

// A CTA's work: a row block of a kv head, and a split's tiles.
struct Item {
  int blk, split, n_splits, g, first, count, pages;
};

// Of a group's CTAs the row blocks vary fastest (the CTAs that read the same tiles run side by
// side), then the splits, then the kv heads; *share: where the item's shares start.
__device__ __forceinline__ Item item_of(const PrefixTable& t, int log_g, size_t* share) {
  const int c = (int)blockIdx.x;
  const PrefixTable::Group& q = t.group[t.group_of_cta(c)];
  const int rows = q.count << log_g;
  const int blocks = (rows + kRows - 1) / kRows, at = c - q.cta0;
  if (share) *share = (size_t)q.part0 + (size_t)at * min(rows, kRows);
  return Item{at % blocks, at / blocks % q.splits, q.splits, at / blocks / q.splits,
              q.first, q.count, q.pages};
}

// What brings a half's part of a softmax to the maximum M of both (as part_factor of the span
// decode: a part without a weight is 0, one of NaN scores goes on, an infinite O stays one).
__device__ __forceinline__ float half_factor(float m, float l, float M) {
  return m == -CUDART_INF_F ? (l == 0.f ? 0.f : 1.f) : fmaxf(ex2(m - M), FLT_MIN);
}

template <int P>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ Params p, const __grid_constant__ PrefixTable table,
                  int log_g, const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ unsigned char smem_raw[];
  constexpr int PPT = kTokens / P;  // pages of a tile
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Bars& bars = *reinterpret_cast<Bars*>(smem + Smem::bars);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);  // (uniform to the compiler)
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars.q_full, 1);
    for (int i = 0; i < kSlots; ++i)
      for (int kv = 0; kv < 2; ++kv) {
        mbar_init(&bars.full[i][kv], 1);
        mbar_init(&bars.free[i][kv], 1);
      }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.p_full[t], 8);
    }
    mbar_init(&bars.pv_done, 1);
    mbar_init(&bars.o_full, 1);
    mbar_init(&bars.drain, 1);
    bars.give_up = bars.fetched[0] = bars.fetched[1] = 0;
    fence_mbar_init();
  }
  if (warp == 10) tmem_alloc(&bars.tmem);
  if (warp == 8 && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v)
                 : "memory");
  const int lg = log_g, G = 1 << lg;
  const Item it = item_of(table, lg, nullptr);
  const int tok0 = it.blk * (kRows >> lg), tok1 = min(it.count, tok0 + (kRows >> lg));
  const int tiles = (it.pages + PPT - 1) / PPT;
  const int j0 = tiles * it.split / it.n_splits;
  int j1 = tiles * (it.split + 1) / it.n_splits;
  pdl_wait();
  pdl_trigger();  // the tails' launch, which waits for this one only at its end

  // Pages for the fetch warps: 32 at a time, a page per lane, the next 32 on their way (the first
  // ones beside the lengths); entries behind the prefix's end repeat its last page (its tokens are
  // hidden there).
  auto entry = [&](int i) {
    return p.block_table[(size_t)it.first * p.max_pages + min(i, it.pages - 1)];
  };
  int now = 0, next = 0;
  if (warp == 8 || warp == 9) {
    now = entry(j0 * PPT + lane);
    next = entry(j0 * PPT + 32 + lane);
  }
  auto length = [&](int seq) {
    const int L = p.seq_lens[seq];
    if (L >= 0 && (long long)L <= (long long)p.max_pages * P) return L;
    record_at<kSitePrefix>(p, QUEST_ERR_BAD_LENGTH, seq, -1);
    return 0;
  };
  int most = 0;
  for (int i = tok0 + lane; i < tok1; i += 32) most = max(most, length(it.first + i));
  // the end of what some row sees
  const int end = min(__reduce_max_sync(0xffffffffu, most), it.pages * P);
  j1 = max(j0, min(j1, (end + kTokens - 1) / kTokens));
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&bars.tmem);
  volatile int* give_up = &bars.give_up;

  const int n = j1 - j0;  // the CTA's tiles

  // A row's places for maxima and sums (of its halves, of a row that is taken again), in the
  // queries' space once the last product is done.
  auto stash = [&](int t, int row) {
    return reinterpret_cast<float2*>(smem + Smem::q) + t * kRows + row;
  };
  bool again = false;
  bool ok = true;
  float m = -CUDART_INF_F, l = 0.f;  // of a softmax thread's half
  const int half = warp >> 2, row = threadIdx.x & 127;
  const bool mine = warp < 8 && tok0 + (row >> lg) < tok1;
  const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
  if (warp >= 8) {
    if (warp < 10) {
      // ---- fetch: warp 8 the queries and K tiles, warp 9 the V tiles
      const int kv = warp == 9;
      if (!kv && elect_lane()) {
        mbar_arrive_expect_tx(&bars.q_full, kTile);
        for (int i = 0; i < 2; ++i)
          tma_3d(smem + Smem::q + i * kHalf, &map_q, 64 * i, it.g * G, it.first + tok0, &bars.q_full);
      }
      __syncwarp();
      auto checked = [&](int phys, int i) {
        if (phys >= 0 && phys < p.num_phys) return phys;
        if (i < it.pages) record_at<kSitePrefix>(p, QUEST_ERR_BAD_PAGE, it.first, i);
        return 0;
      };
      now = checked(now, j0 * PPT + lane);
      int slot = 0;
      uint32_t ph = 1;  // (of the phase before a slot's first: over)
      int j = j0;
      for (; j < j1; ++j) {
        // (a test of the waits: the last V tile of a work item never comes)
        if (kv && j == j1 - 1 && (p.debug_flags & QUEST_DEBUG_WITHHOLD_VALUES)) break;
        const int at = (j - j0) * PPT & 31;
        if (at == 0 && j > j0) {
          now = checked(next, j * PPT + lane);
          next = entry(j * PPT + 32 + lane);
        }
        if (j - j0 >= kSlots &&
            !__all_sync(0xffffffffu, wait_at<kSitePrefix>(p, &bars.free[slot][kv], ph, give_up)))
          break;
        const bool leader = elect_lane();
        if (leader) mbar_arrive_expect_tx(&bars.full[slot][kv], kTile);
#pragma unroll
        for (int e = 0; e < PPT; ++e) {
          const int phys = __shfl_sync(0xffffffffu, now, at + e);
          if (leader)
            tma_page(smem + Smem::kv + (2 * slot + kv) * kTile + e * P * kHeadDim * 2,
                     kv ? &map_v : &map_k, (phys * p.Hkv + it.g) * (P / 8), &bars.full[slot][kv]);
        }
        __syncwarp();
        if (++slot == kSlots) {
          slot = 0;
          ph ^= 1u;
        }
      }
      if (lane == 0) bars.fetched[kv] = j - j0;
    } else {
      // ---- issue
      const uint64_t q_desc = smem_desc(smem_u32(smem + Smem::q), 16, kAtomBytes);
      const uint64_t k_desc = smem_desc(smem_u32(smem + Smem::kv), 16, kGroupBytes);
      const uint64_t v_desc = smem_desc(smem_u32(smem + Smem::kv + kTile), kAtomBytes, kGroupBytes);
      constexpr uint32_t kSlotStep = 2 * kTile >> 4;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_at<kSitePrefix>(p, bar, parity, give_up)) != 0;
      };
      auto qk = [&](int buffer, int slot) {
        if (elect_lane()) {
#pragma unroll
          for (int k = 0; k < kHeadDim / 16; ++k) {
            const uint32_t oq = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
            const uint32_t ok = ((k >> 2) * kAtomBytes + (k & 3) * 32) >> 4;
            mma_ss(tmem + buffer * kTokens, q_desc + oq, k_desc + slot * kSlotStep + ok, kIdescQK,
                   k > 0);
          }
          commit(&bars.s_full[buffer]);
          commit(&bars.free[slot][0]);
        }
        __syncwarp();
      };
      int ks = 1, vs = 0;  // slots of the next K and of the V tile
      uint32_t kph = 0, vph = 0;
      ok = n > 0 && wait(&bars.q_full, 0) && wait(&bars.full[0][0], 0);
      if (ok) {
        fence_after();
        qk(0, 0);
      }
      for (int i = 0; ok && i < n; ++i) {
        if (i + 1 < n) {  // (its buffer held the weights of tile i - 1, which P V has been given)
          if (!(ok = wait(&bars.full[ks][0], kph))) break;
          fence_after();
          qk((i + 1) & 1, ks);
          if (++ks == kSlots) {
            ks = 0;
            kph ^= 1u;
          }
        }
        if (!(ok = wait(&bars.full[vs][1], vph))) break;
        // values that no row of the CTA sees may be anything: 0 * NaN is not 0
        const int behind = end - (j0 + i) * kTokens;
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
        if (!(ok = wait(&bars.p_full[i & 1], (uint32_t)(i >> 1) & 1))) break;
        fence_after();
        if (elect_lane()) {
#pragma unroll
          for (int k = 0; k < kTokens / 16; ++k)  // the first half's four, then the other's
            mma_ts(tmem + 256 + (k >> 2) * kHeadDim,
                   tmem + (i & 1) * kTokens + (k >> 2) * 64 + 8 * (k & 3),
                   v_desc + (uint32_t)(vs * kSlotStep + k * (2 * kGroupBytes >> 4)), kIdescPV,
                   i > 0 || (k & 3) > 0);
          commit(&bars.free[vs][1]);
          commit(i + 1 < n ? &bars.pv_done : &bars.o_full);
        }
        __syncwarp();
        if (++vs == kSlots) {
          vs = 0;
          vph ^= 1u;
        }
      }
    }
  } else {
    // ---- softmax: a thread a row's 64 tokens
    // the last position that the row sees; the least of the warp's rows, which go together
    const int pr = mine ? min(length(it.first + tok0 + (row >> lg)), end) - 1 : end - 1;
    const int least = __reduce_min_sync(0xffffffffu, pr);
    const bool some = __any_sync(0xffffffffu, mine);
    const uint32_t s_col = tmem + lanes + 64 * half, o_col = tmem + lanes + 256 + 128 * half;
    for (int i = 0; i < n; ++i) {
      const uint32_t phase = (uint32_t)(i >> 1) & 1;
      ok = __all_sync(0xffffffffu, wait_at<kSitePrefix>(p, &bars.s_full[i & 1], phase, give_up));
      if (!ok) break;
      if (some) {  // (without a query in the warp's rows their weights may be anything)
        fence_after();
        const uint32_t s_now = s_col + (i & 1) * kTokens;
        float s[64];
        tmem_ld32(s_now, reinterpret_cast<uint32_t*>(s));
        tmem_ld32(s_now + 32, reinterpret_cast<uint32_t*>(s) + 32);
        tmem_wait_ld();
        const int base = (j0 + i) * kTokens + 64 * half;
        if (base + 63 > least) {
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (base + k > pr) s[k] = -CUDART_INF_F;
        }
        float best[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int k = 0; k < 64; k += 4)
#pragma unroll
          for (int e = 0; e < 2; ++e) best[e] = max3(best[e], s[k + e], s[k + 2 + e]);
        const float top = fmaxf(best[0], best[1]) * p.qscale;
        if (__any_sync(0xffffffffu, top > m + kLazy)) {
          const float mn = fmaxf(m, top);
          const float f = mn == -CUDART_INF_F ? 1.f : ex2(m - mn);
          m = mn;
          l *= f;
          if (i > 0) {
            ok = __all_sync(0xffffffffu, wait_at<kSitePrefix>(p, &bars.pv_done, (uint32_t)(i - 1) & 1,
                                                              give_up));
            if (!ok) break;
            fence_after();
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
        }
        uint32_t w[32];
        uint64_t sum[2] = {0, 0};
        const float shift = kBias - (m == -CUDART_INF_F ? 0.f : m);
        const uint64_t shift2 = pair(shift, shift), scale2 = pair(p.qscale, p.qscale);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float a, c;
          unpair(fma2(pair(s[2 * k], s[2 * k + 1]), scale2, shift2), a, c);
          a = ex2(a);
          c = ex2(c);
          sum[k & 1] = add2(sum[k & 1], pair(a, c));
          w[k] = pack2(a, c);
        }
        tmem_st32(s_now, w);
        float a, c;
        unpair(add2(sum[0], sum[1]), a, c);
        l += a + c;
        tmem_wait_st();
        fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full[i & 1]);
    }
    // the last product, and with it all (where none ran, the queries have landed)
    if (ok)
      ok = __all_sync(0xffffffffu, wait_at<kSitePrefix>(p, n > 0 ? &bars.o_full : &bars.q_full, 0,
                                                        give_up));
    if (ok) *stash(half, row) = make_float2(m, l);
  }
  __syncthreads();
  fence_after();
  if (warp < 8 && __all_sync(0xffffffffu, ok && *give_up == 0)) {
    // ---- the row's share: warps 0-3 the dims 0-63 of it, warps 4-7 the others
    const float2 other = *stash(half ^ 1, row);
    const float M = fmaxf(m, other.x);
    const float f_mine = half_factor(m, l, M), f_other = half_factor(other.x, other.y, M);
    const float Z = fmaf(l, f_mine, other.y * f_other);
    const float f0 = half ? f_other : f_mine, f1 = half ? f_mine : f_other;
    const bool none = Z == 0.f;  // (a NaN sum is not: its NaN goes out)
    bool odd = false;            // some of the row's O is not finite
    size_t slot;
    item_of(table, lg, &slot);
    slot += row;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t o[32], x[32];
      const int dim = 64 * half + 32 * u;
      tmem_ld32(tmem + lanes + 256 + dim, o);  // (without a tile anything: it is not used)
      tmem_ld32(tmem + lanes + 384 + dim, x);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        o[k] = __float_as_uint(fmaf(__uint_as_float(x[k]), f1, __uint_as_float(o[k]) * f0));
        odd |= (o[k] & 0x7f800000u) == 0x7f800000u;
        if (none || n == 0) o[k] = 0u;  // (it may be 0 * NaN)
      }
      if (mine) {  // whole sectors: a lane's row is 512 B from its neighbour's
#pragma unroll
        for (int e = 0; e < 4; ++e)
          store8(p.part_acc + slot * kHeadDim + dim + 8 * e, o + 8 * e);
      }
      __syncwarp();
    }
    if (mine && half == 0) {
      p.part_ml[2 * slot] = M;
      p.part_ml[2 * slot + 1] = Z;
    }
    again = mine && odd && !none && Z <= FLT_MAX;
    // (maximum and sum of a row that has to be taken again, below; a sum < 0: it has not)
    *stash(2 + half, row) = again ? make_float2(M, Z) : make_float2(0.f, -1.f);
  }
  fence_before();
  bool any_again = __syncthreads_or(again);
  fence_after();
  if (*give_up) {  // (nobody sets it any more)
    // A wait ran out: copies and products in flight end before their memory goes.  (Otherwise the
    // results were waited for, and with them everything that went into them.)
    any_again = false;
    if (warp == 10) {
      if (elect_lane()) commit(&bars.drain);  // the products that this thread issued
      __syncwarp();
      settle(&bars.drain, 0);
    } else if ((warp == 8 || warp == 9) && lane < kSlots) {
      // copies into slot `lane`: its phases so far
      const int phases = (bars.fetched[warp == 9] + kSlots - 1 - lane) / kSlots;
      if (phases > 0) settle(&bars.full[lane][warp == 9], (uint32_t)(phases - 1) & 1);
    } else if (warp == 8 && lane == kSlots) {
      settle(&bars.q_full, 0);
    }
    __syncthreads();
  }
  if (warp == 10) tmem_free(tmem);

  // An infinity or NaN among the values of a tile reaches all of its rows, as 0 * NaN, those too
  // that do not see its token.  Such a row (its scores are finite, its O is not) is taken again
  // from what it sees, by a warp, a token at a time.
  if (any_again) {
    size_t share;
    item_of(table, lg, &share);
    for (int r = warp; r < (tok1 - tok0) * G; r += kPrefixThreads / 32) {
      const float2 a0 = *stash(2, r), a1 = *stash(3, r);
      if (a0.y < 0.f && a1.y < 0.f) continue;  // warp-uniform
      const float m_r = a0.y < 0.f ? a1.x : a0.x;
      const int seq = it.first + tok0 + (r >> lg);
      const int last = min(min(length(seq), end), j1 * kTokens);
      const uint2 qw = *reinterpret_cast<const uint2*>(
          p.q + ((size_t)seq * p.Hq + ((size_t)it.g << lg) + (r & (G - 1))) * kHeadDim + 4 * lane);
      const float2 qa = h2f(qw.x), qb = h2f(qw.y);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int page = j0 * PPT; page * P < last; ++page) {
        const int phys = p.block_table[(size_t)it.first * p.max_pages + page];
        if (phys < 0 || phys >= p.num_phys) continue;
        const size_t from = ((size_t)phys * p.Hkv + it.g) * P * kHeadDim + 4 * lane;
#pragma unroll 4
        for (int k = 0; k < P; ++k) {
          if (page * P + k >= last) break;
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
      *reinterpret_cast<float4*>(p.part_acc + (share + r) * kHeadDim + 4 * lane) =
          make_float4(acc[0], acc[1], acc[2], acc[3]);
    }
  }
}

}  // namespace

cudaError_t launch_prefix(const Params& p, const PrefixTable& t, cudaStream_t s) {
  Params pp = p;
  const int G = p.Hq / p.Hkv;
  int log_g = G == 8 ? 3 : G / 2;
  CUtensorMap mq, mk, mv;
  const cuuint64_t qd[3] = {kHeadDim, (cuuint64_t)p.Hq, (cuuint64_t)p.B};
  const cuuint64_t qs[2] = {kHeadDim * 2, (cuuint64_t)p.Hq * kHeadDim * 2};
  const cuuint32_t qb[3] = {64, (cuuint32_t)G, (cuuint32_t)(kRows / G)};
  cudaError_t e = make_map(&mq, p.q, 3, qd, qs, qb);
  if (e != cudaSuccess) return e;
  // a pool as [8-row group][half of the dims][row][64 dims]
  const cuuint64_t kd[4] = {64, 8, 2, (cuuint64_t)p.num_phys * p.Hkv * (p.P / 8)};
  const cuuint64_t ks[3] = {kHeadDim * 2, kHeadDim, 8 * kHeadDim * 2};
  const cuuint32_t kb[4] = {64, 8, 2, (cuuint32_t)(p.P / 8)};
  if ((e = make_map(&mk, p.k_pool, 4, kd, ks, kb)) != cudaSuccess) return e;
  if ((e = make_map(&mv, p.v_pool, 4, kd, ks, kb)) != cudaSuccess) return e;
  const void* fn = p.P == 16 ? (const void*)prefix_kernel<16> : (const void*)prefix_kernel<32>;
  const size_t smem = Smem::total + 1024;
  if ((e = ensure_smem(fn, smem)) != cudaSuccess) return e;
  void* args[] = {&pp, const_cast<PrefixTable*>(&t), &log_g, &mq, &mk, &mv};
  return launch_pdl(fn, dim3((unsigned)t.ctas), dim3(kPrefixThreads), smem, s, args);
}

}  // namespace quest
