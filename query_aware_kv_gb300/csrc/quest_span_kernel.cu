// quest_span_kernel.cu - split-K attention of single query tokens over a run of pages of a
// paged cache, on matrix instructions fed straight from global memory.
//
// One row is (query token, kv head): its G = 1..8 query heads attend over a list of pages
// (every page, a selection, or the pages of a few sink tokens and of a sliding window):
//   out_h = sum_t softmax_t(q_h . k_t / sqrt(128)) v_t,   lse_h = log sum_t exp(...)
// The cache is fp16, or e4m3 with an fp32 scale per (page, kv head) and an fp16 open page.
//
// What bounds it: DRAM.  A token costs 512 B (fp16) or 256 B (e4m3) and 512 G flops.  On
// the FP32 lanes eight heads over an e4m3 cache would need 54 TFMA/s at the copy rate, more
// than the card has; mma.m16n8k16 takes the G heads as its eight columns and needs under a
// fifth of that pipe.  tcgen05 would need the e4m3 tokens widened into shared memory first
// (q is fp16, and both operands of one product have the same type) and buys nothing while
// the pipe idles.
//
// Layout: a warp takes 16 tokens at a time, K and V go from global memory to the registers
// of the lanes that multiply them, with no shared memory, barrier or wait in the loop: the
// order of the contraction index is free, so lane (r, c) (r = lane / 4, c = lane % 4) owns
// whole 16-byte pieces of K rows r and r + 8, and for V the 16-byte pieces at its r of the
// tokens {2c, 2c+1, 2c+8, 2c+9}, whose columns a byte permute turns into V^T fragments.
//   S^T [16 tokens x 8 heads] = K Q^T          (8 mma)
//   O^T [128 dims  x 8 heads] += V^T P         (8 mma for the upper halves of P's fp32
//                                               values and 8 for the lower ones)
// P is split into two fp16 numbers (22 bits), so that its rounding stays below that of the
// fp32 sums; the second product costs nothing next to the loads.  The running maximum moves
// only when a score exceeds it by more than kLazy (in log2 units): weights are
// 2^(s - m + kBias), so that the largest stay below 2^(kBias + kLazy) = 2^14 and the small
// ones keep fp16's full precision down to 2^-22 of the reference.
//
// Measured (calls back to back): eight ragged 32K sequences of 32 heads, 4K window, fp16:
// 81.0 us, 6.63 TB/s; full e4m3 attention over four 64K sequences of 32 / 8 heads: 94.4 us,
// 5.7 TB/s; 16 ragged e4m3 sequences of 32 / 8 heads, 8K window: 56 us, 4.8 TB/s (256 CTAs on
// 304 places, each waiting on its loads: DRAM at 58 %).  Tried and slower: equal runs of all
// rows' pages (a run that crosses into a new row pays that row's latency again), and copies
// through shared memory with cp.async (128 us for the 94.4).  A CTA that takes its pages again (a NaN or
// an infinity among the values that it sees) is slow: the 94.4 us become 1.8 ms.
#include <math_constants.h>

#include <algorithm>
#include <cfloat>

#include "quest_device.cuh"

namespace quest {

namespace {

constexpr int kSms = 152;  // of a GB300
constexpr int kMaxSplitsSpan = 64;
constexpr int kMinBlocks = 4;  // 16-token blocks of a split, at least
constexpr int kClusterSplits = 8;  // splits of a row whose CTAs are a cluster, at most
constexpr float kBias = 8.f;
constexpr float kLazy = 6.f;

// D += A B, A 16x16 (row), B 16x8 (col), fp16 with fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8x8 transpose of b16 over the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two e4m3 numbers (16 bits) widened to fp16, exactly.
__device__ __forceinline__ uint32_t widen(uint32_t two) {
  uint32_t y;
  asm("{\n\t.reg .b16 t;\n\tmov.b32 {t, _}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(y)
      : "r"(two));
  return y;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ uint32_t pack(__half a, __half b) {
  const __half2 h = __halves2half2(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The address of `local` in the shared memory of CTA `rank` of the cluster, and a float there.
__device__ __forceinline__ uint32_t peer_at(const void* local, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  return a;
}
__device__ __forceinline__ float peer_float(uint32_t at) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ void cluster_barrier() {
  __syncthreads();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// Which dims a lane holds.  k-step s of K Q^T multiplies dims dk .. dk + 3 of lane column c;
// tile m of V^T P owns dims dv and dv + 1 of lane row r.  The e4m3 pieces are 16 dims wide,
// the fp16 pieces 8; each keeps 64 or 128 B contiguous over the lanes of a load.
template <bool N8> __device__ __forceinline__ int dk(int s, int c) {
  return N8 ? 64 * (s >> 2) + 16 * c + 4 * (s & 3) : 32 * (s >> 1) + 8 * c + 4 * (s & 1);
}
template <bool N8> __device__ __forceinline__ int dv(int m, int r) {
  return N8 ? 16 * r + 2 * m : 64 * (m >> 2) + 8 * r + 2 * (m & 3);
}

// The part of a row's softmax that one warp holds: reference maximum and (this lane's share
// of the) sum for heads 2c and 2c + 1, and O^T.
struct State {
  float m[2], l[2];
  float acc[8][4];
};

// What brings a part of a softmax (reference m, sum l) to the reference M of all parts.  A part
// without a weight has m = -inf and l = 0.  Scores that are NaN move no maximum but make l one: with
// m = -inf too such a part is not left out, its NaN goes on.  Whether a row has seen a token is read
// from its sum alone.  A part's share may be an infinity (of a visible value), which no factor may
// turn into 0 * inf: the smallest normal number adds nothing to any other sum.
__device__ __forceinline__ float part_factor(float m, float l, float M) {
  return m == -CUDART_INF_F ? (l == 0.f ? 0.f : 1.f) : fmaxf(exp2f(m - M), FLT_MIN);
}
// Output and log-sum-exp of a row: A = sum of weights times values, Z = sum of weights.
__device__ __forceinline__ __half row_out(float A, float Z) {
  return __float2half_rn(Z == 0.f ? 0.f : A / Z);
}
__device__ __forceinline__ float row_lse(float M, float Z) {
  return Z == 0.f ? -CUDART_INF_F : (M - kBias + log2f(Z)) * 0.6931471805599453f;
}

// Scores of a block (16 tokens) to weights: updates m, l and rescales acc when the
// reference moves; returns P^T as fp16 pairs, upper and lower parts.
__device__ __forceinline__ void weigh(State& st, float (&s)[4], uint32_t& h0, uint32_t& h1,
                                      uint32_t& l0, uint32_t& l1) {
  const bool over = fmaxf(s[0], s[2]) > st.m[0] + kLazy || fmaxf(s[1], s[3]) > st.m[1] + kLazy;
  if (__any_sync(0xffffffffu, over)) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = fmaxf(s[e], s[2 + e]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float m = fmaxf(st.m[e], top);
      const float f = m == -CUDART_INF_F ? 1.f : exp2f(st.m[e] - m);
      st.m[e] = m;
      st.l[e] *= f;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        st.acc[t][e] *= f;
        st.acc[t][2 + e] *= f;
      }
    }
  }
  float w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float ref = st.m[i & 1] == -CUDART_INF_F ? 0.f : st.m[i & 1];
    w[i] = exp2f(s[i] - ref + kBias);
    st.l[i & 1] += w[i];
  }
  __half hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hi[i] = __float2half_rn(w[i]);
    lo[i] = __float2half_rn(w[i] - __half2float(hi[i]));
  }
  h0 = transpose8x8(pack(hi[0], hi[1]));
  h1 = transpose8x8(pack(hi[2], hi[3]));
  l0 = transpose8x8(pack(lo[0], lo[1]));
  l1 = transpose8x8(pack(lo[2], lo[3]));
}

// acc[m] += scale * V^T P for one tile m, from this lane's V fragments.
template <bool kScaled>
__device__ __forceinline__ void add_tile(State& st, int m, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t h0, uint32_t h1, uint32_t l0,
                                         uint32_t l1, float scale) {
  if constexpr (kScaled) {
    float t[4] = {0.f, 0.f, 0.f, 0.f};
    mma16816(t, a0, a1, a2, a3, l0, l1);
    mma16816(t, a0, a1, a2, a3, h0, h1);
#pragma unroll
    for (int i = 0; i < 4; ++i) st.acc[m][i] = fmaf(t[i], scale, st.acc[m][i]);
  } else {
    mma16816(st.acc[m], a0, a1, a2, a3, l0, l1);
    mma16816(st.acc[m], a0, a1, a2, a3, h0, h1);
  }
}

// Scores masked to the visible tokens: token t is visible if t < end and (t < sink_end or
// t >= lo).
struct Visible {
  int end, lo, sink_end;
  __device__ __forceinline__ bool token(int t) const {
    return t < end && (t < sink_end || t >= lo);
  }
  __device__ __forceinline__ bool all16(int t) const {
    return t + 16 <= end && (t + 16 <= sink_end || t >= lo);
  }
};

// One 16-token block whose K / V rows are fp16 at kp / vp (row stride 128): the open page
// of a narrow cache, in the narrow kernel's dims.
__device__ __forceinline__ void open_block(State& st, const uint32_t (&qf)[8][2],
                                           const __half* kp, const __half* vp, int t0,
                                           const Visible& vis, float qscale, int r, int c) {
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint4 a[2], z[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      a[u] = *reinterpret_cast<const uint4*>(kp + r * kHeadDim + 64 * half + 16 * c + 8 * u);
      z[u] = *reinterpret_cast<const uint4*>(kp + (r + 8) * kHeadDim + 64 * half + 16 * c + 8 * u);
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int i = 2 * (w & 1);
      mma16816(s, word(a[w >> 1], i), word(z[w >> 1], i), word(a[w >> 1], i + 1),
               word(z[w >> 1], i + 1), qf[4 * half + w][0], qf[4 * half + w][1]);
    }
  }
  const int ta = t0 + r, tz = t0 + r + 8;
  s[0] = vis.token(ta) ? s[0] * qscale : -CUDART_INF_F;
  s[1] = vis.token(ta) ? s[1] * qscale : -CUDART_INF_F;
  s[2] = vis.token(tz) ? s[2] * qscale : -CUDART_INF_F;
  s[3] = vis.token(tz) ? s[3] * qscale : -CUDART_INF_F;
  uint32_t h0, h1, l0, l1;
  weigh(st, s, h0, h1, l0, l1);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = 2 * c + (j & 1) + 8 * (j >> 1);
      v[j] = vis.token(t0 + t) ? *reinterpret_cast<const uint4*>(vp + t * kHeadDim + 16 * r + 8 * u)
                               : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      add_tile<false>(st, 4 * u + i, __byte_perm(word(v[0], i), word(v[1], i), 0x5410),
                      __byte_perm(word(v[0], i), word(v[1], i), 0x7632),
                      __byte_perm(word(v[2], i), word(v[3], i), 0x5410),
                      __byte_perm(word(v[2], i), word(v[3], i), 0x7632), h0, h1, l0, l1, 1.f);
  }
}

// K and V of one block, as loaded.
template <bool N8>
struct Block {
  static constexpr int kN = N8 ? 4 : 8;
  uint4 k[kN], v[kN];
};

template <bool N8>
__device__ __forceinline__ void load_k(Block<N8>& x, const unsigned char* kp, int r, int c) {
  if constexpr (N8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x.k[i] = ld_stream_v4(kp + (r + 8 * (i >> 1)) * kHeadDim + 64 * (i & 1) + 16 * c);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x.k[i] = ld_stream_v4(kp + (r + 8 * (i >> 2)) * 2 * kHeadDim + 64 * (i & 3) + 16 * c);
  }
}
template <bool N8>
__device__ __forceinline__ void load_v(Block<N8>& x, const unsigned char* vp, int r, int c) {
  if constexpr (N8) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x.v[j] = ld_stream_v4(vp + (2 * c + (j & 1) + 8 * (j >> 1)) * kHeadDim + 16 * r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x.v[j] = ld_stream_v4(vp + (2 * c + ((j >> 1) & 1) + 8 * (j >> 2)) * 2 * kHeadDim + 128 * (j & 1) +
                      16 * r);
  }
}

template <bool N8>
__device__ __forceinline__ void scores(const Block<N8>& x, const uint32_t (&qf)[8][2],
                                       float (&s)[4]) {
  float u[4] = {0.f, 0.f, 0.f, 0.f};
  s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    uint32_t a0, a1, a2, a3;
    if constexpr (N8) {
      const uint32_t p = word(x.k[t >> 2], t & 3), z = word(x.k[2 + (t >> 2)], t & 3);
      a0 = widen(p);
      a2 = widen(p >> 16);
      a1 = widen(z);
      a3 = widen(z >> 16);
    } else {
      const int i = 2 * (t & 1);
      a0 = word(x.k[t >> 1], i);
      a2 = word(x.k[t >> 1], i + 1);
      a1 = word(x.k[4 + (t >> 1)], i);
      a3 = word(x.k[4 + (t >> 1)], i + 1);
    }
    mma16816((t & 1) ? u : s, a0, a1, a2, a3, qf[t][0], qf[t][1]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] += u[i];
}

// Values of tokens that the row does not see may be anything (a slot never written, a
// token behind the window): their weight is 0, and 0 * NaN would not be.
template <bool N8>
__device__ __forceinline__ void zero_hidden(Block<N8>& x, const Visible& vis, int t0, int c) {
#pragma unroll
  for (int j = 0; j < Block<N8>::kN; ++j) {
    const int e = N8 ? j : j >> 1;
    if (!vis.token(t0 + 2 * c + (e & 1) + 8 * (e >> 1))) x.v[j] = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <bool N8>
__device__ __forceinline__ void accumulate(State& st, const Block<N8>& x, uint32_t h0, uint32_t h1,
                                           uint32_t l0, uint32_t l1, float vscale) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (N8) {
      // bytes (d, d + 1) of two tokens: {t0 d, t1 d, t0 d+1, t1 d+1}
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t sel = e ? 0x7362 : 0x5140;
        const uint32_t p = __byte_perm(word(x.v[0], i), word(x.v[1], i), sel);
        const uint32_t z = __byte_perm(word(x.v[2], i), word(x.v[3], i), sel);
        add_tile<true>(st, 2 * i + e, widen(p), widen(p >> 16), widen(z), widen(z >> 16), h0, h1,
                       l0, l1, vscale);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t a = word(x.v[u], i), b = word(x.v[2 + u], i);
        const uint32_t y = word(x.v[4 + u], i), z = word(x.v[6 + u], i);
        add_tile<false>(st, 4 * u + i, __byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632),
                        __byte_perm(y, z, 0x5410), __byte_perm(y, z, 0x7632), h0, h1, l0, l1, 1.f);
      }
    }
  }
}

// What a query token of sequence b attends over: `count` pages, in the row's order.
struct RowShape {
  Visible vis;
  int L, N, n_sink, first, count;
};

__device__ __forceinline__ RowShape row_shape(const SpanParams& sp, int b) {
  const Params& p = sp.p;
  RowShape x;
  x.L = step_len(p, b, p.seq_lens[b], kSiteSpan);
  x.N = (x.L + p.P - 1) / p.P;
  x.vis = Visible{x.L, 0, 0};
  x.n_sink = x.first = 0;
  x.count = x.N;
  if (sp.mode == kSpanWindow) {
    x.vis.lo = max(0, x.L - sp.window);
    x.vis.sink_end = min(sp.sink, x.vis.lo);
    x.first = x.vis.lo / p.P;
    x.n_sink = min((x.vis.sink_end + p.P - 1) / p.P, x.first);
    x.count = x.n_sink + x.N - x.first;
  } else if (sp.mode == kSpanList) {
    x.count = min(p.top_k, x.N);  // at most
  }
  return x;
}

// A weight's two fp16 parts times an infinity are NaN (the lower part is 0 or of either sign), and
// so is a weight below fp16's range.  Where a head's O is not finite although its scores are, the
// warps of the CTA take the CTA's pages again, token by token, lane l the dims 4 l .. 4 l + 3 with
// fp32 weights against the CTA's maximum: what leaves is then what the row sees, infinities as
// infinities.  red: this warp's shares, [G][128].  list: the pages of kSpanList, `count` of them.
template <bool N8, int kSpanWarps>
__device__ __forceinline__ void take_again(const SpanParams& sp, int row, int split,
                                           const int* list, int count,
                                           const float (&s_m)[kSpanWarps][8], float* red) {
  const Params& p = sp.p;
  const int b = row / p.Hkv, g = row % p.Hkv, G = p.Hq / p.Hkv, P = p.P;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RowShape x = row_shape(sp, b);
  if (sp.mode == kSpanList) count = max(0, min(count, x.count));
  else count = x.count;
  const int i1 = count * (split + 1) / p.n_splits;
  const int open_page = (N8 && x.L % P) ? x.L / P : -1;
#pragma unroll 1
  for (int h = 0; h < G; ++h) {
    float M = -CUDART_INF_F;
    for (int w = 0; w < kSpanWarps; ++w) M = fmaxf(M, s_m[w][h]);
    const uint2 qw = *reinterpret_cast<const uint2*>(
        p.q + ((size_t)b * p.Hq + (size_t)g * G + h) * kHeadDim + 4 * lane);
    const float2 qa = h2f(qw.x), qb = h2f(qw.y);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int i = count * split / p.n_splits + warp; i < i1; i += kSpanWarps) {
      const int lp = sp.mode == kSpanDense ? i
                     : sp.mode == kSpanList ? list[i]
                     : i < x.n_sink ? i : x.first + i - x.n_sink;
      if (lp < 0 || lp >= x.N) continue;
      const bool open = lp == open_page;
      const int phys = open ? 0 : p.block_table[(size_t)b * p.max_pages + lp];
      if (phys < 0 || phys >= p.num_phys) continue;
      const size_t at = (size_t)phys * p.Hkv + g;
      const float ks = N8 && !open ? p.qscale * sp.nar.k_scale[at] : p.qscale;
      const float vs = N8 && !open ? sp.nar.v_scale[at] : 1.f;
#pragma unroll 1
      for (int k = 0; k < P; ++k) {
        if (!x.vis.token(lp * P + k)) continue;
        uint2 kw, vw;
        if (N8 && !open) {
          const size_t from = (at * P + k) * kHeadDim + 4 * lane;
          const uint32_t kc = *reinterpret_cast<const uint32_t*>(sp.nar.k_pool + from);
          const uint32_t vc = *reinterpret_cast<const uint32_t*>(sp.nar.v_pool + from);
          kw = make_uint2(widen(kc), widen(kc >> 16));
          vw = make_uint2(widen(vc), widen(vc >> 16));
        } else {
          const size_t from = ((open ? (size_t)row : at) * P + k) * kHeadDim + 4 * lane;
          kw = *reinterpret_cast<const uint2*>((open ? sp.nar.k_open : p.k_pool) + from);
          vw = *reinterpret_cast<const uint2*>((open ? sp.nar.v_open : p.v_pool) + from);
        }
        const float2 ka = h2f(kw.x), kb = h2f(kw.y), va = h2f(vw.x), vb = h2f(vw.y);
        const float s =
            ks * warp_sum(fmaf(qa.x, ka.x, qa.y * ka.y) + fmaf(qb.x, kb.x, qb.y * kb.y));
        // (as for parts: no weight but that of a score of -inf is 0)
        const float w = s == -CUDART_INF_F ? 0.f : vs * fmaxf(exp2f(s - M + kBias), FLT_MIN);
        acc[0] = fmaf(w, va.x, acc[0]);
        acc[1] = fmaf(w, va.y, acc[1]);
        acc[2] = fmaf(w, vb.x, acc[2]);
        acc[3] = fmaf(w, vb.y, acc[3]);
      }
    }
    *reinterpret_cast<float4*>(red + h * kHeadDim + 4 * lane) =
        make_float4(acc[0], acc[1], acc[2], acc[3]);
  }
}

// grid rows * n_splits (split fastest): split s of a row takes the s-th share of its pages,
// warp w of the CTA every kSpanWarps-th page of that.  A split row's parts are joined through
// the shared memory of a cluster (the row's CTAs), or by the CTA that comes last to the row.
// kSelect (a chain step without a top-K kernel): every CTA of a row takes the row's selection from
// the scores itself, the same in each; split 0 also writes the caller's copy.
template <bool N8, int kSpanWarps, int kCtas, int kDepth, bool kSelect>
__global__ void __launch_bounds__(32 * kSpanWarps, kCtas) span_kernel(SpanParams sp) {
  constexpr int kSpanThreads = 32 * kSpanWarps;
  __shared__ float s_m[kSpanWarps][8], s_l[kSpanWarps][8];
  __shared__ __align__(16) float s_red[kSpanWarps][8 * kHeadDim];
  __shared__ float s_part[2][8];  // a part's maxima and sums, for the cluster
  __shared__ int s_flag;
  const Params& p = sp.p;
  pdl_wait();
  pdl_trigger();  // the next call's CTAs may take the places that this one's free
  const int split = (int)(blockIdx.x % (unsigned)p.n_splits);
  const int row = (int)(blockIdx.x / (unsigned)p.n_splits);  // b * Hkv + g
  const int b = row / p.Hkv, g = row % p.Hkv;
  const int G = p.Hq / p.Hkv, P = p.P;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;

  const RowShape shape = row_shape(sp, b);
  const int L = shape.L, N = shape.N, n_sink = shape.n_sink, first = shape.first;
  const Visible vis = shape.vis;
  int count = shape.count;
  const int* list = nullptr;
  if (sp.mode == kSpanList) {
    int given = 0;
    if constexpr (kSelect) {
      extern __shared__ __align__(16) unsigned char s_sel[];
      int* scratch = reinterpret_cast<int*>(s_sel + topk_smem_bytes(p.max_pages));  // [256]
      int* kept = scratch + 256;                                                    // [top_k]
      topk_row<kSpanThreads, false>(p.scores + (size_t)row * p.max_pages, N, p.top_k,
                                    p.sink_pages, p.local_pages, kept, &s_flag,
                                    topk_smem_at(s_sel, p.max_pages), scratch);
      __syncthreads();
      list = kept;
      given = s_flag;
      if (split == 0) {
        for (int i = threadIdx.x; i < p.top_k; i += kSpanThreads)
          p.sel_idx[(size_t)row * p.top_k + i] = kept[i];
        if (threadIdx.x == 0) p.sel_count[row] = given;
      }
    } else {
      list = p.sel_idx + (size_t)row * p.top_k;
      given = p.sel_count[row];
    }
    if ((given < 0 || given > count) && threadIdx.x == 0 && split == 0)
      report(p, QUEST_ERR_BAD_SELECTION, b, given, kSiteSelection);
    count = max(0, min(given, count));
  }
  const int i0 = count * split / p.n_splits, i1 = count * (split + 1) / p.n_splits;

  // ---- the query: head r of the group in lane (r, c)'s K Q^T columns
  const size_t head0 = (size_t)b * p.Hq + (size_t)g * G;
  uint32_t qf[8][2];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    uint2 w = make_uint2(0u, 0u);
    if (r < G)
      w = *reinterpret_cast<const uint2*>(p.q + (head0 + r) * kHeadDim + dk<N8>(t, c));
    qf[t][0] = w.x;
    qf[t][1] = w.y;
  }

  State st;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    st.m[e] = -CUDART_INF_F;
    st.l[e] = 0.f;
  }
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) st.acc[m][e] = 0.f;

  const unsigned char* k_pool =
      N8 ? sp.nar.k_pool : reinterpret_cast<const unsigned char*>(p.k_pool);
  const unsigned char* v_pool =
      N8 ? sp.nar.v_pool : reinterpret_cast<const unsigned char*>(p.v_pool);
  const int row_bytes = N8 ? kHeadDim : 2 * kHeadDim;
  const int open_page = (N8 && L % P) ? L / P : -1;
  const int per_page = P / 16;
  bool has_open = false;

  // ---- the warp's pages, 32 at a time: lane j looks the j-th one up
  for (int base = i0 + warp; base < i1; base += 32 * kSpanWarps) {
    const int mine = base + kSpanWarps * lane;
    int lp = -1, phys = 0, ok = 0;
    float ks = p.qscale, vs = 1.f;
    if (mine < i1) {
      lp = sp.mode == kSpanDense ? mine
           : sp.mode == kSpanList ? list[mine]
           : mine < n_sink ? mine : first + mine - n_sink;
      if (lp < 0 || lp >= N) {
        report(p, QUEST_ERR_BAD_SELECTION, b, lp, kSiteSelection);
      } else if (lp == open_page) {
        ok = 2;
      } else {
        phys = p.block_table[(size_t)b * p.max_pages + lp];
        if (phys < 0 || phys >= p.num_phys) {
          report(p, QUEST_ERR_BAD_PAGE, b, lp, kSiteSpan);
          phys = 0;
        } else {
          ok = 1;
          if constexpr (N8) {
            ks *= sp.nar.k_scale[(size_t)phys * p.Hkv + g];
            vs = sp.nar.v_scale[(size_t)phys * p.Hkv + g];
          }
        }
      }
    }
    has_open |= __any_sync(0xffffffffu, ok == 2);
    // blocks of the pages to stream; a page that is not (unmapped, open) is left out
    unsigned live = __ballot_sync(0xffffffffu, ok == 1);
    if (!live) continue;
    // kDepth blocks on their way: K of the next one is asked for as soon as the scores are
    // taken, V once the values are
    Block<N8> x[kDepth];
    struct Next {
      size_t off;
      int t0, valid;
      float ks, vs;
    } nx[kDepth];
    int sub = 0;
    auto take = [&]() {
      Next n;
      n.valid = live != 0u;
      const int j = n.valid ? __ffs(live) - 1 : 0;
      n.off = (((size_t)__shfl_sync(0xffffffffu, phys, j) * p.Hkv + g) * P + 16 * sub) * row_bytes;
      n.t0 = __shfl_sync(0xffffffffu, lp, j) * P + 16 * sub;
      n.ks = N8 ? __shfl_sync(0xffffffffu, ks, j) : p.qscale;
      n.vs = N8 ? __shfl_sync(0xffffffffu, vs, j) : 1.f;
      if (++sub == per_page) {
        sub = 0;
        live &= live - 1u;
      }
      return n;
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      nx[d] = take();
      if (nx[d].valid) {
        load_k<N8>(x[d], k_pool + nx[d].off, r, c);
        load_v<N8>(x[d], v_pool + nx[d].off, r, c);
      }
    }
    while (nx[0].valid) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (nx[d].valid) {
          const Next now = nx[d];
          float s[4];
          scores<N8>(x[d], qf, s);
          nx[d] = take();
          if (nx[d].valid) load_k<N8>(x[d], k_pool + nx[d].off, r, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] *= now.ks;
          if (!vis.all16(now.t0)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!vis.token(now.t0 + r + 8 * (i >> 1))) s[i] = -CUDART_INF_F;
            zero_hidden<N8>(x[d], vis, now.t0, c);
          }
          uint32_t h0, h1, l0, l1;
          weigh(st, s, h0, h1, l0, l1);
          accumulate<N8>(st, x[d], h0, h1, l0, l1, now.vs);
          if (nx[d].valid) load_v<N8>(x[d], v_pool + nx[d].off, r, c);
        }
      }
    }
  }
  if (N8 && has_open) {
    const size_t o = ((size_t)b * p.Hkv + g) * P * kHeadDim;
    for (int sub = 0; sub < per_page; ++sub)
      if (open_page * P + 16 * sub < vis.end)
        open_block(st, qf, sp.nar.k_open + o + sub * 16 * kHeadDim,
                   sp.nar.v_open + o + sub * 16 * kHeadDim, open_page * P + 16 * sub, vis,
                   p.qscale, r, c);
  }

  // ---- the warps' states into one
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], o);
  if (r == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s_m[warp][2 * c + e] = st.m[e];
      s_l[warp][2 * c + e] = st.l[e];
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int h = 2 * c + e;
    if (h < G) {
      float M = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kSpanWarps; ++w) M = fmaxf(M, s_m[w][h]);
      const float f = part_factor(st.m[e], st.l[e], M);
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        *reinterpret_cast<float2*>(&s_red[warp][h * kHeadDim + dv<N8>(m, r)]) =
            make_float2(st.acc[m][e] * f, st.acc[m][2 + e] * f);
      }
    }
  }
  __syncthreads();
  const size_t slot0 = (size_t)row * p.n_splits * G;  // parts: [row][split][head]
  const size_t mine = slot0 + (size_t)split * G;
  for (int pass = 0;; ++pass) {
    bool odd = false;  // (found on the sums: a check of every warp's O cost the e4m3 rows 2 %)
    for (int o = threadIdx.x; o < G * kHeadDim; o += kSpanThreads) {
      const int h = o / kHeadDim, d = o % kHeadDim;
      float M = -CUDART_INF_F, Z = 0.f, A = 0.f;
#pragma unroll
      for (int w = 0; w < kSpanWarps; ++w) M = fmaxf(M, s_m[w][h]);
#pragma unroll
      for (int w = 0; w < kSpanWarps; ++w) {
        A += s_red[w][o];
        Z = fmaf(s_l[w][h], part_factor(s_m[w][h], s_l[w][h], M), Z);
      }
      odd |= !(fabsf(A) <= FLT_MAX) && Z <= FLT_MAX;
      if (p.n_splits == 1) {
        p.out[(head0 + h) * kHeadDim + d] = row_out(A, Z);
        if (d == 0 && p.lse) p.lse[head0 + h] = row_lse(M, Z);
      } else if (sp.cluster) {
        s_red[0][o] = A;  // (this thread's alone to read and write)
        if (d == 0) {
          s_part[0][h] = M;
          s_part[1][h] = Z;
        }
      } else {
        p.part_acc[(mine + h) * kHeadDim + d] = A;
        if (d == 0) {
          p.part_ml[2 * (mine + h)] = M;
          p.part_ml[2 * (mine + h) + 1] = Z;
        }
      }
    }
    if (!__syncthreads_or(odd) || pass) break;
    const int* list = p.sel_idx + (size_t)row * p.top_k;
    int given = 0;
    if constexpr (kSelect) {
      extern __shared__ __align__(16) unsigned char s_sel[];
      list = reinterpret_cast<const int*>(s_sel + topk_smem_bytes(p.max_pages)) + 256;
      given = s_flag;
    } else if (sp.mode == kSpanList) {
      given = p.sel_count[row];
    }
    take_again<N8, kSpanWarps>(sp, row, split, list, given, s_m, s_red[warp]);
    __syncthreads();
  }
  if (p.n_splits > 1 && sp.cluster) {
    // ---- every CTA of the row (rank = split) joins its share of the outputs
    const int n = p.n_splits;
    cluster_barrier();
    for (int o = split * kSpanThreads + (int)threadIdx.x; o < G * kHeadDim;
         o += n * kSpanThreads) {
      const int h = o / kHeadDim, d = o % kHeadDim;
      float m[kClusterSplits], z[kClusterSplits], a[kClusterSplits];
#pragma unroll
      for (int e = 0; e < kClusterSplits; ++e) {
        const int from = min(e, n - 1);
        m[e] = peer_float(peer_at(&s_part[0][h], from));
        z[e] = peer_float(peer_at(&s_part[1][h], from));
        a[e] = peer_float(peer_at(&s_red[0][o], from));
      }
      float M = -CUDART_INF_F, Z = 0.f, A = 0.f;
#pragma unroll
      for (int e = 0; e < kClusterSplits; ++e) M = fmaxf(M, m[e]);
#pragma unroll
      for (int e = 0; e < kClusterSplits; ++e) {
        const float f = e >= n ? 0.f : part_factor(m[e], z[e], M);
        Z = fmaf(z[e], f, Z);
        A = e < n ? fmaf(a[e], f, A) : A;
      }
      p.out[(head0 + h) * kHeadDim + d] = row_out(A, Z);
      if (d == 0 && p.lse) p.lse[head0 + h] = row_lse(M, Z);
    }
    cluster_barrier();  // no CTA leaves while another may still read its shared memory
  } else if (p.n_splits > 1) {
    // ---- the last CTA of the row joins its parts
    const int n = p.n_splits;
    if (arrive_last<kSpanThreads, false>(&p.decode_arrive[row], (unsigned)n, &s_flag)) {
      auto slot = [&](int s, int h) { return slot0 + (size_t)s * G + h; };
      float* msc = &s_red[0][0];  // [G][n] scales
      for (int h = warp; h < G; h += kSpanWarps) {
        float M = -CUDART_INF_F, Z = 0.f;
        for (int s = lane; s < n; s += 32) M = fmaxf(M, __ldcg(p.part_ml + 2 * slot(s, h)));
        M = warp_max(M);
        for (int s = lane; s < n; s += 32) {
          const float ms = __ldcg(p.part_ml + 2 * slot(s, h));
          const float ls = __ldcg(p.part_ml + 2 * slot(s, h) + 1);
          const float f = part_factor(ms, ls, M);
          msc[h * n + s] = f;
          Z = fmaf(ls, f, Z);
        }
        Z = warp_sum(Z);
        if (lane == 0) {
          s_m[0][h] = M;
          s_l[0][h] = Z;
        }
      }
      __syncthreads();
      // four outputs a thread; threads left over take every groups-th part of the same ones (one
      // output a thread took 27 us where this takes 17: four e4m3 rows of eight heads, 64 splits)
      const int units = G * kHeadDim / 4, groups = max(1, kSpanThreads / units);
      float4* shares = reinterpret_cast<float4*>(&s_red[1][0]);  // [groups][units]
      for (int u0 = 0; u0 < units; u0 += kSpanThreads) {
        const int u = groups > 1 ? (int)threadIdx.x % units : u0 + (int)threadIdx.x;
        const int grp = groups > 1 ? (int)threadIdx.x / units : 0;
        const int h = u / (kHeadDim / 4);
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = grp; s0 < n; s0 += 8 * groups) {  // eight loads side by side
          float4 x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int s = s0 + e * groups;
            x[e] = s < n ? __ldcg(reinterpret_cast<const float4*>(p.part_acc + slot(s, h) * kHeadDim) +
                                  u % (kHeadDim / 4))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float f = msc[h * n + min(s0 + e * groups, n - 1)];
            A.x = fmaf(x[e].x, f, A.x);
            A.y = fmaf(x[e].y, f, A.y);
            A.z = fmaf(x[e].z, f, A.z);
            A.w = fmaf(x[e].w, f, A.w);
          }
        }
        shares[grp * units + u] = A;
      }
      __syncthreads();
      for (int o = threadIdx.x; o < G * kHeadDim; o += kSpanThreads) {
        const int h = o / kHeadDim, d = o % kHeadDim;
        const float M = s_m[0][h], Z = s_l[0][h];
        float A = 0.f;
        for (int grp = 0; grp < groups; ++grp)
          A += reinterpret_cast<const float*>(shares)[grp * units * 4 + o];
        p.out[(head0 + h) * kHeadDim + d] = row_out(A, Z);
        if (d == 0 && p.lse) p.lse[head0 + h] = row_lse(M, Z);
      }
      if (threadIdx.x == 0) p.decode_arrive[row] = 0u;
    }
  }

  // ---- a step that appended: the last CTA of the launch (all have read the lengths by then)
  // advances every sequence that had room and a mapped page for its token
  if (p.chain_append && arrive_last<kSpanThreads, false>(p.exited, gridDim.x, &s_flag)) {
    for (int b = threadIdx.x; b < p.B; b += kSpanThreads) {
      const int L0 = p.seq_lens[b];
      if (L0 >= 0 && (long long)L0 + 1 <= (long long)p.max_pages * P) {
        const int phys = p.block_table[(size_t)b * p.max_pages + L0 / P];
        if (phys >= 0 && phys < p.num_phys) p.seq_lens[b] = L0 + 1;
      }
    }
    if (threadIdx.x == 0) *p.exited = 0u;
  }
}

}  // namespace

// Launch shapes: warps of a CTA, CTAs that an SM holds, blocks in flight a warp.  A narrow
// block is 32 registers a lane and leaves room for 16 warps of one block (at 128 registers a lane,
// of which the compiler spills 56 bytes, 64 where the CTAs select; no shape without a spill has
// been measured); an fp16 block is 64, for 8 warps of two.  With more rows than SMs the fp16 rows get CTAs of four warps, two of
// which share an SM: eight sequences of 32 heads with a 4K window took 85.6 us at 8 warps and
// 81.4 at 4, one sequence of 8 heads over 64K tokens 48.4 at 8 and 55.2 at 4.
struct SpanShape {
  int warps, ctas;
  const void* fn;
};

static SpanShape span_shape(bool narrow, long long rows) {
  if (narrow) return {8, 2, (const void*)span_kernel<true, 8, 2, 1, false>};
  if (rows > kSms) return {4, 2, (const void*)span_kernel<false, 4, 2, 2, false>};
  return {8, 1, (const void*)span_kernel<false, 8, 1, 2, false>};
}

// Splits of a row: as many as fit the GPU together with the other rows' in one wave, with a few
// blocks for every split.  A second wave costs more than the places that stay empty in the
// first (32 rows of 64K tokens: 96 us at 9 splits, 288 CTAs on 304 places, 143 us at 10), unless
// two waves fill much better than one (64 rows: 84 % and 95 %; ragged ones took 86 us at 4
// splits and 66 at 9).
struct SpanSplits {
  int n;
  bool cluster;
};

static SpanSplits span_splits(const SpanParams& sp, const SpanShape& shape, int pages) {
  const long long rows = (long long)sp.p.B * sp.p.Hkv;
  if (rows > kSplitRows) return {1, false};
  if (sp.run_pages)
    return {std::max(1, std::min((pages + sp.run_pages - 1) / sp.run_pages, kMaxSplitsSpan)),
            false};
  const long long slots = (long long)kSms * shape.ctas;
  long long s = std::max<long long>(1, slots / rows);
  const long long two = 2 * slots / rows;
  if (rows * s * 100 < slots * 88 && rows * two * 100 >= 2 * slots * 94) s = two;
  const int blocks = pages * (sp.p.P / 16);
  const int n =
      (int)std::max<long long>(1, std::min<long long>({s, blocks / kMinBlocks, kMaxSplitsSpan}));
  // Short rows (a warp of eight splits has eight blocks at most) wait on latencies, and three of
  // them are those of the parts through global memory: their CTAs are a cluster instead (e4m3,
  // 12 rows of eight heads, window 1000: 8.7 us against 12.5, 8000: 17.0 and 17.6, 16000: 26.1
  // and 21.0).  Up to 128 SMs' worth, which clusters of eight find room for at once.
  const int few = std::min(n, kClusterSplits);
  if (few > 1 && blocks <= few * shape.warps * 8 && rows * few <= 128LL * shape.ctas)
    return {few, true};
  return {n, false};
}

SpanChoice span_choice(const SpanParams& sp, bool narrow, int pages) {
  const SpanShape shape = span_shape(narrow, (long long)sp.p.B * sp.p.Hkv);
  const SpanSplits splits = span_splits(sp, shape, pages);
  return {splits.n, splits.cluster, kSms * shape.ctas};
}

size_t span_max_parts(int batch, int hkv, bool user) {
  const long long rows = (long long)batch * hkv;
  if (rows > kSplitRows) return 0;
  return user ? rows * kMaxSplitsSpan : std::min<long long>(rows * kMaxSplitsSpan, 4 * kSms);
}

// Where a narrow chain step selects: for MHA rows of at most 4096 pages whose CTAs are all
// resident, in the span decode's own CTAs (one launch less: 1K tokens and 4 heads 12.7 -> 11.2
// us), otherwise in a kernel of its own.
bool span_selects(const SpanParams& sp, int pages) {
  const long long rows = (long long)sp.p.B * sp.p.Hkv;
  const SpanShape shape = span_shape(true, rows);
  return sp.p.Hq == sp.p.Hkv && sp.p.max_pages <= 4096 &&
         rows * span_splits(sp, shape, pages).n <= (long long)kSms * shape.ctas;
}

cudaError_t launch_span(const SpanParams& sp, bool narrow, int pages, cudaStream_t s) {
  const long long rows = (long long)sp.p.B * sp.p.Hkv;
  const SpanShape shape = span_shape(narrow, rows);
  SpanParams pp = sp;
  const SpanSplits splits = span_splits(sp, shape, pages);
  pp.p.n_splits = splits.n;
  pp.cluster = splits.cluster ? 1 : 0;
  void* args[] = {&pp};
  const dim3 grid((unsigned)(rows * splits.n)), block(32 * shape.warps);
  const int together = splits.cluster ? splits.n : 1;
  if (!sp.p.chain_select) return launch_pdl(shape.fn, grid, block, 0, s, args, together);
  const void* fn = (const void*)span_kernel<true, 8, 2, 1, true>;
  const size_t smem = topk_smem_bytes(sp.p.max_pages) + 256 * 4 + (size_t)sp.p.top_k * 4;
  const cudaError_t e = ensure_smem(fn, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(fn, grid, block, smem, s, args, together);
}

}  // namespace quest
