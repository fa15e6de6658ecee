// quest_rotary_kernels.cu - rotary positions: heads turned by their tokens' positions, alone or
// on the way into a paged cache.
//
// A head's first rotary_dim dims are pairs (x_a, x_b); the pair i of the token at position t is
// turned by the angle t f_i:
//   y_a = m (x_a cos - x_b sin),   y_b = m (x_b cos + x_a sin)
// with pairs (i, i + rotary_dim / 2) or (2i, 2i + 1); the other dims pass through.
//
// Angles: f_i comes as a fraction of a turn in 2^-64 units, so t f_i mod 1 is one 64-bit integer
// product whose overflow drops the whole turns exactly, at any 32-bit position.  Its upper 32
// bits (an angle within 2^-32 of a turn, 1.5e-9) lose their quarter turns, the rest goes through
// polynomials whose sums have two parts; the turn itself is in fp32, rounded once to the output's
// type.
//
// Bound by DRAM: a value costs its read and its write, and 3 flops.  Measured: 8192 tokens of 40
// fp16 heads out of rows of 48 in 27 us (168 MB, 6.3 TB/s), 1999 tokens of 24 bf16 heads in 4.2 (25
// MB), 4 tokens in 2.2, which is the launch and two round trips (calls of a graph, one after another).  A half-warp takes a row of
// 128 dims, lane c two pieces of 4 dims whose four pairs are whole within the lane for either
// layout (rotary_dim is a multiple of 8), so nothing is exchanged between lanes.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "quest_device.cuh"
#include "quest_narrow.cuh"

namespace quest {

namespace {

// ---- types: four values of a row
template <class T> struct Four;
template <> struct Four<__half> {
  typedef uint2 raw;
  static __device__ __forceinline__ void get(const raw& r, float (&x)[4]) {
    const float2 a = h2f(r.x), b = h2f(r.y);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  }
  static __device__ __forceinline__ raw put(const float (&x)[4]) {
    return make_uint2(as_u32(__floats2half2_rn(x[0], x[1])), as_u32(__floats2half2_rn(x[2], x[3])));
  }
};
template <> struct Four<__nv_bfloat16> {
  typedef uint2 raw;
  static __device__ __forceinline__ void get(const raw& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x << 16); x[1] = __uint_as_float(r.x & 0xffff0000u);
    x[2] = __uint_as_float(r.y << 16); x[3] = __uint_as_float(r.y & 0xffff0000u);
  }
  static __device__ __forceinline__ raw put(const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};
template <> struct Four<float> {
  typedef float4 raw;
  static __device__ __forceinline__ void get(const raw& r, float (&x)[4]) {
    x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
  }
  static __device__ __forceinline__ raw put(const float (&x)[4]) {
    return make_float4(x[0], x[1], x[2], x[3]);
  }
};

// ---- the turn of a position
// m cos and m sin of the angle, the two at half a unit in the last place and little more: what is lost
// beside the last rounding is kept as a second fp32 number up to it (a cosine that is off by twice as
// much moves twice as many of the turned values to the neighbour of the right fp16 number).
__device__ __forceinline__ void cos_sin(const quest_rope_t& rope, int i, long long pos, float& c,
                                        float& s) {
  // (a product modulo 2^64 is the same for signed and unsigned factors)
  const uint32_t at = (uint32_t)(rope.turns[i] * (uint64_t)pos >> 32);
  // the nearest quarter turn and the rest, within an eighth of a turn, as r + r_low half turns
  const uint32_t quarter = at + 0x20000000u >> 30;
  const int rest = (int)(at - (quarter << 30));
  const float r = (float)rest * 0x1p-31f, r_low = (float)(rest - (int)(float)rest) * 0x1p-31f;
  const float u = r * r, u_low = fmaf(2.f * r, r_low, fmaf(r, r, -u));
  // sin(pi r) = r (pi + u A(u)) and cos(pi r) = 1 + u (B0 + u B(u)): A and B0 + u B interpolated at
  // the Chebyshev nodes of [0, 1/16]; pi and B0 in two parts, the other coefficients in fp32, with
  // which the sine is within 1.4e-9 and the cosine within 2.2e-10.  (sincospif,
  // which reduces its argument once more, made a block's table its longest part.)
  constexpr float kPi = 0x1.921fb6p+1f, kPiLow = -0x1.777a5cp-24f;
  constexpr float kB0 = -0x1.3bd3ccp+2f, kB0Low = -0x1.313d3p-23f;
  float a = fmaf(0x1.4cb762p-4f, u, -0x1.32ce1ep-1f);
  a = fmaf(a, u, 0x1.466bc2p+1f);
  a = fmaf(a, u, -0x1.4abbcep+2f);
  a = fmaf(a, u, kPiLow);
  const float p = r * kPi;
  const float p_low = fmaf(r, a, fmaf(r_low, kPi, fmaf(r, kPi, -p)));
  float b = fmaf(0x1.db6492p-3f, u, -0x1.55cb98p+0f);
  b = fmaf(b, u, 0x1.03c1eap+2f);
  const float t = u * kB0, q = 1.f + t;
  const float q_low =
      fmaf(u, fmaf(b, u, kB0Low), fmaf(u_low, kB0, fmaf(u, kB0, -t))) + ((1.f - q) + t);
  const float m = rope.magnitude, m_low = rope.magnitude_low;
  const float sine = fmaf(p, m, fmaf(p, m_low, p_low * m));
  const float cosine = fmaf(q, m, fmaf(q, m_low, q_low * m));
  const float x = quarter & 1u ? sine : cosine, y = quarter & 1u ? cosine : sine;
  c = quarter + 1u & 2u ? -x : x;
  s = quarter & 2u ? -y : y;
}

// Lane c's two pieces (offsets in dims), and whether they are turned.
struct Pieces {
  int a, b;
  bool turned;
};
__device__ __forceinline__ Pieces pieces(const quest_rope_t& rope, int c) {
  const int rd = rope.rotary_dim;
  Pieces x;
  x.turned = 8 * c < rd;
  const bool halves = x.turned && !rope.interleaved;
  x.a = halves ? 4 * c : 8 * c;
  x.b = halves ? rd / 2 + 4 * c : 8 * c + 4;
  return x;
}

// The lane's four pairs, turned.  cs: cosines and sines of pairs 4c .. 4c + 3.
template <bool kInter>
__device__ __forceinline__ void turn(float (&a)[4], float (&b)[4], const float2 (&cs)[4]) {
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
      a[2 * i] = fmaf(x, cs[i].x, -y * cs[i].y);
      a[2 * i + 1] = fmaf(y, cs[i].x, x * cs[i].y);
      b[2 * i] = fmaf(z, cs[2 + i].x, -w * cs[2 + i].y);
      b[2 * i + 1] = fmaf(w, cs[2 + i].x, z * cs[2 + i].y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[i], y = b[i];
      a[i] = fmaf(x, cs[i].x, -y * cs[i].y);
      b[i] = fmaf(y, cs[i].x, x * cs[i].y);
    }
  }
}
__device__ __forceinline__ void turn(bool inter, float (&a)[4], float (&b)[4], const float2 (&cs)[4]) {
  if (inter) turn<true>(a, b, cs);
  else turn<false>(a, b, cs);
}

// ------------------------------------------------------------------------------------
// rotate: heads [tokens][heads][128], out of place or in place.  A half-warp takes `per`
// heads of one token: the cosines and sines are taken once for all of them.
// ------------------------------------------------------------------------------------
struct RotateParams {
  quest_rope_t rope;
  const void* x;
  void* out;
  const int* positions;
  long long x_stride, out_stride;  // elements a token
  long long units;                 // tokens * groups of heads
  int heads, groups, per;
  int transposed;
};
constexpr int kRotateThreads = 128;

template <class T>
__global__ void __launch_bounds__(kRotateThreads) rotate_kernel(
    const __grid_constant__ RotateParams r) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane & 15;
  const long long unit = (long long)blockIdx.x * (kRotateThreads / 16) + (threadIdx.x >> 4);
  if (unit >= r.units) return;
  const long long t = unit / r.groups;
  const int h0 = (int)(unit % r.groups) * r.per, h1 = min(r.heads, h0 + r.per);
  typedef typename Four<T>::raw raw;
  const Pieces at = pieces(r.rope, c);
  const T* x = static_cast<const T*>(r.x) + t * r.x_stride;
  T* out = static_cast<T*>(r.out) + t * r.out_stride;
  const int pos = r.positions[t];
  constexpr int R = 4;  // rows on their way together
  raw p[R], z[R];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const T* row = x + (size_t)min(h + i, h1 - 1) * kHeadDim;
      p[i] = *reinterpret_cast<const raw*>(row + at.a);
      z[i] = *reinterpret_cast<const raw*>(row + at.b);
    }
  };
  load(h0);  // (beside the position and its cosines)
  float2 cs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = make_float2(1.f, 0.f);
    if (at.turned) cos_sin(r.rope, 4 * c + i, pos, cs[i].x, cs[i].y);
    if (r.transposed) cs[i].y = -cs[i].y;
  }
#pragma unroll 1
  for (int h = h0; h < h1; h += R) {
    if (h > h0) load(h);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (h + i >= h1) break;
      if (at.turned) {
        float a[4], b[4];
        Four<T>::get(p[i], a);
        Four<T>::get(z[i], b);
        turn(r.rope.interleaved != 0, a, b, cs);
        p[i] = Four<T>::put(a);
        z[i] = Four<T>::put(b);
      }
      T* row = out + (size_t)(h + i) * kHeadDim;
      *reinterpret_cast<raw*>(row + at.a) = p[i];
      *reinterpret_cast<raw*>(row + at.b) = z[i];
    }
  }
}

// ------------------------------------------------------------------------------------
// writes into a cache
// ------------------------------------------------------------------------------------
// Four 16-bit values of the source type as four halves, unchanged or turned.
template <class T>
__device__ __forceinline__ uint2 to_half(uint2 r) {
  if constexpr (sizeof(T) == 2 && !std::is_same<T, __half>::value) {
    float x[4];
    Four<T>::get(r, x);
    return Four<__half>::put(x);
  }
  return r;
}
template <class T>
__device__ __forceinline__ void turn_row(const Pieces& at, bool inter, const float2* table, uint2& p,
                                         uint2& z) {
  if (at.turned) {
    float2 cs[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 two = *reinterpret_cast<const float4*>(table + 2 * i);
      cs[2 * i] = make_float2(two.x, two.y);
      cs[2 * i + 1] = make_float2(two.z, two.w);
    }
    float a[4], b[4];
    Four<T>::get(p, a);
    Four<T>::get(z, b);
    turn(inter, a, b, cs);
    p = Four<__half>::put(a);
    z = Four<__half>::put(b);
  } else {
    p = to_half<T>(p);
    z = to_half<T>(z);
  }
}
// Eight values of a V row.
template <class T>
__device__ __forceinline__ uint4 to_half8(const uint4& r) {
  const uint2 a = to_half<T>(make_uint2(r.x, r.y)), b = to_half<T>(make_uint2(r.z, r.w));
  return make_uint4(a.x, a.y, b.x, b.y);
}

// Cosines and sines of `rows` positions from `pos`, [row][64]: every thread one pair's of every
// (threads / 64)-th row.
template <int NT>
__device__ __forceinline__ void fill_table(const quest_rope_t& rope, long long pos, int rows,
                                           float2 (*table)[64]) {
  const int i = threadIdx.x & 63;
  if (i < rope.rotary_dim / 2) {
    for (int r = threadIdx.x >> 6; r < rows; r += NT / 64) {
      float c, s;
      cos_sin(rope, i, pos + r, c, s);
      table[r][i] = make_float2(c, s);
    }
  }
}

// The box of a lane's pieces over the rows seen so far (minima and maxima of packed halves are
// exact).
struct PieceBox {
  __half2 mn[4], mx[4];
  bool any;
};
__device__ __forceinline__ void clear(PieceBox& x) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x.mn[e] = x.mx[e] = __float2half2_rn(0.f);
  x.any = false;
}
__device__ __forceinline__ void widen(PieceBox& x, const uint2& p, const uint2& z) {
  const uint32_t w[4] = {p.x, p.y, z.x, z.y};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x.mn[e] = x.any ? __hmin2(x.mn[e], as_h2(w[e])) : as_h2(w[e]);
    x.mx[e] = x.any ? __hmax2(x.mx[e], as_h2(w[e])) : as_h2(w[e]);
  }
  x.any = true;
}
// Both half-warps' boxes into the page's record: replaced, or widened where the page had tokens.
__device__ __forceinline__ void store_box(const Params& p, PieceBox& x, const Pieces& at, int b,
                                          int g, int page, bool had_tokens, int hw) {
  const bool other = __shfl_xor_sync(0xffffffffu, x.any ? 1 : 0, 16) != 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 mn = as_h2(__shfl_xor_sync(0xffffffffu, as_u32(x.mn[e]), 16));
    const __half2 mx = as_h2(__shfl_xor_sync(0xffffffffu, as_u32(x.mx[e]), 16));
    if (other) {
      x.mn[e] = x.any ? __hmin2(x.mn[e], mn) : mn;
      x.mx[e] = x.any ? __hmax2(x.mx[e], mx) : mx;
    }
  }
  __half* row = p.meta + box_offset(p, b, g, page) + hw * kHeadDim;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint2* to = reinterpret_cast<uint2*>(row + (e ? at.b : at.a));
    __half2 v0 = hw ? x.mx[2 * e] : x.mn[2 * e], v1 = hw ? x.mx[2 * e + 1] : x.mn[2 * e + 1];
    if (had_tokens) {
      const uint2 old = *to;
      v0 = hw ? __hmax2(v0, as_h2(old.x)) : __hmin2(v0, as_h2(old.x));
      v1 = hw ? __hmax2(v1, as_h2(old.y)) : __hmin2(v1, as_h2(old.y));
    }
    *to = make_uint2(as_u32(v0), as_u32(v1));
  }
}

struct WriteParams {
  Params p;
  NarrowPtrs nar;  // narrow caches only
  quest_rope_t rope;
  const void* q;   // null: not turned
  const void* k;
  const void* v;
  long long q_seq, q_tok, k_seq, k_tok, v_seq, v_tok;  // strides in elements
  __half* q_out;
  const int* offsets;  // per sequence, or null
  int n;
};

constexpr int kWriteWarps = 4;
constexpr int kWriteThreads = 32 * kWriteWarps;
constexpr int kQHeads = 2 * kWriteWarps;  // query heads of a block

// Rows [r0, r1) of a page (tokens t0 + r) from a K-like source, turned: to `out` (row stride
// `out_row`), and into the box where there is one.  One warp; half-warp hw takes every second row,
// eight of them on their way together.
template <class T, bool kBox>
__device__ __forceinline__ void turn_rows(const T* in, long long in_tok, __half* out, size_t out_row,
                                          int rows, const Pieces& at, bool inter,
                                          const float2 (*table)[64], int lane, PieceBox& box) {
  const int hw = lane >> 4, c = lane & 15;
  constexpr int R = 8;
#pragma unroll 1
  for (int r0 = hw; r0 < rows; r0 += 2 * R) {
    uint2 p[R], z[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const T* row = in + min(r0 + 2 * i, rows - 1) * in_tok;
      p[i] = __ldcs(reinterpret_cast<const uint2*>(row + at.a));
      z[i] = __ldcs(reinterpret_cast<const uint2*>(row + at.b));
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = r0 + 2 * i;
      if (r < rows) {
        turn_row<T>(at, inter, &table[r][4 * c], p[i], z[i]);
        *reinterpret_cast<uint2*>(out + r * out_row + at.a) = p[i];
        *reinterpret_cast<uint2*>(out + r * out_row + at.b) = z[i];
        if constexpr (kBox) widen(box, p[i], z[i]);
      }
    }
  }
}
// Rows of 128 16-bit values on their way to L2 (while the block makes its table).
template <class T>
__device__ __forceinline__ void prefetch_rows(const T* in, long long in_tok, int rows, int lane) {
  for (int i = lane; i < 2 * rows; i += 32)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(in + (i >> 1) * in_tok + (i & 1) * 64));
}
template <class T>
__device__ __forceinline__ void copy_rows(const T* in, long long in_tok, __half* out, int rows,
                                          int lane) {
  const int hw = lane >> 4, c = lane & 15;
  constexpr int R = 8;
#pragma unroll 1
  for (int r0 = hw; r0 < rows; r0 += 2 * R) {
    uint4 x[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      x[i] = __ldcs(reinterpret_cast<const uint4*>(in + min(r0 + 2 * i, rows - 1) * in_tok + 8 * c));
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (r0 + 2 * i < rows)
        *reinterpret_cast<uint4*>(out + (r0 + 2 * i) * kHeadDim + 8 * c) = to_half8<T>(x[i]);
  }
}

// ---- chunks.  grid (blocks of kv heads, then blocks of query heads; pages a chunk can touch; B):
// block (x, j, b) has logical page L / P + j of sequence b.  In the first columns warp w writes
// the page's new tokens of kv head 4x + w (keys turned, values, box); in the others it turns two
// query heads of the same tokens.  The block's cosines and sines are a table in shared memory: a
// position's 64 pairs are taken once for its four (eight) heads.  (Blocks of a head a
// warp, or of eight warps, fill more tables and more waves: 519 tokens of four sequences into a
// narrow cache took 18 and 19 us instead of 14.)
// Measured: 32K tokens of 32 query and 32 kv heads 245 us (1.64 GB, 6.7 TB/s).
template <class T, int P>
__device__ __forceinline__ void queries(const WriteParams& w, int b, int h0, int t0, int t1, int L,
                                        const Pieces& at, const float2 (*table)[64], int lane) {
  const Params& p = w.p;
  PieceBox none;
  for (int h = h0; h < min(h0 + 2, p.Hq); ++h)
    turn_rows<T, false>(static_cast<const T*>(w.q) + b * w.q_seq + (t0 - L) * w.q_tok + h * kHeadDim,
                        w.q_tok, w.q_out + (((size_t)b * w.n + (t0 - L)) * p.Hq + h) * kHeadDim,
                        (size_t)p.Hq * kHeadDim, t1 - t0, at, w.rope.interleaved != 0, table, lane,
                        none);
}

// What a warp of a block reads of tokens [t0, t1): its kv head's keys and values, or its queries.
// (Of pages of 16 tokens: 32K tokens of 32 heads 245 us for 250.  Twice as much a block is too much at
// once: 271 for 253 at 32 tokens; and the narrow pages' kernel took 276 for 256 and 317 for 286.)
template <class T>
__device__ __forceinline__ void prefetch_tokens(const WriteParams& w, int b, int t0, int t1, int L,
                                                int kv_blocks, int warp, int lane) {
  if ((int)blockIdx.x >= kv_blocks) {
    const int h0 = ((int)blockIdx.x - kv_blocks) * kQHeads + 2 * warp;
    for (int h = h0; h < min(h0 + 2, w.p.Hq); ++h)
      prefetch_rows(static_cast<const T*>(w.q) + b * w.q_seq + (t0 - L) * w.q_tok + h * kHeadDim,
                    w.q_tok, t1 - t0, lane);
  } else if (const int g = (int)blockIdx.x * kWriteWarps + warp; g < w.p.Hkv) {
    prefetch_rows(static_cast<const T*>(w.k) + b * w.k_seq + (t0 - L) * w.k_tok + g * kHeadDim,
                  w.k_tok, t1 - t0, lane);
    prefetch_rows(static_cast<const T*>(w.v) + b * w.v_seq + (t0 - L) * w.v_tok + g * kHeadDim,
                  w.v_tok, t1 - t0, lane);
  }
}

template <class T, int P>
__global__ void __launch_bounds__(kWriteThreads) rotary_prefill_kernel(
    const __grid_constant__ WriteParams w) {
  __shared__ __align__(16) float2 table[P][64];
  pdl_wait();
  const Params& p = w.p;
  const int b = blockIdx.z, n = w.n;
  const int kv_blocks = (p.Hkv + kWriteWarps - 1) / kWriteWarps;
  const int L = p.seq_lens[b];
  if (L < 0 || (long long)L + n > (long long)p.max_pages * P) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
      report(p, QUEST_ERR_BAD_LENGTH, b, -1, kSiteAppend);
    return;
  }
  const int page = L / P + (int)blockIdx.y;
  const int t0 = max(page * P, L), t1 = min(page * P + P, L + n);  // new tokens of this page
  if (t0 >= t1) return;  // (all of these are the block's)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hw = lane >> 4;
  if constexpr (P == 16) prefetch_tokens<T>(w, b, t0, t1, L, kv_blocks, warp, lane);
  fill_table<kWriteThreads>(w.rope, (long long)t0 + (w.offsets ? w.offsets[b] : 0), t1 - t0, table);
  __syncthreads();
  const Pieces at = pieces(w.rope, lane & 15);
  if ((int)blockIdx.x >= kv_blocks) {
    queries<T, P>(w, b, ((int)blockIdx.x - kv_blocks) * kQHeads + 2 * warp, t0, t1, L, at, table,
                  lane);
    return;
  }
  const int g = (int)blockIdx.x * kWriteWarps + warp;
  if (g >= p.Hkv) return;
  const int phys = p.block_table[(size_t)b * p.max_pages + page];
  if (phys < 0 || phys >= p.num_phys) {
    if (lane == 0 && g == 0) report(p, QUEST_ERR_BAD_PAGE, b, page, kSiteAppend);
    return;
  }
  const size_t to = (((size_t)phys * p.Hkv + g) * P + (t0 - page * P)) * kHeadDim;
  PieceBox box;
  clear(box);
  turn_rows<T, true>(static_cast<const T*>(w.k) + b * w.k_seq + (t0 - L) * w.k_tok + g * kHeadDim,
                     w.k_tok, p.k_pool + to, kHeadDim, t1 - t0, at, w.rope.interleaved != 0, table,
                     lane, box);
  copy_rows<T>(static_cast<const T*>(w.v) + b * w.v_seq + (t0 - L) * w.v_tok + g * kHeadDim, w.v_tok,
               p.v_pool + to, t1 - t0, lane);
  store_box(p, box, at, b, g, page, page * P < L, hw);
}

// One complete page of a narrow cache, one warp: rows [0, s0) from the open page, the others from
// the chunk (a narrow page's scale needs all of its rows, so they stay in registers).  `k` and `v`
// point to the first new row of the page.
template <class T, int P>
__device__ __forceinline__ void turn_page(const WriteParams& w, int b, int g, int page, int phys,
                                          int s0, const T* k, const T* v, const Pieces& at,
                                          const float2 (*table)[64], int lane) {
  const Params& p = w.p;
  const int hw = lane >> 4, c = lane & 15;
  const size_t open = ((size_t)b * p.Hkv + g) * P * kHeadDim;
  const size_t to = (size_t)phys * p.Hkv + g;
  uint4 row[P / 2];
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    const int t = hw + 2 * i;
    uint2 x, z;
    if (t < s0) {
      x = *reinterpret_cast<const uint2*>(w.nar.k_open + open + t * kHeadDim + at.a);
      z = *reinterpret_cast<const uint2*>(w.nar.k_open + open + t * kHeadDim + at.b);
    } else {
      x = __ldcs(reinterpret_cast<const uint2*>(k + (t - s0) * w.k_tok + at.a));
      z = __ldcs(reinterpret_cast<const uint2*>(k + (t - s0) * w.k_tok + at.b));
    }
    row[i] = make_uint4(x.x, x.y, z.x, z.y);
  }
  PieceBox box;
  clear(box);
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    const int t = hw + 2 * i;
    if (t >= s0) {
      uint2 x = make_uint2(row[i].x, row[i].y), z = make_uint2(row[i].z, row[i].w);
      turn_row<T>(at, w.rope.interleaved != 0, &table[t - s0][4 * c], x, z);
      row[i] = make_uint4(x.x, x.y, z.x, z.y);
      widen(box, x, z);
    }
  }
  {
    const float s = page_scale<P>(row), inv = 1.f / s;  // both powers of two: exact
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      unsigned char* code = w.nar.k_pool + (to * P + hw + 2 * i) * kHeadDim;
      *reinterpret_cast<uint32_t*>(code + at.a) = encode4(row[i].x, row[i].y, inv);
      *reinterpret_cast<uint32_t*>(code + at.b) = encode4(row[i].z, row[i].w, inv);
    }
    if (lane == 0) w.nar.k_scale[to] = s;
  }
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    const int t = hw + 2 * i;
    row[i] = t < s0 ? *reinterpret_cast<const uint4*>(w.nar.v_open + open + t * kHeadDim + 8 * c)
                    : to_half8<T>(__ldcs(reinterpret_cast<const uint4*>(v + (t - s0) * w.v_tok + 8 * c)));
  }
  {
    const float s = page_scale<P>(row), inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < P / 2; ++i)
      *reinterpret_cast<uint2*>(w.nar.v_pool + (to * P + hw + 2 * i) * kHeadDim + 8 * c) =
          make_uint2(encode4(row[i].x, row[i].y, inv), encode4(row[i].z, row[i].w, inv));
    if (lane == 0) w.nar.v_scale[to] = s;
  }
  store_box(p, box, at, b, g, page, s0 > 0, hw);
}

// A chunk into a narrow cache; grid as above.  The blocks of the first page also write what the chunk
// leaves in the open page: they alone read its old rows, which the page that the chunk completes
// takes first.  A chunk that does not fit, or that meets an unmapped page, leaves the open page and
// its box alone (the launch that advances the lengths finds the same).
//
// Registers are bounded for warps' sake: 32K tokens of 32 kv heads take 170 us so at page size 16 and
// 182 at 32, whose warps hold 32 rows.  With cosines in one part these were 163 and 176, then 169 at the
// compiler's 96 registers, and 177 and 211 in blocks of eight warps, four for the keys and four for the
// values.  (Without the turn 134 and 141: the rest is its instructions, between the loads of a page and
// its stores.)
template <class T, int P>
__global__ void __launch_bounds__(kWriteThreads, P == 16 ? 7 : 4) rotary_pages_kernel(
    const __grid_constant__ WriteParams w) {
  __shared__ __align__(16) float2 table[P][64];
  pdl_wait();
  const Params& p = w.p;
  const int b = blockIdx.z, n = w.n;
  const int kv_blocks = (p.Hkv + kWriteWarps - 1) / kWriteWarps;
  const int L = p.seq_lens[b];
  if (L < 0 || (long long)L + n > (long long)p.max_pages * P) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
      report(p, QUEST_ERR_BAD_LENGTH, b, -1, kSiteAppend);
    return;
  }
  const int page = L / P + (int)blockIdx.y;
  const int t0 = max(page * P, L), t1 = min(page * P + P, L + n);
  const bool for_q = (int)blockIdx.x >= kv_blocks;
  const bool whole = t1 == page * P + P;
  const int e = blockIdx.y == 0 && !for_q ? (L + n) % P : 0;  // rows that the chunk leaves open
  if (t0 >= t1 || (!for_q && !whole && e == 0)) return;  // (the block's)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long shift = w.offsets ? w.offsets[b] : 0;
  const Pieces at = pieces(w.rope, lane & 15);
  if (for_q || whole) fill_table<kWriteThreads>(w.rope, t0 + shift, t1 - t0, table);
  __syncthreads();
  if (for_q) {
    queries<T, P>(w, b, ((int)blockIdx.x - kv_blocks) * kQHeads + 2 * warp, t0, t1, L, at, table,
                  lane);
    return;
  }
  const int g = (int)blockIdx.x * kWriteWarps + warp, s0 = t0 - page * P;
  bool bad = false;
  if (e > 0 || (blockIdx.y == 0 && s0 > 0)) {  // the open page: every touched page has to be mapped
    const int last = (L + n - 1) / P;
#pragma unroll 8
    for (int pg = page + lane; pg <= last; pg += 32) {
      const int entry = p.block_table[(size_t)b * p.max_pages + pg];
      bad |= entry < 0 || entry >= p.num_phys;
    }
    bad = __any_sync(0xffffffffu, bad);
  }
  if (whole && g < p.Hkv) {
    const int phys = p.block_table[(size_t)b * p.max_pages + page];
    const bool mapped = phys >= 0 && phys < p.num_phys;
    if (!mapped && g == 0 && lane == 0) report(p, QUEST_ERR_BAD_PAGE, b, page, kSiteAppend);
    if (mapped && !(bad && s0 > 0))
      turn_page<T, P>(w, b, g, page, phys, s0,
                      static_cast<const T*>(w.k) + b * w.k_seq + (t0 - L) * w.k_tok + g * kHeadDim,
                      static_cast<const T*>(w.v) + b * w.v_seq + (t0 - L) * w.v_tok + g * kHeadDim,
                      at, table, lane);
  }
  if (e == 0) return;  // (the block's)
  const int open = (L + n) / P, o0 = max(open * P, L), r0 = o0 - open * P;
  __syncthreads();  // the table, and the open page's old rows, have been read
  fill_table<kWriteThreads>(w.rope, o0 + shift, e - r0, table);
  __syncthreads();
  if (g >= p.Hkv) return;
  if (bad) {
    const int phys = p.block_table[(size_t)b * p.max_pages + open];
    if ((phys < 0 || phys >= p.num_phys) && g == 0 && lane == 0)
      report(p, QUEST_ERR_BAD_PAGE, b, open, kSiteAppend);
    return;
  }
  const size_t to = (((size_t)b * p.Hkv + g) * P + r0) * kHeadDim;
  PieceBox box;
  clear(box);
  turn_rows<T, true>(static_cast<const T*>(w.k) + b * w.k_seq + (o0 - L) * w.k_tok + g * kHeadDim,
                     w.k_tok, w.nar.k_open + to, kHeadDim, e - r0, at, w.rope.interleaved != 0, table,
                     lane, box);
  copy_rows<T>(static_cast<const T*>(w.v) + b * w.v_seq + (o0 - L) * w.v_tok + g * kHeadDim, w.v_tok,
               w.nar.v_open + to, e - r0, lane);
  store_box(p, box, at, b, g, open, r0 > 0, lane >> 4);
}

// ---- one token per sequence: a block per sequence, a half-warp a row (keys with their boxes,
// values, queries).  The token that completes a narrow page takes the page's other rows from the
// open page, a warp per kv head.
constexpr int kAppendThreads = 512;

template <class T, int P, bool kNarrow>
__global__ void __launch_bounds__(kAppendThreads) rotary_append_kernel(
    const __grid_constant__ WriteParams w) {
  __shared__ __align__(16) float2 table[1][64];
  const Params& p = w.p;
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 15;
  const bool inter = w.rope.interleaved != 0;
  const Pieces at = pieces(w.rope, c);
  pdl_wait();
  pdl_trigger();  // the decode that follows may start its prologue
  const T* k = static_cast<const T*>(w.k) + b * w.k_seq;
  const T* v = static_cast<const T*>(w.v) + b * w.v_seq;
  // A half-warp's row u: a key, a value, or a query; the first is on its way beside the length, the
  // length beside the table entry, and every thread looks both up itself: nobody waits for a barrier.
  const int kv = 2 * p.Hkv, rows = kv + (w.q ? p.Hq : 0);
  auto source = [&](int u) {
    return u < p.Hkv ? k + u * kHeadDim
           : u < kv  ? v + (u - p.Hkv) * kHeadDim
                     : static_cast<const T*>(w.q) + b * w.q_seq + (u - kv) * kHeadDim;
  };
  uint2 x = make_uint2(0u, 0u), z = x;
  auto load = [&](int u) {
    x = *reinterpret_cast<const uint2*>(source(u) + at.a);
    z = *reinterpret_cast<const uint2*>(source(u) + at.b);
  };
  int u = threadIdx.x >> 4;
  if (u < rows) load(u);
  const int L = p.seq_lens[b];
  const int offset = w.offsets ? w.offsets[b] : 0;
  const bool fits = L >= 0 && (long long)L + 1 <= (long long)p.max_pages * P;
  const int page = fits ? L / P : 0, slot = fits ? L % P : 0;
  const int phys = p.block_table[(size_t)b * p.max_pages + page];
  const bool mapped = phys >= 0 && phys < p.num_phys;
  if (!fits || !mapped) {  // (the block's)
    if (threadIdx.x == 0)
      report(p, fits ? QUEST_ERR_BAD_PAGE : QUEST_ERR_BAD_LENGTH, b, fits ? page : -1, kSiteAppend);
    return;
  }
  const bool whole = kNarrow && slot == P - 1;
  if constexpr (kNarrow) {
    if (whole) {
      fill_table<kAppendThreads>(w.rope, (long long)L + offset, 1, table);
      __syncthreads();
      for (int g = warp; g < p.Hkv; g += kAppendThreads / 32)
        turn_page<T, P>(w, b, g, page, phys, slot, k + g * kHeadDim, v + g * kHeadDim, at, table, lane);
    }
  }
  float2 cs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at.turned)
      cos_sin(w.rope, 4 * c + i, (long long)L + offset, cs[i].x, cs[i].y);
#pragma unroll 1
  for (; u < rows; u += kAppendThreads / 16) {
    const bool is_k = u < p.Hkv, is_v = !is_k && u < kv;
    const int h = is_k ? u : is_v ? u - p.Hkv : u - kv;
    __half* to = w.q_out + ((size_t)b * p.Hq + h) * kHeadDim;
    if (is_k || is_v) {
      const size_t at_kv = (((size_t)(kNarrow ? b : phys) * p.Hkv + h) * P + slot) * kHeadDim;
      if constexpr (kNarrow) to = (is_k ? w.nar.k_open : w.nar.v_open) + at_kv;
      else to = (is_k ? p.k_pool : p.v_pool) + at_kv;
    }
    if (!(whole && (is_k || is_v))) {
      if (at.turned && !is_v) {
        float a[4], e[4];
        Four<T>::get(x, a);
        Four<T>::get(z, e);
        turn(inter, a, e, cs);
        x = Four<__half>::put(a);
        z = Four<__half>::put(e);
      } else {
        x = to_half<T>(x);
        z = to_half<T>(z);
      }
      *reinterpret_cast<uint2*>(to + at.a) = x;
      *reinterpret_cast<uint2*>(to + at.b) = z;
      if (is_k) {
        __half* box = p.meta + box_offset(p, b, h, page);
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // (minimum, maximum) x (piece a, piece b)
          uint2* at_box = reinterpret_cast<uint2*>(box + (e >> 1) * kHeadDim + ((e & 1) ? at.b : at.a));
          uint2 mine = (e & 1) ? z : x;
          if (slot != 0) {
            const uint2 old = *at_box;
            mine = (e >> 1) ? make_uint2(as_u32(__hmax2(as_h2(mine.x), as_h2(old.x))),
                                         as_u32(__hmax2(as_h2(mine.y), as_h2(old.y))))
                            : make_uint2(as_u32(__hmin2(as_h2(mine.x), as_h2(old.x))),
                                         as_u32(__hmin2(as_h2(mine.y), as_h2(old.y))));
          }
          *at_box = mine;
        }
      }
    }
    if (u + kAppendThreads / 16 < rows) load(u + kAppendThreads / 16);
  }
  __syncthreads();  // (every thread has read the length)
  if (threadIdx.x == 0) p.seq_lens[b] = L + 1;
}

template <class T, int P>
cudaError_t write(const WriteParams& w, bool narrow, cudaStream_t s) {
  WriteParams ww = w;
  void* args[] = {&ww};
  const Params& p = w.p;
  if (w.n == 1) {
    const void* fn = narrow ? (const void*)rotary_append_kernel<T, P, true>
                            : (const void*)rotary_append_kernel<T, P, false>;
    return launch_pdl(fn, dim3(p.B), dim3(kAppendThreads), 0, s, args);
  }
  const unsigned heads = (unsigned)((p.Hkv + kWriteWarps - 1) / kWriteWarps);
  const unsigned q_blocks = w.q ? (unsigned)((p.Hq + kQHeads - 1) / kQHeads) : 0u;
  const unsigned pages = (unsigned)((w.n + P - 1) / P + 1);
  const dim3 grid(heads + q_blocks, pages, p.B), block(kWriteThreads);
  const void* fn = narrow ? (const void*)rotary_pages_kernel<T, P>
                          : (const void*)rotary_prefill_kernel<T, P>;
  const cudaError_t e = launch_pdl(fn, grid, block, 0, s, args);
  return e == cudaSuccess ? launch_advance_lengths(p, w.n, s) : e;
}

}  // namespace

cudaError_t launch_rotate(const RotateCall& r, cudaStream_t s) {
  RotateParams p{};
  p.rope = *r.rope;
  p.x = r.x;
  p.out = r.out;
  p.positions = r.positions;
  p.x_stride = r.x_stride;
  p.out_stride = r.out_stride;
  p.heads = r.heads;
  p.transposed = r.transposed;
  // Eight heads a half-warp share a position's cosines (8192 tokens of 40 heads: 28.1 us, 33 at four,
  // 56 at two; 1999 tokens of 24: 4.8, 5.1 and 7.7); few rows take two, for their latency (4 tokens of
  // 32 heads: 3.5 us at eight, 3.1 at two).
  p.per = (long long)r.tokens * r.heads >= 16384 ? 8 : 2;
  p.groups = (r.heads + p.per - 1) / p.per;
  p.units = (long long)r.tokens * p.groups;
  void* args[] = {&p};
  const void* fn = r.dtype == QUEST_FP16   ? (const void*)rotate_kernel<__half>
                   : r.dtype == QUEST_BF16 ? (const void*)rotate_kernel<__nv_bfloat16>
                                           : (const void*)rotate_kernel<float>;
  constexpr int per_block = kRotateThreads / 16;
  return launch_pdl(fn, dim3((unsigned)((p.units + per_block - 1) / per_block)), dim3(kRotateThreads),
                    0, s, args);
}

cudaError_t launch_rotary_write(const Params& p, const NarrowPtrs* nar, const quest_rope_t& rope,
                                const quest_rotary_io_t& io, cudaStream_t s) {
  WriteParams w{};
  w.p = p;
  if (nar) w.nar = *nar;
  w.rope = rope;
  w.q = io.q;
  w.k = io.k;
  w.v = io.v;
  w.q_seq = io.q_stride[0];
  w.q_tok = io.q_stride[1];
  w.k_seq = io.k_stride[0];
  w.k_tok = io.k_stride[1];
  w.v_seq = io.v_stride[0];
  w.v_tok = io.v_stride[1];
  w.q_out = static_cast<__half*>(io.q_out);
  w.offsets = io.position_offsets;
  w.n = io.n_tokens;
  if (io.dtype == QUEST_FP16)
    return p.P == 16 ? write<__half, 16>(w, nar != nullptr, s) : write<__half, 32>(w, nar != nullptr, s);
  return p.P == 16 ? write<__nv_bfloat16, 16>(w, nar != nullptr, s)
                   : write<__nv_bfloat16, 32>(w, nar != nullptr, s);
}

}  // namespace quest
