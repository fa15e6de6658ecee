// quest_narrow_kernels.cu - writing an 8-bit ("narrow") paged cache: chunks of a prompt and
// single tokens.
//
// A page of P tokens of one kv head becomes e4m3 once it is complete: with a = max |x| over
// its finite values, the scale is the smallest power of two s = 2^e with a <= 448 s (448 is
// the largest e4m3 number; s = 1 when a = 0) and the code of x is x / s rounded to the
// nearest e4m3 number, ties to even, infinities to +-448.  A power of two costs no precision
// in a floating format, makes x / s and code * s exact, and so makes the code a function
// of the page's values alone: a prompt in one call, in chunks or token by token gives the
// same bytes.  Until a page is complete its rows stay fp16 in the sequence's open page, so
// nothing is ever quantised twice.  K and V have scales of their own.  The page's box is
// formed from the fp16 keys ("Guide to Quest", Solution step 1), so that the selection is
// that of the fp16 cache.
//
// Bound by DRAM: a token and kv head is 512 B in and 256 B out.  One warp holds a page's K
// rows (then its V rows) in registers, so the maximum, the box and the codes take one read.
// Measured: the pages of a 32K prompt of 32 heads in 125 us (839 MB, 6.7 TB/s: the copy rate).
#include "quest_device.cuh"
#include "quest_narrow.cuh"

namespace quest {

namespace {

constexpr int kNarrowWarps = 4;
constexpr int kNarrowThreads = 32 * kNarrowWarps;

// The widest box seen so far of this lane's dims (8 of them, over the rows of a half-warp).
struct Box {
  __half2 mn[4], mx[4];
  bool any;
};

__device__ __forceinline__ void widen_box(Box& x, const uint4& row) {
  const uint32_t w[4] = {row.x, row.y, row.z, row.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x.mn[e] = x.any ? __hmin2(x.mn[e], as_h2(w[e])) : as_h2(w[e]);
    x.mx[e] = x.any ? __hmax2(x.mx[e], as_h2(w[e])) : as_h2(w[e]);
  }
  x.any = true;
}

// The two half-warps' boxes into one, and into the page's record (over what it holds when
// the page already had tokens).
__device__ __forceinline__ void store_box(const Params& p, Box& x, int b, int g, int page,
                                          bool had_tokens, int lane) {
  const int hw = lane >> 4, c = lane & 15;
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
  uint4* at = reinterpret_cast<uint4*>(p.meta + box_offset(p, b, g, page) + hw * kHeadDim + 8 * c);
  uint32_t w[4];
  const uint4 old = had_tokens ? *at : make_uint4(0u, 0u, 0u, 0u);
  const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    __half2 v = hw ? x.mx[e] : x.mn[e];
    if (had_tokens) v = hw ? __hmax2(v, as_h2(o[e])) : __hmin2(v, as_h2(o[e]));
    w[e] = as_u32(v);
  }
  *at = make_uint4(w[0], w[1], w[2], w[3]);
}

// One complete page of one kv head, one warp: rows [0, s0) from the open page, the rest
// from `in` (row stride `stride` halves).  Half-warp hw holds rows hw, hw + 2, ...; lane c
// dims [8c, 8c + 8).
template <int P>
__device__ __forceinline__ void load_rows(uint4 (&row)[P / 2], const __half* open,
                                          const __half* in, size_t stride, int s0, int hw, int c) {
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    const int t = hw + 2 * i;
    row[i] = t < s0 ? *reinterpret_cast<const uint4*>(open + t * kHeadDim + 8 * c)
                    : __ldcs(reinterpret_cast<const uint4*>(in + (size_t)(t - s0) * stride + 8 * c));
  }
}

template <int P>
__device__ __forceinline__ void encode_rows(const uint4 (&row)[P / 2], unsigned char* pool,
                                            float* scale, int lane) {
  const int hw = lane >> 4, c = lane & 15;
  const float s = page_scale<P>(row), inv = 1.f / s;  // both powers of two: exact
#pragma unroll
  for (int i = 0; i < P / 2; ++i)
    __stcs(reinterpret_cast<uint2*>(pool + (hw + 2 * i) * kHeadDim + 8 * c),
           make_uint2(encode4(row[i].x, row[i].y, inv), encode4(row[i].z, row[i].w, inv)));
  if (lane == 0) *scale = s;
}

template <int P>
__device__ __forceinline__ void encode_page(const Params& p, const NarrowPtrs& nar, int b, int g,
                                            int page, int phys, int s0, const __half* k,
                                            const __half* v, size_t stride, int lane) {
  const int hw = lane >> 4, c = lane & 15;
  const size_t open = ((size_t)b * p.Hkv + g) * P * kHeadDim;
  const size_t at = (size_t)phys * p.Hkv + g;
  uint4 row[P / 2];
  load_rows<P>(row, nar.k_open + open, k, stride, s0, hw, c);
  Box box;
  box.any = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) box.mn[e] = box.mx[e] = __float2half2_rn(0.f);
#pragma unroll
  for (int i = 0; i < P / 2; ++i)
    if (hw + 2 * i >= s0) widen_box(box, row[i]);
  encode_rows<P>(row, nar.k_pool + at * P * kHeadDim, nar.k_scale + at, lane);
  load_rows<P>(row, nar.v_open + open, v, stride, s0, hw, c);
  encode_rows<P>(row, nar.v_pool + at * P * kHeadDim, nar.v_scale + at, lane);
  store_box(p, box, b, g, page, s0 > 0, lane);
}

// Rows [s0, e) of the open page from `k` / `v`, and the page's box; one warp.
template <int P>
__device__ __forceinline__ void fill_open(const Params& p, const NarrowPtrs& nar, int b, int g,
                                          int page, int s0, int e, const __half* k,
                                          const __half* v, size_t stride, int lane) {
  const int hw = lane >> 4, c = lane & 15;
  const size_t open = ((size_t)b * p.Hkv + g) * P * kHeadDim + 8 * c;
  Box box;
  box.any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) box.mn[i] = box.mx[i] = __float2half2_rn(0.f);
  constexpr int R = 4;  // rows of a half-warp on their way together
#pragma unroll 1
  for (int tb = s0 + hw; tb < e; tb += 2 * R) {
    uint4 kk[R], vv[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const size_t at = (size_t)(min(tb + 2 * i, e - 1) - s0) * stride + 8 * c;
      kk[i] = *reinterpret_cast<const uint4*>(k + at);
      vv[i] = *reinterpret_cast<const uint4*>(v + at);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = tb + 2 * i;
      if (t < e) {
        *reinterpret_cast<uint4*>(nar.k_open + open + t * kHeadDim) = kk[i];
        *reinterpret_cast<uint4*>(nar.v_open + open + t * kHeadDim) = vv[i];
        widen_box(box, kk[i]);
      }
    }
  }
  store_box(p, box, b, g, page, s0 > 0, lane);
}

// The complete pages of a chunk: grid (ceil(Hkv / 4), pages a chunk can complete, B), block
// (z, j, b): logical page L / P + j of sequence b, warp w its kv head 4z + w.  Heads vary
// fastest, so that the blocks in flight read whole token rows of the chunk.
template <int P>
__global__ void __launch_bounds__(kNarrowThreads) narrow_pages_kernel(Params p, NarrowPtrs nar,
                                                                      const __half* k,
                                                                      const __half* v, int n) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, lane = threadIdx.x & 31;
  const int g = blockIdx.x * kNarrowWarps + (threadIdx.x >> 5);
  const int L = p.seq_lens[b];
  if (L < 0 || (long long)L + n > (long long)p.max_pages * P) return;  // the open kernel reports
  const int page = L / P + (int)blockIdx.y;
  if ((long long)(page + 1) * P > (long long)L + n || g >= p.Hkv) return;  // warp-uniform
  const int phys = p.block_table[(size_t)b * p.max_pages + page];
  if (phys < 0 || phys >= p.num_phys) return;
  const int s0 = max(0, L - page * P);
  // The open page becomes complete: not where the chunk meets an unmapped page.  (Asked of the
  // first page alone, and by the block index: by s0 every block paid, 155 us for the 32K prompt's
  // 150.)
  if (blockIdx.y == 0 && s0 > 0) {
    const int last = (L + n - 1) / P;
    bool bad = false;
#pragma unroll 8
    for (int pg = page + lane; pg <= last; pg += 32) {
      const int at = p.block_table[(size_t)b * p.max_pages + pg];
      bad |= at < 0 || at >= p.num_phys;
    }
    if (__any_sync(0xffffffffu, bad)) return;
  }
  const size_t stride = (size_t)p.Hkv * kHeadDim;
  const size_t in = ((size_t)b * n + (page * P + s0 - L)) * stride + (size_t)g * kHeadDim;
  encode_page<P>(p, nar, b, g, page, phys, s0, k + in, v + in, stride, lane);
}

// What a chunk leaves in the open page, then the lengths: grid (ceil(Hkv / 4), B).  Every
// block of a sequence checks the block-table entries of the touched pages itself (a chunk
// that does not fit, or that meets an unmapped page, leaves the open page and the length
// alone); the last block of the sequence advances its length.
template <int P>
__global__ void __launch_bounds__(kNarrowThreads) narrow_open_kernel(Params p, NarrowPtrs nar,
                                                                     const __half* k,
                                                                     const __half* v, int n) {
  __shared__ int s_flag;
  pdl_wait();  // before any read: the lengths and the table may be an earlier call's work
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int g = blockIdx.x * kNarrowWarps + (threadIdx.x >> 5);
  const int L = p.seq_lens[b];
  const bool fits = L >= 0 && (long long)L + n <= (long long)p.max_pages * P;
  int bad = -1;  // a touched page that is not mapped
  if (fits) {
    const int last = (L + n - 1) / P;
    const int* table = p.block_table + (size_t)b * p.max_pages;
    // eight entries a thread on their way together (one at a time, a 32K prompt's 2048 entries
    // took 10 us)
    for (int pg = L / P + (int)threadIdx.x; pg <= last; pg += 8 * kNarrowThreads) {
      int phys[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) phys[i] = table[min(pg + i * kNarrowThreads, last)];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (phys[i] < 0 || phys[i] >= p.num_phys) bad = min(pg + i * kNarrowThreads, last);
    }
    if (bad >= 0 && blockIdx.x == 0) report(p, QUEST_ERR_BAD_PAGE, b, bad, kSiteAppend);
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    report(p, QUEST_ERR_BAD_LENGTH, b, -1, kSiteAppend);
  }
  const bool ok = fits && !__syncthreads_or(bad >= 0);
  const int e = ok ? (L + n) % P : 0;
  if (e > 0 && g < p.Hkv) {
    const int page = (L + n) / P;
    const int s0 = max(0, L - page * P);
    const size_t stride = (size_t)p.Hkv * kHeadDim;
    const size_t in = ((size_t)b * n + (page * P + s0 - L)) * stride + (size_t)g * kHeadDim;
    fill_open<P>(p, nar, b, g, page, s0, e, k + in, v + in, stride, lane);
  }
  if (arrive_last<kNarrowThreads, false>(&p.seq_done[b], gridDim.x, &s_flag) &&
      threadIdx.x == 0) {
    p.seq_done[b] = 0u;
    if (ok) p.seq_lens[b] = L + n;
  }
}

// One token per sequence: grid (ceil(Hkv / 4), B).  The token that completes its page takes
// the page's other rows from the open page and encodes it; any other joins the open page.
template <int P>
__global__ void __launch_bounds__(kNarrowThreads) narrow_append_kernel(Params p, NarrowPtrs nar,
                                                                       const __half* k_new,
                                                                       const __half* v_new) {
  __shared__ int s_flag;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int g = blockIdx.x * kNarrowWarps + (threadIdx.x >> 5);
  const int L = p.seq_lens[b];
  bool ok = L >= 0 && (long long)L + 1 <= (long long)p.max_pages * P;
  int phys = -1;
  if (!ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(p, QUEST_ERR_BAD_LENGTH, b, -1, kSiteAppend);
  } else {
    phys = p.block_table[(size_t)b * p.max_pages + L / P];
    if (phys < 0 || phys >= p.num_phys) {
      if (blockIdx.x == 0 && threadIdx.x == 0)
        report(p, QUEST_ERR_BAD_PAGE, b, L / P, kSiteAppend);
      ok = false;
    }
  }
  if (ok && g < p.Hkv) {
    const int slot = L % P;
    const size_t in = ((size_t)b * p.Hkv + g) * kHeadDim;
    if (slot == P - 1)
      encode_page<P>(p, nar, b, g, L / P, phys, slot, k_new + in, v_new + in, 0, lane);
    else
      fill_open<P>(p, nar, b, g, L / P, slot, slot + 1, k_new + in, v_new + in, 0, lane);
  }
  if (arrive_last<kNarrowThreads, false>(&p.seq_done[b], gridDim.x, &s_flag) &&
      threadIdx.x == 0) {
    p.seq_done[b] = 0u;
    if (ok) p.seq_lens[b] = L + 1;
  }
}

// The page bounds of a decode step that appends: the estimate (as quest_estimate's, boxes
// through L2), whose CTA that has the new token's page first lets a warp write the token and
// its box, so that the step needs no launch of its own for them.  grid (scoring tiles, B * Hkv).
// The lengths stay: every kernel of the step sees the token (chain_append), the last one
// advances them.
template <int G, int P>
__global__ void __launch_bounds__(kConsumerThreads) narrow_estimate_kernel(Params p,
                                                                           NarrowPtrs nar) {
  pdl_wait();
  const int tile = blockIdx.x, bg = blockIdx.y, b = bg / p.Hkv, g = bg % p.Hkv;
  bool appended = false;
  const int L = load_len_step(p, b, kSiteScore, &appended);
  const int N = (L + P - 1) / P;
  const int p0 = tile * p.score_tile_pages;
  const int np = min(p.score_tile_pages, p.max_pages - p0);
  const int n_live = max(0, min(N - p0, np));
  float* row = p.scores + (size_t)bg * p.max_pages + p0;
  for (int i = n_live + (int)threadIdx.x; i < np; i += blockDim.x) row[i] = -CUDART_INF_F;
  if (!appended) {
    if ((long long)L == (long long)p.max_pages * P && tile == 0 && g == 0 && threadIdx.x == 0)
      report(p, QUEST_ERR_BAD_LENGTH, b, -1, kSiteAppend);  // no room for the new token
  } else {
    const int page = (L - 1) / P, slot = (L - 1) % P;
    if (page >= p0 && page < p0 + n_live) {  // block-uniform
      if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int phys = p.block_table[(size_t)b * p.max_pages + page];
        const size_t in = ((size_t)b * p.Hkv + g) * kHeadDim;
        if (phys < 0 || phys >= p.num_phys) {
          if (lane == 0) report(p, QUEST_ERR_BAD_PAGE, b, page, kSiteAppend);
        } else if (slot == P - 1) {
          encode_page<P>(p, nar, b, g, page, phys, slot, p.k_new + in, p.v_new + in, 0, lane);
        } else {
          fill_open<P>(p, nar, b, g, page, slot, slot + 1, p.k_new + in, p.v_new + in, 0, lane);
        }
      }
      __syncthreads();
    }
  }
  if (n_live > 0) score_tile<G, false, true>(p, b, g, p0, n_live, row, (size_t)p.max_pages);
}

template <int P>
const void* narrow_estimate_fn(int G) {
  switch (G) {
    case 1: return (const void*)narrow_estimate_kernel<1, P>;
    case 2: return (const void*)narrow_estimate_kernel<2, P>;
    case 4: return (const void*)narrow_estimate_kernel<4, P>;
    default: return (const void*)narrow_estimate_kernel<8, P>;
  }
}

}  // namespace

cudaError_t launch_narrow_estimate(const Params& p, const NarrowPtrs& nar, int G,
                                   cudaStream_t s) {
  Params pp = p;
  NarrowPtrs np = nar;
  void* args[] = {&pp, &np};
  return launch_pdl(p.P == 16 ? narrow_estimate_fn<16>(G) : narrow_estimate_fn<32>(G),
                    dim3(p.n_score_tiles, p.B * p.Hkv), dim3(kConsumerThreads), 0, s, args);
}

cudaError_t launch_narrow_prefill(const Params& p, const NarrowPtrs& nar, const __half* k,
                                  const __half* v, int n, cudaStream_t s) {
  Params pp = p;
  NarrowPtrs np = nar;
  void* args[] = {&pp, &np, &k, &v, &n};
  const unsigned heads = (unsigned)((p.Hkv + kNarrowWarps - 1) / kNarrowWarps);
  const void* pages = p.P == 16 ? (const void*)narrow_pages_kernel<16>
                                : (const void*)narrow_pages_kernel<32>;
  const void* open = p.P == 16 ? (const void*)narrow_open_kernel<16>
                               : (const void*)narrow_open_kernel<32>;
  const unsigned most = (unsigned)((n + p.P - 1) / p.P);  // L % P + n < (most + 1) P
  cudaError_t e = launch_pdl(pages, dim3(heads, most, p.B), dim3(kNarrowThreads), 0, s, args);
  if (e != cudaSuccess) return e;
  return launch_pdl(open, dim3(heads, p.B), dim3(kNarrowThreads), 0, s, args);
}

cudaError_t launch_narrow_append(const Params& p, const NarrowPtrs& nar, const __half* k_new,
                                 const __half* v_new, cudaStream_t s) {
  Params pp = p;
  NarrowPtrs np = nar;
  void* args[] = {&pp, &np, &k_new, &v_new};
  const unsigned heads = (unsigned)((p.Hkv + kNarrowWarps - 1) / kNarrowWarps);
  const void* fn = p.P == 16 ? (const void*)narrow_append_kernel<16>
                             : (const void*)narrow_append_kernel<32>;
  return launch_pdl(fn, dim3(heads, p.B), dim3(kNarrowThreads), 0, s, args);
}

}  // namespace quest
