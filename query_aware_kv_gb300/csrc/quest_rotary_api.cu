// quest_rotary_api.cu - the C entry points of rotary positions (declared in include/quest.h):
// the frequencies' fixed-point form, argument checks and dispatch.  No call allocates memory or
// synchronises.
#include <cmath>
#include <cstdio>

#include "quest_internal.h"

using namespace quest;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int bad(const char* message) { return set_last_error(QUEST_ERR_INVALID_ARG, message); }

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return QUEST_OK;
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return set_last_error(QUEST_ERR_CUDA, msg);
}

bool rotary_dim_ok(int d) { return d >= 8 && d <= kHeadDim && d % 8 == 0; }

int check_rope(const quest_rope_t* rope) {
  if (!rope) return bad("rope is NULL");
  if (!rotary_dim_ok(rope->rotary_dim) || (rope->interleaved & ~1) ||
      !std::isfinite(rope->magnitude) || !std::isfinite(rope->magnitude_low))
    return bad("rope: not filled by quest_rope_init");
  return QUEST_OK;
}

bool strides_ok(const int64_t* s) { return s[0] % 8 == 0 && s[1] % 8 == 0; }

// The checks of a write beside those of its cache.
int check_write(const quest_rope_t* rope, const quest_rotary_io_t* io, int batch, int max_pages,
                int page_size, bool* nothing) {
  *nothing = false;
  int rc = check_rope(rope);
  if (rc) return rc;
  if (!io) return bad("io is NULL");
  if (io->dtype != QUEST_FP16 && io->dtype != QUEST_BF16)
    return bad("dtype must be QUEST_FP16 or QUEST_BF16");
  if (io->n_tokens < 0) return bad("n_tokens must be >= 0");
  if (batch == 0 || io->n_tokens == 0) {
    *nothing = true;
    return QUEST_OK;
  }
  if ((long long)io->n_tokens > (long long)max_pages * page_size)
    return bad("n_tokens exceeds max_pages * page_size");
  if (!io->k || !io->v || !aligned(io->k, 16) || !aligned(io->v, 16))
    return bad("k / v must be non-NULL and 16-byte aligned");
  if (!io->q != !io->q_out) return bad("q and q_out go together");
  if (!aligned(io->q, 16) || !aligned(io->q_out, 16)) return bad("q / q_out must be 16-byte aligned");
  if (!strides_ok(io->k_stride) || !strides_ok(io->v_stride) || (io->q && !strides_ok(io->q_stride)))
    return bad("strides must be multiples of 8 elements");
  if (!aligned(io->position_offsets, 4)) return bad("position_offsets must be 4-byte aligned");
  return QUEST_OK;
}

}  // namespace

extern "C" {

int quest_rope_init(quest_rope_t* rope, int32_t rotary_dim, int32_t interleaved,
                    const double* inv_freq, double magnitude) {
  if (!rope || !inv_freq) return bad("rope / inv_freq is NULL");
  if (!rotary_dim_ok(rotary_dim)) return bad("rotary_dim must be 8, 16, ..., 128");
  if (interleaved & ~1) return bad("interleaved must be 0 or 1");
  if (!std::isfinite((float)magnitude)) return bad("magnitude must be finite");
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!(std::fabs(inv_freq[i]) <= 1e6)) return bad("inv_freq must be finite and at most 1e6");
  *rope = quest_rope_t{};
  rope->rotary_dim = rotary_dim;
  rope->interleaved = interleaved;
  rope->magnitude = (float)magnitude;
  rope->magnitude_low = (float)(magnitude - (double)rope->magnitude);
  // 1 / (2 pi) as the sum of two doubles; the product with f as hi + lo, its whole turns dropped
  const double r_hi = 0x1.45f306dc9c883p-3, r_lo = -0x1.6b01ec5417056p-57;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::fabs(inv_freq[i]), hi = f * r_hi;
    const double lo = std::fma(f, r_hi, -hi) + f * r_lo;
    const double x = std::ldexp(hi - std::floor(hi), 64);  // below 2^64, and exact
    const uint64_t whole = (uint64_t)x;
    const uint64_t turns =
        whole + (uint64_t)(int64_t)std::llrint(x - (double)whole + std::ldexp(lo, 64));
    rope->turns[i] = inv_freq[i] < 0 ? 0u - turns : turns;
  }
  return QUEST_OK;
}

int quest_rotate(const quest_rope_t* rope, const void* x, int64_t x_stride,
                 const int32_t* positions, int32_t n_tokens, int32_t num_heads, int32_t dtype,
                 int32_t transposed, void* out, int64_t out_stride, quest_stream_t stream) {
  const int rc = check_rope(rope);
  if (rc) return rc;
  if (dtype < QUEST_FP16 || dtype > QUEST_FP32)
    return bad("dtype must be QUEST_FP16, QUEST_BF16 or QUEST_FP32");
  if (n_tokens < 0 || num_heads < 1) return bad("n_tokens must be >= 0 and num_heads >= 1");
  if (transposed & ~1) return bad("transposed must be 0 or 1");
  if (n_tokens == 0) return QUEST_OK;
  if (!x || !out || !aligned(x, 16) || !aligned(out, 16))
    return bad("x / out must be non-NULL and 16-byte aligned");
  if (!positions || !aligned(positions, 4)) return bad("positions must be non-NULL and 4-byte aligned");
  if (x_stride % 8 || out_stride % 8) return bad("strides must be multiples of 8 elements");
  if (n_tokens > 1 && out_stride < (int64_t)num_heads * kHeadDim)
    return bad("out_stride must be at least num_heads * 128");
  if (n_tokens > 1 && x == out && x_stride != out_stride)
    return bad("in place, x and out need the same stride");
  if ((long long)n_tokens * num_heads > 0x7fffffffLL * 8) return bad("too many rows");
  const RotateCall r{rope, x, out, positions, x_stride, out_stride, n_tokens, num_heads, dtype,
                     transposed};
  return launched(launch_rotate(r, static_cast<cudaStream_t>(stream)), "quest_rotate");
}

int quest_prefill_rotary(const quest_cache_t* cache, const quest_rope_t* rope,
                         const quest_rotary_io_t* io, void* ws, size_t ws_bytes,
                         quest_stream_t stream) {
  int rc = check_cache_desc(cache);
  if (rc) return rc;
  bool nothing;
  if ((rc = check_write(rope, io, cache->batch, cache->max_pages, cache->page_size, &nothing)) ||
      nothing)
    return rc;
  if ((rc = check_workspace(ws, ws_bytes, sizeof(WsHeader)))) return rc;
  Params p{};
  p.B = cache->batch;
  p.Hq = cache->num_q_heads;
  p.Hkv = cache->num_kv_heads;
  p.P = cache->page_size;
  p.max_pages = cache->max_pages;
  p.num_phys = cache->num_phys;
  p.k_pool = static_cast<__half*>(cache->k_pool);
  p.v_pool = static_cast<__half*>(cache->v_pool);
  p.meta = static_cast<__half*>(cache->meta);
  p.block_table = cache->block_table;
  p.seq_lens = cache->seq_lens;
  p.status = &static_cast<WsHeader*>(ws)->status;
  return launched(launch_rotary_write(p, nullptr, *rope, *io, static_cast<cudaStream_t>(stream)),
                  "quest_prefill_rotary");
}

int quest_narrow_prefill_rotary(const quest_narrow_cache_t* cache, const quest_rope_t* rope,
                                const quest_rotary_io_t* io, void* ws, size_t ws_bytes,
                                quest_stream_t stream) {
  int rc = check_narrow_desc(cache);
  if (rc) return rc;
  bool nothing;
  if ((rc = check_write(rope, io, cache->batch, cache->max_pages, cache->page_size, &nothing)) ||
      nothing)
    return rc;
  Params p{};
  NarrowPtrs nar{};
  if ((rc = narrow_write_params(cache, ws, ws_bytes, &p, &nar))) return rc;
  return launched(launch_rotary_write(p, &nar, *rope, *io, static_cast<cudaStream_t>(stream)),
                  "quest_narrow_prefill_rotary");
}

}  // extern "C"
