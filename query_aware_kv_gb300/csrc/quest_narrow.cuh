// quest_narrow.cuh - the encoding of an 8-bit page, shared by the kernels that write one.
#pragma once

#include "quest_device.cuh"

namespace quest {

__device__ __forceinline__ __half2 as_h2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// The scale of a page whose largest finite magnitude is `top` (a widened fp16 number, so
// never subnormal in fp32): 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_of(float top) {
  if (top == 0.f) return 1.f;
  const uint32_t bits = __float_as_uint(top);
  const uint32_t e = (bits >> 23) - 8u + ((bits & 0x7fffffu) > 0x600000u ? 1u : 0u);
  return __uint_as_float(e << 23);
}

// Four halves (two words) times inv, as four e4m3 codes.
__device__ __forceinline__ uint32_t encode4(uint32_t a, uint32_t b, float inv) {
  const float2 x = __half22float2(as_h2(a)), y = __half22float2(as_h2(b));
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(x.x * inv), "f"(x.y * inv), "f"(y.x * inv), "f"(y.y * inv));
  return r;
}

// The scale of a page whose rows a warp holds (half-warp hw the rows hw, hw + 2, ..., 8 halves a
// lane of each).
template <int P>
__device__ __forceinline__ float page_scale(const uint4 (&row)[P / 2]) {
  __half2 top = __float2half2_rn(0.f);
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    top = __hmax2(top, __hmax2(__hmax2(__habs2(as_h2(row[i].x)), __habs2(as_h2(row[i].y))),
                               __hmax2(__habs2(as_h2(row[i].z)), __habs2(as_h2(row[i].w)))));
  }
  float a = warp_max(fmaxf(__low2float(top), __high2float(top)));
  if (isinf(a)) {  // an infinity among the values: the finite ones set the scale
    a = 0.f;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const uint32_t w[4] = {row[i].x, row[i].y, row[i].z, row[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = __half22float2(__habs2(as_h2(w[e])));
        if (v.x < CUDART_INF_F) a = fmaxf(a, v.x);
        if (v.y < CUDART_INF_F) a = fmaxf(a, v.y);
      }
    }
    a = warp_max(a);
  }
  return scale_of(a);
}

}  // namespace quest
