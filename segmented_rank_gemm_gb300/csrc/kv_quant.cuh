// kv_quant.cuh -- a group of 16 values to its 4-bit codes and e4m3 scale (include/lora_kv.h: the
// 4-bit format), for the kernels that write the cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv_decode.cuh"
#include "kv_kernels.h"
#include "lora_common.cuh"

namespace lora {

__device__ __forceinline__ float e4m3_value(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// Codes of 16 values, pair j by get(j), whose quotients by s round to -7 .. 7, y = 1 / s correctly rounded.  The
// quotient is Markstein's: q = x y is corrected twice by its remainder, x - q s, exact in one
// fused multiply-add once q is within one unit in the last place, which makes the last result the
// correctly rounded x / s -- as a division, with one reciprocal for the group.  Adding
// 1.5 2^23 rounds to an integer, ties to even, and leaves it in the low bits; a shifted add
// puts it in its nibble, and what the sums carry besides is one constant.
template <bool IS_V, class Get>
__device__ __forceinline__ uint2 codes_of(const Get& get, float s, float y) {
  const float2 y2 = make_float2(y, y), minus_s = make_float2(-s, -s);
  const float2 magic = make_float2(12582912.f, 12582912.f);
  uint32_t code[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    code[h] = 0x11111111u * (8u - 0x4B400000u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = get(4 * h + j);
      float2 q = mul2(x, y2);
      q = fma2(fma2(q, minus_s, x), y2, q);
      q = fma2(fma2(q, minus_s, x), y2, q);
      q = add2(q, magic);
      code[h] += __float_as_uint(q.x) << (4 * kv_nibble(IS_V, 2 * j));
      code[h] += __float_as_uint(q.y) << (4 * kv_nibble(IS_V, 2 * j + 1));
    }
  }
  return make_uint2(code[0], code[1]);
}

// Writes a group, pair j by get(j), of a cache of scale g.  top: its largest magnitude but for NaN
// elements, of which there are some if `nan`.
template <bool IS_V, class Get>
__device__ __forceinline__ void write_codes(const Get& get, float top, bool nan, float g, uint8_t* codes,
                                            uint8_t* scale) {
  const uint8_t sb = static_cast<uint8_t>(
      __nv_cvt_float_to_fp8(__fdiv_rn(top, 7.f * g), __NV_SATFINITE, __NV_E4M3));
  const float s = e4m3_value(sb) * g;
  const float y = __frcp_rn(s);
  uint2 code;
  // (the range keeps every product and remainder of a quotient from a half up a normal number)
  if (!nan && s > 0x1p-60f && s < 0x1p60f && top * y < 7.49f) {
    code = codes_of<IS_V>(get, s, y);
  } else {  // zeros, saturated scales, the smallest scales, NaN: division and clamp by element
    code = make_uint2(0u, 0u);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = j & 1 ? get(j / 2).y : get(j / 2).x;
      float q = s > 0.f ? rintf(__fdiv_rn(x, s)) : 0.f;
      q = q != q ? 0.f : fminf(fmaxf(q, -7.f), 7.f);
      (j < 8 ? code.x : code.y) |= static_cast<uint32_t>(static_cast<int>(q) + 8)
                                   << (4 * kv_nibble(IS_V, j & 7));
    }
  }
  *reinterpret_cast<uint2*>(codes) = code;
  *scale = sb;
}

// Writes the group of bf16 pairs w.
template <bool IS_V>
__device__ __forceinline__ void write_group(const uint4 lo, const uint4 hi, float g, uint8_t* codes,
                                            uint8_t* scale) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  // the largest magnitude; a NaN if there is one
  __nv_bfloat162 top2 = __habs2(reinterpret_cast<const __nv_bfloat162&>(w[0]));
#pragma unroll
  for (int j = 1; j < 8; ++j)
    top2 = __hmax2_nan(top2, __habs2(reinterpret_cast<const __nv_bfloat162&>(w[j])));
  float top = __bfloat162float(__hmax_nan(top2.x, top2.y));
  const bool nan = top != top;
  if (nan) {
    top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[j])), fabsf(bf16_hi(w[j]))));
  }
  write_codes<IS_V>([&](int j) { return make_float2(bf16_lo(w[j]), bf16_hi(w[j])); }, top, nan, g, codes, scale);
}

// Writes the group of fp32 pairs x.
template <bool IS_V>
__device__ __forceinline__ void write_group(const float2 (&x)[8], float g, uint8_t* codes, uint8_t* scale) {
  float top = 0.f;  // a NaN if there is one
#pragma unroll
  for (int j = 0; j < 8; ++j) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(x[j].x), "f"(x[j].y));
  const bool nan = top != top;
  if (nan) {
    top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fmaxf(fabsf(x[j].x), fabsf(x[j].y)));
  }
  write_codes<IS_V>([&](int j) { return x[j]; }, top, nan, g, codes, scale);
}

}  // namespace lora
