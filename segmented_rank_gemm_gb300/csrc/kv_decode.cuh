// kv_decode.cuh -- the 4-bit cache's values in registers, and the small instructions the
// attention kernels share.
//
// Decoding, per pair of 4-bit codes n in two halves of a register: n OR the bits of 1024 gives
// 1024 + n (1024 + 16 n for the next code up), and one fused multiply-add
// (1024 + n) s - 1032 s = (n - 8) s, exact in fp16 because 1032 s = 8 129 s has at most 11
// significant bits.  One shift serves the two other codes of a half: 9 instructions for 8 codes.
// Values are scaled by 2^-5, which keeps 1032 s within fp16 (s <= 448) and n s exact (s is a
// multiple of 2^-9).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lora_common.cuh"

namespace lora {

constexpr float kKvUnit = 32.f;  // decoded values times this are the cache's (before its scale)

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// (a & mask) | bits, one instruction (written out: two immediates are else split in two).
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(bits));
  return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Each half of v twice.
__device__ __forceinline__ uint32_t both_lo(uint32_t v) { return prmt(v, v, 0x1010); }
__device__ __forceinline__ uint32_t both_hi(uint32_t v) { return prmt(v, v, 0x3232); }
// a * b + c of two floats at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// The scales of 4-bit codes, for a pair's low (s0, c0) and next (s1, c1) codes.
struct Decode {
  uint32_t s0, c0, s1, c1;
};
__device__ __forceinline__ Decode decode_scales(uint32_t s) {  // two e4m3 values as fp16
  Decode d;
  d.s0 = mul_f16x2(s, 0x28002800u);     // s 2^-5
  d.c0 = mul_f16x2(d.s0, 0xE408E408u);  // -1032 s 2^-5
  d.s1 = mul_f16x2(d.s0, 0x2C002C00u);  // s 2^-9
  d.c1 = mul_f16x2(d.s0, 0xD480D480u);  // -72 s 2^-5
  return d;
}
// The four pairs of codes of y: nibbles i of both halves.
__device__ __forceinline__ void decode4(uint32_t y, const Decode& d, uint32_t (&o)[4]) {
  const uint32_t y8 = y >> 8;
  o[0] = fma_f16x2(and_or(y, 0x000F000Fu, 0x64006400u), d.s0, d.c0);
  o[1] = fma_f16x2(and_or(y, 0x00F000F0u, 0x64006400u), d.s1, d.c1);
  o[2] = fma_f16x2(and_or(y8, 0x000F000Fu, 0x64006400u), d.s0, d.c0);
  o[3] = fma_f16x2(and_or(y8, 0x00F000F0u, 0x64006400u), d.s1, d.c1);
}
// The same with pairs 1 and 3 sixteen times as large, which spares a product a scale: their
// (1024 + 16 n) s - 1152 s = 16 (n - 8) s, exact too.
struct Decode16 {
  uint32_t s, c0, c1;
};
__device__ __forceinline__ Decode16 decode_scales16(uint32_t s) {
  Decode16 d;
  d.s = mul_f16x2(s, 0x28002800u);     // s 2^-5
  d.c0 = mul_f16x2(d.s, 0xE408E408u);  // -1032 s 2^-5
  d.c1 = mul_f16x2(d.s, 0xE480E480u);  // -1152 s 2^-5
  return d;
}
__device__ __forceinline__ void decode4(uint32_t y, const Decode16& d, uint32_t (&o)[4]) {
  const uint32_t y8 = y >> 8;
  o[0] = fma_f16x2(and_or(y, 0x000F000Fu, 0x64006400u), d.s, d.c0);
  o[1] = fma_f16x2(and_or(y, 0x00F000F0u, 0x64006400u), d.s, d.c1);
  o[2] = fma_f16x2(and_or(y8, 0x000F000Fu, 0x64006400u), d.s, d.c0);
  o[3] = fma_f16x2(and_or(y8, 0x00F000F0u, 0x64006400u), d.s, d.c1);
}
// The same in bf16 (7 bits of mantissa: 128 + n, one code a half at a time, 11 instructions for 8
// codes, in the cache's own unit): n s has at most 7 significant bits and 136 s = 8 17 s at most 8.
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
struct DecodeBf16 {
  uint32_t s, c;
};
// The scale in byte `at` of v (e4m3, not negative), times 2^-120 of `unit` (bf16 pair): its
// exponent and mantissa moved to bf16's places are its value times 2^-120.
__device__ __forceinline__ DecodeBf16 decode_scale_bf16(uint32_t v, int at, uint32_t unit) {
  DecodeBf16 d;
  d.s = mul_bf16x2(prmt(v, 0u, 0x4040u + 0x0101u * at) << 4, unit);
  d.c = mul_bf16x2(d.s, 0xC308C308u);  // -136 s
  return d;
}
__device__ __forceinline__ void decode4(uint32_t y, const DecodeBf16& d, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = fma_bf16x2(and_or(y >> (4 * i), 0x000F000Fu, 0x43004300u), d.s, d.c);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Whether a barrier's phase is complete, without waiting.  A wait, even for a phase long complete,
// takes about 160 cycles from its instruction to the branch on its result; asked for ahead of
// other work, the answer costs nothing.
__device__ __forceinline__ uint32_t mbar_peek(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done;
}

// Loads that stay behind the wait for the kernel before (a const or read-only load may be moved
// ahead of it).
__device__ __forceinline__ int32_t load_in_order(const int32_t* p) {
  int32_t r;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(r) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t load_in_order(const uint8_t* p) {
  uint32_t r;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(r) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ uint2 load_in_order(const uint2* p) {
  uint2 r;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ uint4 load_in_order(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// a / b of non-negative values, in 32 bits where they fit (a 64-bit division takes longer than a
// load from L2).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

}  // namespace lora
