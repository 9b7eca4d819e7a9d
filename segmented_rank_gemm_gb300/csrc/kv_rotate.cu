// kv_rotate.cu -- queries and keys turned by their positions, keys and values written to the
// 4-bit cache on the way (include/lora_kv.h: lora_kv_append_rotated).
//
// Per rotated pair of dimensions (a, b) and its angle's (c, s) = (cos, sin) at the row's position,
//     a' = a c - b s,   b' = b c + a s
// in fp32, every product and sum rounded by itself: the keys' codes are then the same wherever the
// same definition is computed, as their quotients are.  Queries are rounded to bf16; keys are
// quantised from fp32, without a rounding to bf16 between.
//
// Bound: bytes for large batches, the launch and two dependent loads (position, then angles) for
// small ones.  Work split: blocks of keys, of values and of queries in one launch.  A thread of keys
// or values takes two groups of 16 dimensions -- the two halves of 16 pairs where pairs are half a
// rotation apart, neighbours else -- so that a pair is loaded and its angle read once; a thread of
// queries takes 8 pairs of kQHeads heads, which share their angles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_decode.cuh"
#include "kv_kernels.h"
#include "kv_quant.cuh"
#include "lora_common.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kQHeads = 4;

// a b + c d of two floats at once.  The sums are scalar: packed ones are fused with the packed products
// before them, which spares the product's rounding (seen in results where the terms cancel).
__device__ __forceinline__ float2 sum_of_products(float2 a, float2 b, float2 c, float2 d) {
  const float2 x = mul2(a, b), y = mul2(c, d);
  return make_float2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}
__device__ __forceinline__ float2 bf16x2_values(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

// Words w0[i] and w1[i] (bf16 pairs) of N words turned to x0 and x1, with 2 N angles (c, s) at `at`.
// Apart: element e of w0 is paired with element e of w1; else a word is a pair, w0's angles first.
template <int N, bool APART>
__device__ __forceinline__ void turn(const uint32_t (&w0)[N], const uint32_t (&w1)[N], const float2* angles,
                                     float2 (&x0)[N], float2 (&x1)[N]) {
  float4 cs[N];
#pragma unroll
  for (int i = 0; i < N; ++i) cs[i] = __ldg(reinterpret_cast<const float4*>(angles) + i);
  if constexpr (APART) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 a = bf16x2_values(w0[i]), b = bf16x2_values(w1[i]);
      const float2 c = make_float2(cs[i].x, cs[i].z), s = make_float2(cs[i].y, cs[i].w);
      x0[i] = sum_of_products(a, c, b, make_float2(-s.x, -s.y));
      x1[i] = sum_of_products(b, c, a, s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
      const float2 ab = bf16x2_values(i < N ? w0[i % N] : w1[i % N]);
      const float c = i & 1 ? cs[i / 2].z : cs[i / 2].x, s = i & 1 ? cs[i / 2].w : cs[i / 2].y;
      const float2 y = sum_of_products(ab, make_float2(c, c), make_float2(ab.y, ab.x), make_float2(-s, s));
      if (i < N) x0[i % N] = y;
      else x1[i % N] = y;
    }
  }
}

__device__ __forceinline__ void load_words(const __nv_bfloat16* src, uint32_t (&w)[8]) {
  const uint4 a = load_in_order(reinterpret_cast<const uint4*>(src));
  const uint4 b = load_in_order(reinterpret_cast<const uint4*>(src) + 1);
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

// Two groups of 16 dimensions of one token and head of K or V, a thread.
template <int D, bool APART, bool IS_V>
__device__ __forceinline__ void write_pair(const KvRotateArgs& a, unsigned i) {
  constexpr unsigned kPairs = D / 32;
  const KvPages& pg = a.pages;
  const unsigned per = pg.heads * kPairs;  // of a token
  if (i >= a.T * per) return;
  const unsigned t = i / per, r = i - t * per;
  const int head = r / kPairs, p = r % kPairs;
  const int slot = load_in_order(a.slots + t), pos = load_in_order(a.position + t);
  const bool rotated = !IS_V && p * 32 < a.rotary;
  const int g0 = APART && rotated ? p : 2 * p, g1 = APART && rotated ? p + a.rotary / 32 : 2 * p + 1;
  const __nv_bfloat16* src = IS_V ? static_cast<const __nv_bfloat16*>(a.v) + static_cast<size_t>(t) * a.ldv
                                  : static_cast<const __nv_bfloat16*>(a.k) + static_cast<size_t>(t) * a.ldk;
  src += head * D;
  uint32_t w0[8], w1[8];
  load_words(src + g0 * 16, w0);
  load_words(src + g1 * 16, w1);
  const bool there = static_cast<unsigned>(slot) < static_cast<unsigned>(pg.num_pages) << pg.page_shift;
  const bool known = static_cast<unsigned>(pos) < static_cast<unsigned>(a.max_position);
  if (!there || !known) {
    if (r == 0 && !IS_V && ((!there && slot != -1) || !known)) atomicOr(a.err, LORA_ERRF_BAD_ID);
    return;
  }
  const int at = slot & ((1 << pg.page_shift) - 1), token = at & (kKvBlock - 1);
  uint8_t* const blk = pg.base + pg.block(slot >> pg.page_shift, head, at / kKvBlock);
  const auto codes = [&](int g) {
    return blk + (IS_V ? kv_v_code_at(D, token, g * 8) : kv_k_code_at(D, token, g * 8));
  };
  const auto scale = [&](int g) { return blk + (IS_V ? kv_v_scale_at(D, token, g) : kv_k_scale_at(D, token, g)); };
  if (rotated) {
    float2 x0[8], x1[8];
    turn<8, APART>(w0, w1, a.angles + static_cast<size_t>(pos) * (a.rotary / 2) + p * 16, x0, x1);
    write_group<IS_V>(x0, a.k_scale, codes(g0), scale(g0));
    write_group<IS_V>(x1, a.k_scale, codes(g1), scale(g1));
  } else {
    const float g = IS_V ? a.v_scale : a.k_scale;
    write_group<IS_V>(make_uint4(w0[0], w0[1], w0[2], w0[3]), make_uint4(w0[4], w0[5], w0[6], w0[7]), g,
                      codes(g0), scale(g0));
    write_group<IS_V>(make_uint4(w1[0], w1[1], w1[2], w1[3]), make_uint4(w1[4], w1[5], w1[6], w1[7]), g,
                      codes(g1), scale(g1));
  }
}

// 8 pairs (or 16 dimensions that are not turned) of up to kQHeads heads of one query row, a thread;
// a warp takes the row's dimensions and kQHeads * 32 / (D / 16) heads.
template <int D, bool APART>
__device__ __forceinline__ void turn_queries(const KvRotateArgs& a, unsigned i) {
  constexpr int kSlices = D / 16, kLanes = 32 / kSlices;
  const unsigned chunks = (a.q_heads + kQHeads * kLanes - 1) / (kQHeads * kLanes);
  const unsigned warp = i / 32, t = warp / chunks, lane = i % 32;
  if (t >= static_cast<unsigned>(a.T)) return;
  const int slice = lane % kSlices;
  const int head0 = (warp - t * chunks) * (kQHeads * kLanes) + lane / kSlices;
  const int pos = load_in_order(a.position + t);
  const bool rotated = slice * 16 < a.rotary;
  const int d0 = APART && rotated ? slice * 8 : slice * 16, d1 = APART && rotated ? d0 + a.rotary / 2 : d0 + 8;
  const __nv_bfloat16* const q = static_cast<const __nv_bfloat16*>(a.q) + static_cast<size_t>(t) * a.ldq;
  __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.q_out) + static_cast<size_t>(t) * a.ldqo;
  uint4 v0[kQHeads], v1[kQHeads];
#pragma unroll
  for (int h = 0; h < kQHeads; ++h) {
    const int head = head0 + h * kLanes;
    if (head >= a.q_heads) break;
    v0[h] = load_in_order(reinterpret_cast<const uint4*>(q + head * D + d0));
    v1[h] = load_in_order(reinterpret_cast<const uint4*>(q + head * D + d1));
  }
  if (static_cast<unsigned>(pos) >= static_cast<unsigned>(a.max_position)) {
    if (slice == 0 && head0 == 0) atomicOr(a.err, LORA_ERRF_BAD_ID);
    return;
  }
  const float2* const angles = a.angles + static_cast<size_t>(pos) * (a.rotary / 2) + slice * 8;
#pragma unroll
  for (int h = 0; h < kQHeads; ++h) {
    const int head = head0 + h * kLanes;
    if (head >= a.q_heads) break;
    if (rotated) {
      const uint32_t w0[4] = {v0[h].x, v0[h].y, v0[h].z, v0[h].w}, w1[4] = {v1[h].x, v1[h].y, v1[h].z, v1[h].w};
      float2 x0[4], x1[4];
      turn<4, APART>(w0, w1, angles, x0, x1);  // (the angles are loaded once: they are read-only)
      v0[h] = make_uint4(pack_bf16x2(x0[0].x, x0[0].y), pack_bf16x2(x0[1].x, x0[1].y),
                         pack_bf16x2(x0[2].x, x0[2].y), pack_bf16x2(x0[3].x, x0[3].y));
      v1[h] = make_uint4(pack_bf16x2(x1[0].x, x1[0].y), pack_bf16x2(x1[1].x, x1[1].y),
                         pack_bf16x2(x1[2].x, x1[2].y), pack_bf16x2(x1[3].x, x1[3].y));
    }
    *reinterpret_cast<uint4*>(out + head * D + d0) = v0[h];
    *reinterpret_cast<uint4*>(out + head * D + d1) = v1[h];
  }
}

// The kernel behind may start at once: it reads the cache and the queries behind its own wait.
template <int D, bool APART>
__global__ void __launch_bounds__(kThreads) kv_rotate_kernel(KvRotateArgs a, unsigned kv_blocks) {
  griddep_wait();
  griddep_launch_dependents();
  // the blocks of keys and values evenly among those of queries: how many of the former come before
  const unsigned long long n = 2 * kv_blocks;
  const unsigned before = static_cast<unsigned>(blockIdx.x * n / gridDim.x);
  if ((blockIdx.x + 1) * n / gridDim.x == before)
    turn_queries<D, APART>(a, (blockIdx.x - before) * kThreads + threadIdx.x);
  else if (before & 1)
    write_pair<D, APART, true>(a, (before >> 1) * kThreads + threadIdx.x);
  else
    write_pair<D, APART, false>(a, (before >> 1) * kThreads + threadIdx.x);
}

template <int D, bool APART>
cudaError_t launch(const KvRotateArgs& a, cudaStream_t stream) {
  const auto blocks = [](long long threads) { return static_cast<unsigned>((threads + kThreads - 1) / kThreads); };
  constexpr int kWarpHeads = kQHeads * 32 / (D / 16);
  const unsigned kv = blocks(static_cast<long long>(a.T) * a.pages.heads * (D / 32));
  const unsigned q = blocks(static_cast<long long>(a.T) * ((a.q_heads + kWarpHeads - 1) / kWarpHeads) * 32);
  return launch_dependent(kv_rotate_kernel<D, APART>, dim3(2 * kv + q), kThreads, 0, stream, a, kv);
}

}  // namespace

cudaError_t launch_kv_rotate(const KvRotateArgs& a, cudaStream_t stream) {
  if (a.pages.D == 128) return a.interleaved ? launch<128, false>(a, stream) : launch<128, true>(a, stream);
  return a.interleaved ? launch<64, false>(a, stream) : launch<64, true>(a, stream);
}

}  // namespace lora
