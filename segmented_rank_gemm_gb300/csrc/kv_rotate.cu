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
// small ones.  Work split: blocks of keys, of values and of queries in one launch, evenly among one
// another as the former are bound by instructions and the latter by bytes.  A thread of keys or values
// takes a group of 16 dimensions, a thread of queries 8 pairs of kQHeads heads, which share angles.
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
constexpr int kCtasPerSm = 4;

// a b + c d of two floats at once.  The sums are scalar: packed ones are fused with the packed products
// before them, which spares the product's rounding (seen in results where the terms cancel).
__device__ __forceinline__ float2 sum_of_products(float2 a, float2 b, float2 c, float2 d) {
  const float2 x = mul2(a, b), y = mul2(c, d);
  return make_float2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}
__device__ __forceinline__ float2 bf16x2_values(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

// Word i of two pairs' first elements a and second ones b, turned by two angles (c, s, c, s).
__device__ __forceinline__ float2 turned_a(uint32_t a, uint32_t b, const float4& cs) {
  return sum_of_products(bf16x2_values(a), make_float2(cs.x, cs.z), bf16x2_values(b), make_float2(-cs.y, -cs.w));
}
__device__ __forceinline__ float2 turned_b(uint32_t a, uint32_t b, const float4& cs) {
  return sum_of_products(bf16x2_values(b), make_float2(cs.x, cs.z), bf16x2_values(a), make_float2(cs.y, cs.w));
}
// A word that is a pair, turned by (c, s).
__device__ __forceinline__ float2 turned_pair(uint32_t w, float c, float s) {
  const float2 ab = bf16x2_values(w);
  return sum_of_products(ab, make_float2(c, c), make_float2(ab.y, ab.x), make_float2(-s, s));
}

// Two angles from another lane.  A row's angles are loaded once by the lanes of a warp, a piece (two of
// them) each, and exchanged where they are used: loaded by each thread, 64 or 128 bytes a lane, they
// took three quarters of the L1's cycles (8192 rows of 32 and 8 heads of 128 38 us, 31 exchanged).
__device__ __forceinline__ float4 from_lane(const float4& v, int lane) {
  return make_float4(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane),
                     __shfl_sync(0xffffffffu, v.z, lane), __shfl_sync(0xffffffffu, v.w, lane));
}
__device__ __forceinline__ float4 load_piece(const float2* row, int i) {
  return __ldg(reinterpret_cast<const float4*>(row) + i);
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A group of 16 dimensions of one token and head of K or V, a thread.  Keys: the pairs' other elements,
// where they are in another group, come from the lane that has it.
template <int D, bool APART, bool IS_V>
__device__ __forceinline__ void write_one(const KvRotateArgs& a, unsigned i, unsigned ahead) {
  constexpr unsigned kGroups = D / 16;
  const KvPages& pg = a.pages;
  const unsigned per = pg.heads * kGroups;  // of a token
  const bool some = i < a.T * per;
  if (i + ahead < a.T * per && (i & 3) == 0) {  // a line of a block to come
    const unsigned t = (i + ahead) / per, e = (i + ahead - t * per) * 16;
    prefetch_l2(IS_V ? static_cast<const __nv_bfloat16*>(a.v) + static_cast<size_t>(t) * a.ldv + e
                     : static_cast<const __nv_bfloat16*>(a.k) + static_cast<size_t>(t) * a.ldk + e);
  }
  if (!some) i = a.T * per - kGroups + i % kGroups;  // (for its lane's sake: what it has is not written)
  const unsigned t = i / per, r = i - t * per;
  const int head = r / kGroups, g = r % kGroups, lane = threadIdx.x & 31;
  const int slot = load_in_order(a.slots + t), pos = load_in_order(a.position + t);
  const __nv_bfloat16* const src =
      (IS_V ? static_cast<const __nv_bfloat16*>(a.v) + static_cast<size_t>(t) * a.ldv
            : static_cast<const __nv_bfloat16*>(a.k) + static_cast<size_t>(t) * a.ldk) + head * D + g * 16;
  const uint4 lo = load_in_order(reinterpret_cast<const uint4*>(src));
  const uint4 hi = load_in_order(reinterpret_cast<const uint4*>(src) + 1);
  const bool there = static_cast<unsigned>(slot) < static_cast<unsigned>(pg.num_pages) << pg.page_shift;
  const bool known = static_cast<unsigned>(pos) < static_cast<unsigned>(a.max_position);
  const int at = slot & ((1 << pg.page_shift) - 1), token = at & (kKvBlock - 1);
  uint8_t* const blk = pg.base + (there ? pg.block(slot >> pg.page_shift, head, at / kKvBlock) : 0);
  uint8_t* const codes = blk + (IS_V ? kv_v_code_at(D, token, g * 8) : kv_k_code_at(D, token, g * 8));
  uint8_t* const scale = blk + (IS_V ? kv_v_scale_at(D, token, g) : kv_k_scale_at(D, token, g));
  const bool write = there && known && some;
  if (!IS_V && some && r == 0 && ((!there && slot != -1) || !known)) atomicOr(a.err, LORA_ERRF_BAD_ID);
  if constexpr (IS_V) {
    if (write) write_group<true>(lo, hi, a.v_scale, codes, scale);
    return;
  }
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  const float2* const row = a.angles + static_cast<size_t>(known ? pos : 0) * (a.rotary / 2);
  const int last = a.rotary / 4 - 1, half = a.rotary / 32;  // pieces of a row - 1, groups of half a rotation
  const bool rotated = g * 16 < a.rotary, second = APART && rotated && g >= half;
  const bool one = __all_sync(0xffffffffu, t == __shfl_sync(0xffffffffu, t, 0));  // one token's lanes
  const float4 mine = load_piece(row, min(lane, last));
  const int piece0 = APART ? (second ? g - half : g) * 8 : g * 4;
  float2 x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!APART && (j & 1)) continue;
    const int k = piece0 + (APART ? j : j / 2);
    const float4 cs = one ? from_lane(mine, k & 31) : load_piece(row, min(k, last));
    if constexpr (APART) {
      const uint32_t other = __shfl_sync(0xffffffffu, w[j], !rotated ? lane : second ? lane - half : lane + half);
      x[j] = second ? turned_b(other, w[j], cs) : turned_a(w[j], other, cs);
    } else {
      x[j] = turned_pair(w[j], cs.x, cs.y);
      x[j + 1] = turned_pair(w[j + 1], cs.z, cs.w);
    }
  }
  if (!write) return;
  if (rotated) write_group<false>(x, a.k_scale, codes, scale);
  else write_group<false>(lo, hi, a.k_scale, codes, scale);
}

// 8 pairs (or 16 dimensions that are not turned) of up to kQHeads heads of one query row, a thread;
// a warp takes the row's dimensions and kQHeads * 32 / (D / 16) heads.
template <int D, bool APART>
__device__ __forceinline__ void turn_queries(const KvRotateArgs& a, unsigned i, unsigned ahead) {
  constexpr int kSlices = D / 16, kLanes = 32 / kSlices;
  const unsigned chunks = (a.q_heads + kQHeads * kLanes - 1) / (kQHeads * kLanes);
  const unsigned warp = i / 32, t = warp / chunks, lane = i % 32;
  if (t >= static_cast<unsigned>(a.T)) return;
  const unsigned next = (warp + ahead / 32) / chunks;
  if (next < static_cast<unsigned>(a.T)) {  // the lines of a warp to come, and its angles
    const unsigned chunk = warp + ahead / 32 - next * chunks;
    const int e = chunk * (kQHeads * kLanes * D) + lane * 64;
    if (e < a.q_heads * D) prefetch_l2(static_cast<const __nv_bfloat16*>(a.q) + static_cast<size_t>(next) * a.ldq + e);
    const int pos = load_in_order(a.position + next);
    if (chunk == 0 && static_cast<int>(lane) * 16 < a.rotary / 2 &&
        static_cast<unsigned>(pos) < static_cast<unsigned>(a.max_position))
      prefetch_l2(a.angles + static_cast<size_t>(pos) * (a.rotary / 2) + lane * 16);
  }
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
  if (static_cast<unsigned>(pos) >= static_cast<unsigned>(a.max_position)) {  // (of all lanes)
    if (slice == 0 && head0 == 0) atomicOr(a.err, LORA_ERRF_BAD_ID);
    return;
  }
  const float4 mine =
      load_piece(a.angles + static_cast<size_t>(pos) * (a.rotary / 2), min(static_cast<int>(lane), a.rotary / 4 - 1));
  float4 cs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = from_lane(mine, slice * 4 + i);
#pragma unroll
  for (int h = 0; h < kQHeads; ++h) {
    const int head = head0 + h * kLanes;
    if (head >= a.q_heads) break;
    if (rotated) {
      uint32_t w0[4] = {v0[h].x, v0[h].y, v0[h].z, v0[h].w}, w1[4] = {v1[h].x, v1[h].y, v1[h].z, v1[h].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 x, y;
        if constexpr (APART) {
          x = turned_a(w0[k], w1[k], cs[k]);
          y = turned_b(w0[k], w1[k], cs[k]);
        } else {  // angles 2 k' and 2 k' + 1 of the first words' pairs, then of the second ones'
          const float4 c0 = cs[k / 2], c1 = cs[2 + k / 2];
          x = k & 1 ? turned_pair(w0[k], c0.z, c0.w) : turned_pair(w0[k], c0.x, c0.y);
          y = k & 1 ? turned_pair(w1[k], c1.z, c1.w) : turned_pair(w1[k], c1.x, c1.y);
        }
        w0[k] = pack_bf16x2(x.x, x.y);
        w1[k] = pack_bf16x2(y.x, y.y);
      }
      v0[h] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
      v1[h] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
    }
    *reinterpret_cast<uint4*>(out + head * D + d0) = v0[h];
    *reinterpret_cast<uint4*>(out + head * D + d1) = v1[h];
  }
}

// The kernel behind may start at once: it reads the cache and the queries behind its own wait.
template <int D, bool APART>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv_rotate_kernel(KvRotateArgs a, unsigned kv_blocks, unsigned kv_ahead, unsigned q_ahead) {
  griddep_wait();
  griddep_launch_dependents();
  // the blocks of keys and values evenly among those of queries: how many of the former come before
  const unsigned long long n = 2 * kv_blocks;
  const unsigned before = static_cast<unsigned>(blockIdx.x * n / gridDim.x);
  if ((blockIdx.x + 1) * n / gridDim.x == before)
    turn_queries<D, APART>(a, (blockIdx.x - before) * kThreads + threadIdx.x, q_ahead);
  else if (before & 1)
    write_one<D, APART, true>(a, (before >> 1) * kThreads + threadIdx.x, kv_ahead);
  else
    write_one<D, APART, false>(a, (before >> 1) * kThreads + threadIdx.x, kv_ahead);
}

template <int D, bool APART>
cudaError_t launch(const KvRotateArgs& a, cudaStream_t stream) {
  const auto blocks = [](long long threads) { return static_cast<unsigned>((threads + kThreads - 1) / kThreads); };
  constexpr int kWarpHeads = kQHeads * 32 / (D / 16);
  const unsigned kv = blocks(static_cast<long long>(a.T) * a.pages.heads * (D / 16));
  const unsigned q = blocks(static_cast<long long>(a.T) * ((a.q_heads + kWarpHeads - 1) / kWarpHeads) * 32);
  // what the blocks that follow the resident ones read is asked for a round ahead
  const long long resident = static_cast<long long>(a.num_sms) * kCtasPerSm, all = 2ll * kv + q;
  const unsigned kv_ahead = static_cast<unsigned>(resident * kv / all) * kThreads,
                 q_ahead = static_cast<unsigned>(resident * q / all) * kThreads;
  return launch_dependent(kv_rotate_kernel<D, APART>, dim3(static_cast<unsigned>(all)), kThreads, 0, stream, a, kv,
                          kv_ahead, q_ahead);
}

}  // namespace

cudaError_t launch_kv_rotate(const KvRotateArgs& a, cudaStream_t stream) {
  if (a.pages.D == 128) return a.interleaved ? launch<128, false>(a, stream) : launch<128, true>(a, stream);
  return a.interleaved ? launch<64, false>(a, stream) : launch<64, true>(a, stream);
}

}  // namespace lora
