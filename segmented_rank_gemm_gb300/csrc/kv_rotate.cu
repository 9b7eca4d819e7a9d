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
//
// Measured (32 query heads over 8 of 128): 8192 tokens at positions over 32768 30 us (181 MB, 6.0 TB/s; it
// issues in 61% of its cycles), 512 tokens 3, one 2.  With a thread for two groups of keys the angles
// and addresses cost half, but 84 registers leave 16 warps an SM: 42 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_decode.cuh"
#include "kv_kernels.h"
#include "kv_quant.cuh"
#include "lora_common.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

// (8192 tokens with the read-back 42.9 us with 512 threads a block, 40.4 with 256, 39.0 with 128, 38.8 with 64)
constexpr int kThreads = 128;
constexpr int kQHeads = 4;
constexpr int kCtasPerSm = 8;

__device__ __forceinline__ float2 bf16x2_values(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
// a c - b s and b c + a s of two pairs at once.  The sums are scalar: packed ones are fused with the packed
// products before them, which spares a product's rounding (seen in results where the terms cancel).
__device__ __forceinline__ float2 turned_a(float2 a, float2 b, float2 c, float2 s) {
  const float2 x = mul2(a, c), y = mul2(b, s);
  return make_float2(__fsub_rn(x.x, y.x), __fsub_rn(x.y, y.y));
}
__device__ __forceinline__ float2 turned_b(float2 a, float2 b, float2 c, float2 s) {
  const float2 x = mul2(b, c), y = mul2(a, s);
  return make_float2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}
// One pair, its elements beside each other.
__device__ __forceinline__ float2 turned_pair(float2 ab, float c, float s) {
  const float2 x = mul2(ab, make_float2(c, c)), y = mul2(make_float2(ab.y, ab.x), make_float2(s, s));
  return make_float2(__fsub_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

// Four cosines or sines from another lane.  A row's angles are loaded once by the lanes of a warp, four
// of them each, and exchanged where they are used: loaded by each thread, 64 or 128 bytes a lane, they
// took three quarters of the L1's cycles (8192 rows of 32 and 8 heads of 128 40 us, 33 exchanged).
__device__ __forceinline__ float4 from_lane(const float4& v, int lane) {
  return make_float4(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane),
                     __shfl_sync(0xffffffffu, v.z, lane), __shfl_sync(0xffffffffu, v.w, lane));
}
__device__ __forceinline__ float4 load_piece(const float* row, int i) {
  return __ldg(reinterpret_cast<const float4*>(row) + i);
}
__device__ __forceinline__ float flip(float x, uint32_t sign) { return __uint_as_float(__float_as_uint(x) ^ sign); }
__device__ __forceinline__ float2 low(const float4& v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 high(const float4& v) { return make_float2(v.z, v.w); }

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A group of 16 dimensions of one token and head of K or V, a thread.  Keys: the pairs' other elements,
// where they are in another group, come from the lane that has it.
template <int D, bool APART, bool IS_V>
__device__ __forceinline__ void write_one(const KvRotateArgs& a, unsigned i, unsigned ahead) {
  constexpr unsigned kGroups = D / 16;
  const KvPages& pg = a.pages;
  const unsigned per = pg.heads * kGroups;  // of a token
  const bool some = i < a.T * per;
  if (!some) i = a.T * per - kGroups + i % kGroups;  // (for its lane's sake: what it has is not written)
  const unsigned t = i / per, r = i - t * per;
  const int head = r / kGroups, g = r % kGroups, lane = threadIdx.x & 31;
  const int slot = load_in_order(a.slots + t), pos = load_in_order(a.position + t);
  const __nv_bfloat16* const src =
      (IS_V ? static_cast<const __nv_bfloat16*>(a.v) + static_cast<size_t>(t) * a.ldv
            : static_cast<const __nv_bfloat16*>(a.k) + static_cast<size_t>(t) * a.ldk) + head * D + g * 16;
  if (t + ahead < static_cast<unsigned>(a.T) && (i & 3) == 0)  // a line of a block to come
    prefetch_l2(src + static_cast<size_t>(ahead) * (IS_V ? a.ldv : a.ldk));
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
  const float* const row = a.angles + static_cast<size_t>(known ? pos : 0) * a.rotary;
  const int sines = a.rotary / 8, half = a.rotary / 32;  // the sines' first piece, groups of half a rotation
  const bool rotated = g * 16 < a.rotary, second = APART && rotated && g >= half;
  const bool one = __all_sync(0xffffffffu, t == __shfl_sync(0xffffffffu, t, 0));  // one token's lanes
  const float4 mine = load_piece(row, min(lane, 2 * sines - 1));
  const int piece0 = !rotated ? 0 : APART ? (second ? g - half : g) * 4 : g * 2;
  const int partner = !rotated ? lane : second ? lane - half : lane + half;
  const uint32_t turn = second ? 0u : 0x80000000u;  // the first elements take the sine's product off
  float2 x[8];
#pragma unroll
  for (int j = 0; j < 8; j += APART ? 2 : 4) {  // four angles
    const int k = piece0 + j / (APART ? 2 : 4);
    float4 c = one ? from_lane(mine, k) : load_piece(row, k);
    float4 sn = one ? from_lane(mine, sines + k) : load_piece(row, sines + k);
    if constexpr (APART) {
      sn = make_float4(flip(sn.x, turn), flip(sn.y, turn), flip(sn.z, turn), flip(sn.w, turn));
      const uint32_t o0 = __shfl_sync(0xffffffffu, w[j], partner), o1 = __shfl_sync(0xffffffffu, w[j + 1], partner);
      x[j] = turned_b(bf16x2_values(o0), bf16x2_values(w[j]), low(c), low(sn));
      x[j + 1] = turned_b(bf16x2_values(o1), bf16x2_values(w[j + 1]), high(c), high(sn));
    } else {
      x[j] = turned_pair(bf16x2_values(w[j]), c.x, sn.x);
      x[j + 1] = turned_pair(bf16x2_values(w[j + 1]), c.y, sn.y);
      x[j + 2] = turned_pair(bf16x2_values(w[j + 2]), c.z, sn.z);
      x[j + 3] = turned_pair(bf16x2_values(w[j + 3]), c.w, sn.w);
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
  // a warp to come: its lines, and its angles
  const unsigned next = t + ahead, chunk = warp - t * chunks;
  if (next < static_cast<unsigned>(a.T)) {
    const int e = chunk * (kQHeads * kLanes * D) + lane * 64;
    if (e < a.q_heads * D) prefetch_l2(static_cast<const __nv_bfloat16*>(a.q) + static_cast<size_t>(next) * a.ldq + e);
    const int pos = load_in_order(a.position + next);
    if (chunk == 0 && static_cast<int>(lane) * 32 < a.rotary &&
        static_cast<unsigned>(pos) < static_cast<unsigned>(a.max_position))
      prefetch_l2(a.angles + static_cast<size_t>(pos) * a.rotary + lane * 32);
  }
  const int slice = lane % kSlices;
  const int head0 = chunk * (kQHeads * kLanes) + lane / kSlices;
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
  const int sines = a.rotary / 8, piece0 = rotated ? slice * 2 : 0;
  const float4 mine =
      load_piece(a.angles + static_cast<size_t>(pos) * a.rotary, min(static_cast<int>(lane), 2 * sines - 1));
  float4 c[2], sn[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) c[i] = from_lane(mine, piece0 + i), sn[i] = from_lane(mine, sines + piece0 + i);
#pragma unroll
  for (int h = 0; h < kQHeads; ++h) {
    const int head = head0 + h * kLanes;
    if (head >= a.q_heads) break;
    if (rotated) {
      uint32_t w0[4] = {v0[h].x, v0[h].y, v0[h].z, v0[h].w}, w1[4] = {v1[h].x, v1[h].y, v1[h].z, v1[h].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 u = bf16x2_values(w0[k]), v = bf16x2_values(w1[k]);
        float2 x, y;
        if constexpr (APART) {
          const float2 ck = k & 1 ? high(c[k / 2]) : low(c[k / 2]), sk = k & 1 ? high(sn[k / 2]) : low(sn[k / 2]);
          x = turned_a(u, v, ck, sk);
          y = turned_b(u, v, ck, sk);
        } else {  // the first words' pairs have the first four angles
          const float ca[4] = {c[0].x, c[0].y, c[0].z, c[0].w}, sa[4] = {sn[0].x, sn[0].y, sn[0].z, sn[0].w};
          const float cb[4] = {c[1].x, c[1].y, c[1].z, c[1].w}, sb[4] = {sn[1].x, sn[1].y, sn[1].z, sn[1].w};
          x = turned_pair(u, ca[k], sa[k]);
          y = turned_pair(v, cb[k], sb[k]);
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

// kv_share: the share of blocks that keys and values take, times 2^32, rounded up.  The kernel behind may
// start at once: it reads the cache and the queries behind its own wait.
template <int D, bool APART>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    kv_rotate_kernel(KvRotateArgs a, uint32_t kv_share, unsigned ahead) {
  griddep_wait();
  griddep_launch_dependents();
  // the blocks of keys and values evenly among those of queries: how many of the former come before
  const unsigned before = __umulhi(blockIdx.x, kv_share);
  if (__umulhi(blockIdx.x + 1, kv_share) == before)
    turn_queries<D, APART>(a, (blockIdx.x - before) * kThreads + threadIdx.x, ahead);
  else if (before & 1)
    write_one<D, APART, true>(a, (before >> 1) * kThreads + threadIdx.x, ahead);
  else
    write_one<D, APART, false>(a, (before >> 1) * kThreads + threadIdx.x, ahead);
}

template <int D, bool APART>
cudaError_t launch(const KvRotateArgs& a, cudaStream_t stream) {
  const auto blocks = [](long long threads) { return static_cast<unsigned>((threads + kThreads - 1) / kThreads); };
  constexpr int kWarpHeads = kQHeads * 32 / (D / 16);
  const unsigned kv = blocks(static_cast<long long>(a.T) * a.pages.heads * (D / 16));
  const unsigned q = blocks(static_cast<long long>(a.T) * ((a.q_heads + kWarpHeads - 1) / kWarpHeads) * 32);
  const unsigned long long n = 2ull * kv, all = n + q;
  // what the blocks that follow the resident ones read is asked for half a round, so many tokens, ahead
  // (8192 tokens: 43.4 us not asked for, 41.4 two rounds ahead, 39.0 one, 38.5 half a round)
  const long long ahead = static_cast<long long>(a.T) * a.num_sms * kCtasPerSm / static_cast<long long>(all);
  return launch_dependent(kv_rotate_kernel<D, APART>, dim3(static_cast<unsigned>(all)), kThreads, 0, stream, a,
                          static_cast<uint32_t>(((n << 32) + all - 1) / all),
                          static_cast<unsigned>(std::min<long long>(ahead / 2 + 1, 1 << 30)));
}

}  // namespace

cudaError_t launch_kv_rotate(const KvRotateArgs& a, cudaStream_t stream) {
  if (a.pages.D == 128) return a.interleaved ? launch<128, false>(a, stream) : launch<128, true>(a, stream);
  return a.interleaved ? launch<64, false>(a, stream) : launch<64, true>(a, stream);
}

}  // namespace lora
