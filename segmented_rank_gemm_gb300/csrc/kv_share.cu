// kv_share.cu -- the joining of rows whose request shares a prefix (include/lora_kv.h:
// lora_kv_attend_shared): o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the row's two
// results, M the larger of m_0 and m_1, in fp32, rounded once.
//
// Bound: bytes (D fp32 twice in, D bf16 out of a row and head, mostly from L2) and, for a decode
// batch, the launch.  A warp takes kHeads heads of one row, whose loads are all under way together.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_decode.cuh"
#include "kv_kernels.h"
#include "kv_span.cuh"
#include "lora_common.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;

// The last of offsets[0 .. n) that is <= x (which offsets[0] is): the lanes of a warp cut the
// range in 32.
__device__ __forceinline__ int last_not_above(const int32_t* offsets, int n, int x, int lane) {
  int lo = 0, len = n;  // the answer is in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32, at = lo + lane * step;
    const bool below = lane * step < len && load_in_order(offsets + at) <= x;
    const int k = max(0, 31 - __clz(__ballot_sync(0xffffffffu, below)));
    len = min(step, len - k * step);
    lo += k * step;
  }
  return lo;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_share_join_kernel(KvAttendArgs a, int row_blocks) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) >= row_blocks) {
    // The groups agree with their requests: one with a prefix is a member, and has its group's.
    const int b = (blockIdx.x - row_blocks) * kThreads + threadIdx.x;
    if (b >= a.B) return;
    const Span s = load_span(a, a.groups + b, false);
    if (s.q_len > 0 && s.kind != kSpanWhole) {
      int lo = 0, hi = a.groups;  // the last group that starts at b or before
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.group_offsets[mid] <= b) lo = mid;
        else hi = mid;
      }
      if (b < a.group_offsets[lo] || b >= a.group_offsets[lo + 1] || a.shared[b] != a.prefix_len[lo])
        atomicOr(a.err, LORA_ERRF_BAD_ID);
    }
    return;
  }
  const int chunks = (a.q_heads + kHeads - 1) / kHeads;
  const long long item = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int row = static_cast<int>(item / chunks), head0 = static_cast<int>(item % chunks) * kHeads;
  if (row >= a.T || row < load_in_order(a.q_offsets) || row >= load_in_order(a.q_offsets + a.B)) return;
  const int b = last_not_above(a.q_offsets, a.B, row, lane);
  if (load_span(a, a.groups + b, false).kind == kSpanWhole) return;
  constexpr int VL = D / 32;
  float2 ml[kHeads][2];
  float o[kHeads][2][VL];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    const size_t at = static_cast<size_t>(row) * a.q_heads + min(head0 + h, a.q_heads - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ml[h][i] = __ldcs(a.part_ml[i] + at);
      const float2* src = reinterpret_cast<const float2*>(a.part_o[i] + at * D + lane * VL);
#pragma unroll
      for (int k = 0; k < VL / 2; ++k) {
        const float2 x = __ldcs(src + k);
        o[h][i][2 * k] = x.x;
        o[h][i][2 * k + 1] = x.y;
      }
    }
  }
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (head0 + h >= a.q_heads) break;
    const float m = fmaxf(ml[h][0].x, ml[h][1].x);
    const float w0 = ex2(ml[h][0].x - m), w1 = ex2(ml[h][1].x - m);
    const float l = w0 * ml[h][0].y + w1 * ml[h][1].y;
    const float f = l == 0.f ? 0.f : kKvUnit * a.v_scale / l, f0 = w0 * f, f1 = w1 * f;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) +
                                                static_cast<size_t>(row) * a.ldo + (head0 + h) * D + lane * VL);
#pragma unroll
    for (int k = 0; k < VL / 2; ++k)
      out[k] = pack_bf16x2(f0 * o[h][0][2 * k] + f1 * o[h][1][2 * k],
                           f0 * o[h][0][2 * k + 1] + f1 * o[h][1][2 * k + 1]);
  }
}

template <int D>
cudaError_t launch(const KvAttendArgs& a, cudaStream_t stream) {
  const long long items = static_cast<long long>(a.T) * ((a.q_heads + kHeads - 1) / kHeads);
  const int row_blocks = static_cast<int>((items + kThreads / 32 - 1) / (kThreads / 32));
  return launch_dependent(kv_share_join_kernel<D>, dim3(row_blocks + (a.B + kThreads - 1) / kThreads), kThreads,
                          0, stream, a, row_blocks);
}

}  // namespace

cudaError_t launch_kv_share_join(const KvAttendArgs& a, cudaStream_t stream) {
  return a.pages.D == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace lora
