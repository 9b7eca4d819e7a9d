// kv_share.cu -- the joining of rows whose request shares a prefix (include/lora_kv.h:
// lora_kv_attend_shared): o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the row's two
// results, M the larger of m_0 and m_1, in fp32, rounded once.
//
// A result that the kernel for many rows has in pieces (a group cut between CTAs) is joined here as
// well, by the same rule, with all rows of the batch at once.
//
// Bound: bytes (D fp32 twice in, D bf16 out of a row and head, mostly from L2) and, for a decode
// batch, the launch and one trip to L2.  A warp takes a head of one row.  Measured with 32 heads of 128:
// 512 rows 10 us, 64 rows of 19 pieces each 8.4 (a third of either is the launch).
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

template <int VL>
__device__ __forceinline__ void load_o(const float* src, float (&o)[VL]) {
#pragma unroll
  for (int k = 0; k < VL; k += 2) {
    const float2 x = __ldcg(reinterpret_cast<const float2*>(src + k));
    o[k] = x.x;
    o[k + 1] = x.y;
  }
}

// Joins a row's pieces: their common reference m, the sum l, and this lane's dimensions of O.
template <int D>
__device__ __forceinline__ float2 join_pieces(const KvAttendArgs& a, KvPieces p, int lane, float (&o)[D / 32]) {
  constexpr int VL = D / 32, kPiece = kv_prompt_piece_floats(D);
  // (counts out of range are those of a call that was flagged: nothing wrote them)
  const int n = p.first_cut >= 1 && p.first_cut + p.count <= min(kKvMaxCtas, a.num_sms) + 1 && p.row < kKvPromptRows
                    ? p.count
                    : 0;
  const auto piece = [&](int k) {
    return a.prompt_pieces + static_cast<size_t>(kv_prompt_piece(p.first_cut, k)) * kPiece + p.row;
  };
  float m = -1.7e38f, l = 0.f;
#pragma unroll
  for (int i = 0; i < VL; ++i) o[i] = 0.f;
  for (int k0 = 0; k0 < n; k0 += 32) {
    const bool mine = k0 + lane < n;
    const float mk = mine ? __ldcg(piece(k0 + lane)) : -1.7e38f;
    const float lk = mine ? __ldcg(piece(k0 + lane) + kKvPromptRows) : 0.f;
    float top = fmaxf(m, mk);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float back = ex2(m - top), f = ex2(mk - top);
    m = top;
    float sum = f * lk;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = l * back + sum;
#pragma unroll
    for (int i = 0; i < VL; ++i) o[i] *= back;
    const int some = min(32, n - k0);
#pragma unroll 8
    for (int k = 0; k < some; ++k) {
      float x[VL];
      load_o<VL>(piece(k0 + k) + 2 * kKvPromptRows + p.row * (D - 1) + lane * VL, x);
      const float w = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
      for (int i = 0; i < VL; ++i) o[i] += w * x[i];
    }
  }
  return make_float2(m, l);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_share_join_kernel(KvAttendArgs a, int row_blocks) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) >= row_blocks) {
    const int b = (blockIdx.x - row_blocks) * kThreads + threadIdx.x;
    if (b < a.B) check_group_of(a, b);
    return;
  }
  const long long at = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int row = static_cast<int>(at / a.q_heads), head = static_cast<int>(at - static_cast<long long>(row) * a.q_heads);
  if (row >= a.T) return;
  // all that a row in two whole parts needs, asked for at once
  constexpr int VL = D / 32;
  const int lo = load_in_order(a.q_offsets), hi = load_in_order(a.q_offsets + a.B);
  float2 ml0 = __ldcg(a.part_ml[0] + at), ml1 = __ldcg(a.part_ml[1] + at);
  float o0[VL], o1[VL];
  load_o<VL>(a.part_o[0] + at * D + lane * VL, o0);
  load_o<VL>(a.part_o[1] + at * D + lane * VL, o1);
  if (row < lo || row >= hi) return;
  const bool one = kv_is_row_times(ml0) || KvPieces::only(ml0);
  if (KvPieces::are(ml0)) ml0 = join_pieces<D>(a, KvPieces(ml0), lane, o0);
  float f0, f1 = 0.f;
  if (one) {
    f0 = kv_is_row_times(ml0) ? ml0.x : kv_factor(a, ml0.y);
#pragma unroll
    for (int k = 0; k < VL; ++k) o1[k] = 0.f;
  } else {
    if (KvPieces::are(ml1)) ml1 = join_pieces<D>(a, KvPieces(ml1), lane, o1);
    const float m = fmaxf(ml0.x, ml1.x), w0 = ex2(ml0.x - m), w1 = ex2(ml1.x - m);
    const float f = kv_factor(a, w0 * ml0.y + w1 * ml1.y);
    f0 = w0 * f, f1 = w1 * f;
  }
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(row) * a.ldo +
                                              head * D + lane * VL);
#pragma unroll
  for (int k = 0; k < VL / 2; ++k)
    out[k] = pack_bf16x2(f0 * o0[2 * k] + f1 * o1[2 * k], f0 * o0[2 * k + 1] + f1 * o1[2 * k + 1]);
}

template <int D>
cudaError_t launch(const KvAttendArgs& a, cudaStream_t stream) {
  const long long items = static_cast<long long>(a.T) * a.q_heads;
  const int row_blocks = static_cast<int>((items + kThreads / 32 - 1) / (kThreads / 32));
  return launch_dependent(kv_share_join_kernel<D>, dim3(row_blocks + (a.B + kThreads - 1) / kThreads), kThreads,
                          0, stream, a, row_blocks);
}

}  // namespace

cudaError_t launch_kv_share_join(const KvAttendArgs& a, cudaStream_t stream) {
  return a.pages.D == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace lora
