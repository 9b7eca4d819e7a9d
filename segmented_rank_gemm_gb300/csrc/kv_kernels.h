// kv_kernels.h -- the 4-bit cache's layout in memory and the launchers of its kernels
// (kv_cache.cu: the object, append and read; kv_attend.cu and kv_prompt.cu: attention).
//
// Pages hold blocks of 16 tokens of one head:
//     page -> head -> block of 16 positions -> { K codes | K scales | V codes | V scales }
// so a page's positions of one head are one contiguous run that a single bulk copy fetches.
// Within a block, with D = head_dim (D/2 bytes of codes and D/16 scales a token):
//   K codes  [16][D/2]: token rows, 8 dimensions a 32-bit word, whose nibbles 0..3 hold the even
//            dimensions and 4..7 the odd ones: what decodes to a pair is then a pair of the query.
//   V codes  [16][D/2]: 8 dimensions a word in order; D = 128 swaps the two 32-byte halves of tokens
//            with bit 1 set, so that the lanes of a warp reading one 8-byte piece of 4 tokens hit
//            all banks.
//   K scales and V scales in the order the lanes of the attention's matrix fragments read
//            them (k_scale_at, v_scale_at).
// The rows of a 16 x 16 fragment are the block's tokens in the order frag_token: lane group
// t = 0..3 owns fragment indexes 2t, 2t+1, 2t+8, 2t+9, and any bijection to tokens serves as
// long as keys, values and probabilities use the same one.  This one keeps both the K rows read
// together and the V rows read together on different banks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace lora {

constexpr int kKvBlock = 16;  // tokens of a block
constexpr int kKvGroup = 16;  // dimensions that share a scale

__host__ __device__ constexpr int kv_codes_bytes(int D) { return kKvBlock * D / 2; }
__host__ __device__ constexpr int kv_scales_bytes(int D) { return kKvBlock * D / kKvGroup; }
__host__ __device__ constexpr int kv_block_bytes(int D) {
  return 2 * (kv_codes_bytes(D) + kv_scales_bytes(D));
}
__host__ __device__ constexpr int kv_k_scales(int D) { return kv_codes_bytes(D); }
__host__ __device__ constexpr int kv_v_codes(int D) { return kv_codes_bytes(D) + kv_scales_bytes(D); }
__host__ __device__ constexpr int kv_v_scales(int D) {
  return 2 * kv_codes_bytes(D) + kv_scales_bytes(D);
}

// Nibble of a word's dimension i in 0..7.
__host__ __device__ constexpr int kv_nibble(bool is_v, int i) {
  return is_v ? i : (i >> 1) + 4 * (i & 1);
}

// Token of the block at fragment index r in 0..15.
__host__ __device__ constexpr int kv_frag_token(int r) {
  const int t = (r >> 1) & 3, i0 = r & 1, i1 = r >> 3;
  return ((t & 1) ^ i0) | (t >> 1) << 1 | i0 << 2 | i1 << 3;
}
// Its inverse.
__host__ __device__ constexpr int kv_token_frag(int token) {
  const int b0 = token & 1, b1 = (token >> 1) & 1, i0 = (token >> 2) & 1, i1 = token >> 3;
  return i1 << 3 | b1 << 2 | (b0 ^ i0) << 1 | i0;
}

// Byte offsets within a block.
__host__ __device__ constexpr int kv_k_code_at(int D, int token, int byte) {
  return token * (D / 2) + byte;
}
__host__ __device__ constexpr int kv_v_code_at(int D, int token, int byte) {
  return kv_v_codes(D) + token * (D / 2) + (D == 128 ? byte ^ ((token & 2) << 4) : byte);
}
// K: the lane of fragment row g (0..7) and lane group t reads the scales of rows g and g + 8 for
// the D/64 groups of its D/4 dimensions, together.
__host__ __device__ constexpr int kv_k_scale_at(int D, int token, int group) {
  const int r = kv_token_frag(token), per = D / 64;
  return kv_k_scales(D) + (((r & 7) * 4 + group / per) * 2 + (r >> 3)) * per + group % per;
}
// V: the lane of lane group t reads one group's scales of its four tokens 2t, 2t+1, 2t+8, 2t+9
// (fragment indexes), together.
__host__ __device__ constexpr int kv_v_scale_at(int D, int token, int group) {
  const int r = kv_token_frag(token), t = (r >> 1) & 3;
  return kv_v_scales(D) + (group * 4 + t) * 4 + ((r & 1) | (r >> 3) << 1);
}

struct KvPages {
  uint8_t* base;
  int num_pages, page_shift, heads, D;
  // Byte offset of block `blk` of (page, head).
  __host__ __device__ __forceinline__ size_t block(int page, int head, int blk) const {
    return ((static_cast<size_t>(page) * heads + head) * (size_t(1) << (page_shift - 4)) + blk) *
           kv_block_bytes(D);
  }
};

struct KvAttendArgs {
  KvPages pages;
  const void* q;
  int ldq, q_heads;
  const int32_t *q_offsets, *kv_len, *table;
  int max_blocks, B, T, max_q;
  int group;             // q_heads / kv_heads
  uint32_t group_magic;  // floor(2^32 / group) + 1 (unused for 1)
  // c / group of a row c < 2^26: c (magic group - 2^32) < 2^32 as magic group - 2^32 <= group <= 64.
  __device__ __forceinline__ int token_of(int c) const {
    return group == 1 ? c : static_cast<int>(__umulhi(static_cast<uint32_t>(c), group_magic));
  }
  float scale_log2;  // softmax scale times k_scale times log2(e)
  float v_scale;
  void* out;
  int ldo;
  float* pieces;      // partial results of a group that several warps or CTAs share
  int32_t* arrivals;  // [kKvMaxCtas] CTAs done with the group that starts in a CTA (zeroed)
  // Requests with more rows a cache head than this go to the kernel for many rows.
  int few_rows;
  int many_follow;  // that kernel is launched next
  float* prompt_pieces;      // that kernel's workspaces
  int32_t* prompt_arrivals;  // [kKvMaxCtas] (zeroed)
  int32_t* prompt_claim;     // groups claimed, CTAs done claiming (zeroed)
  int32_t* err;
  int num_sms;
  // What the kernels' span variants (kv_span.cuh) read besides.
  int causal;  // 0: a row sees everything its request has cached (no groups then)
  const int32_t *group_offsets, *prefix_row, *prefix_len;  // [groups + 1], [groups], [groups] (or null)
  const int32_t* shared;  // [B] (or null)
  int groups;
  int alone;  // the groups are checked, but every request is attended by itself
  // Unnormalised results that are joined afterwards, of every row and head of T: O [D], and the
  // reference m with the sum l.  [0]: of a request's own positions, [1]: of its group's prefix.
  float* part_o[2];
  float2* part_ml[2];
};

constexpr int kKvMaxCtas = 1024;

// Floats of the partial results' workspace.
size_t kv_attend_workspace_floats(int num_sms, int D);
cudaError_t launch_kv_attend(const KvAttendArgs& a, cudaStream_t stream);
// The kernel for requests of many rows (kv_prompt.cu); it leaves the other rows alone.
size_t kv_prompt_workspace_floats(int num_sms, int D);
cudaError_t launch_kv_prompt(const KvAttendArgs& a, cudaStream_t stream);
struct KvRotateArgs {
  KvPages pages;
  const void *q, *k, *v;
  void* q_out;
  int ldq, ldqo, ldk, ldv, q_heads;
  const int32_t *position, *slots;
  int T;
  const float* angles;  // [max_position][2][rotary / 2]: cosines, sines
  int max_position, rotary, interleaved;
  float k_scale, v_scale;
  int32_t* err;
  int num_sms;
};
cudaError_t launch_kv_rotate(const KvRotateArgs& a, cudaStream_t stream);
// Joins the results of rows with a shared prefix (kv_share.cu).
cudaError_t launch_kv_share_join(const KvAttendArgs& a, cudaStream_t stream);

}  // namespace lora
