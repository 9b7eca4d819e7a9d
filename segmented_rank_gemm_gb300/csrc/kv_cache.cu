// kv_cache.cu -- the 4-bit key/value cache object, its write and its read-back, and the
// argument checks of the attention over it (include/lora_kv.h).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "lora_common.cuh"
#include "lora_kernels.h"
#include "lora_kv.h"
#include "kv_kernels.h"

namespace lora {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float e4m3_value(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// One group of 16 dimensions of one token and head a thread: 32 bytes in, 8 bytes of codes
// and one scale out.  Bound: bytes, and for small batches the launch.
__global__ void __launch_bounds__(kThreads)
    kv_append_kernel(KvPages pg, const __nv_bfloat16* __restrict__ k, int ldk,
                     const __nv_bfloat16* __restrict__ v, int ldv,
                     const int32_t* __restrict__ slots, int T, float k_scale, float v_scale,
                     int32_t* err) {
  const int groups = pg.heads * pg.D / kKvGroup;  // of a token, K or V
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long n = static_cast<long long>(T) * groups;
  if (i >= 2 * n) return;
  const bool is_v = i >= n;
  const long long e = is_v ? i - n : i;
  const int t = static_cast<int>(e / groups), hg = static_cast<int>(e % groups);
  const int slot = slots[t];
  if (static_cast<unsigned>(slot) >=
      static_cast<unsigned>(pg.num_pages) << pg.page_shift) {
    if (slot != -1 && hg == 0) atomicOr(err, LORA_ERRF_BAD_ID);
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(
      (is_v ? v + static_cast<size_t>(t) * ldv : k + static_cast<size_t>(t) * ldk) + hg * kKvGroup);
  const uint4 lo = __ldg(src), hi = __ldg(src + 1);
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  float x[16], top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[2 * j] = bf16_lo(w[j]);
    x[2 * j + 1] = bf16_hi(w[j]);
    top = fmaxf(top, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));  // ignores NaN
  }
  const float g = is_v ? v_scale : k_scale;
  const uint8_t sb = static_cast<uint8_t>(
      __nv_cvt_float_to_fp8(__fdiv_rn(top, 7.f * g), __NV_SATFINITE, __NV_E4M3));
  const float s = e4m3_value(sb) * g;
  uint32_t code[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float q = s > 0.f ? rintf(__fdiv_rn(x[j], s)) : 0.f;
    q = q != q ? 0.f : fminf(fmaxf(q, -7.f), 7.f);
    code[j >> 3] |= static_cast<uint32_t>(static_cast<int>(q) + 8) << (4 * kv_nibble(is_v, j & 7));
  }
  const int per_head = pg.D / kKvGroup;
  const int head = hg / per_head, group = hg % per_head;
  const int page = slot >> pg.page_shift, pos = slot & ((1 << pg.page_shift) - 1);
  const int token = pos & (kKvBlock - 1);
  uint8_t* blk = pg.base + pg.block(page, head, pos / kKvBlock);
  const int at = is_v ? kv_v_code_at(pg.D, token, group * 8) : kv_k_code_at(pg.D, token, group * 8);
  *reinterpret_cast<uint2*>(blk + at) = make_uint2(code[0], code[1]);
  blk[is_v ? kv_v_scale_at(pg.D, token, group) : kv_k_scale_at(pg.D, token, group)] = sb;
}

__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(KvPages pg, const int32_t* __restrict__ slots, int T, float k_scale,
                   float v_scale, __nv_bfloat16* __restrict__ k, __nv_bfloat16* __restrict__ v,
                   int32_t* err) {
  const int groups = pg.heads * pg.D / kKvGroup;
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long n = static_cast<long long>(T) * groups;
  if (i >= 2 * n) return;
  const bool is_v = i >= n;
  const long long e = is_v ? i - n : i;
  const int t = static_cast<int>(e / groups), hg = static_cast<int>(e % groups);
  const int slot = slots[t];
  uint32_t out[8] = {};
  if (static_cast<unsigned>(slot) < static_cast<unsigned>(pg.num_pages) << pg.page_shift) {
    const int per_head = pg.D / kKvGroup;
    const int head = hg / per_head, group = hg % per_head;
    const int page = slot >> pg.page_shift, pos = slot & ((1 << pg.page_shift) - 1);
    const int token = pos & (kKvBlock - 1);
    const uint8_t* blk = pg.base + pg.block(page, head, pos / kKvBlock);
    const int at =
        is_v ? kv_v_code_at(pg.D, token, group * 8) : kv_k_code_at(pg.D, token, group * 8);
    const uint2 c = *reinterpret_cast<const uint2*>(blk + at);
    const uint8_t sb =
        blk[is_v ? kv_v_scale_at(pg.D, token, group) : kv_k_scale_at(pg.D, token, group)];
    const float s = e4m3_value(sb), g = is_v ? v_scale : k_scale;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t word = j < 4 ? c.x : c.y;
      const int i = 2 * (j & 3);
      const float a = static_cast<float>(static_cast<int>(word >> (4 * kv_nibble(is_v, i)) & 15) - 8);
      const float b = static_cast<float>(static_cast<int>(word >> (4 * kv_nibble(is_v, i + 1)) & 15) - 8);
      out[j] = pack_bf16x2(a * s * g, b * s * g);
    }
  } else if (slot != -1 && hg == 0) {
    atomicOr(err, LORA_ERRF_BAD_ID);
  }
  uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + static_cast<size_t>(t) * groups * kKvGroup +
                                        hg * kKvGroup);
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

}  // namespace
}  // namespace lora

using namespace lora;

struct lora_kv_cache {
  KvPages pages{};
  size_t bytes = 0;
  int max_requests = 0, device = 0, num_sms = 0;
  float k_scale = 1.f, v_scale = 1.f;
  float* pieces = nullptr;      // attention's partial results
  float* prompt_pieces = nullptr;
  int32_t* arrivals = nullptr;  // attention's arrival counts, both kernels' (zero between calls)
  int32_t* err = nullptr;
  char last_error[256] = "";
};

namespace {

constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxRequests = 16384;
// Rows a cache head (query rows times q_heads / kv_heads) up to which a request's attention runs
// in the kernel for few rows.
constexpr int kFewRows = 16;

int fail(lora_kv_cache* c, int code, const char* fmt, ...) {
  if (c) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(c->last_error, sizeof(c->last_error), fmt, ap);
    va_end(ap);
  }
  return code;
}

#define KV_CUDA(C, expr)                                                                    \
  do {                                                                                      \
    cudaError_t e_ = (expr);                                                                \
    if (e_ != cudaSuccess) return fail((C), LORA_ECUDA, "%s: %s", #expr, cudaGetErrorString(e_)); \
  } while (0)

void free_all(lora_kv_cache* c) {
  void* ptrs[] = {c->pages.base, c->pieces, c->prompt_pieces, c->arrivals, c->err};
  for (void* p : ptrs)
    if (p) cudaFree(p);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

extern "C" {

int lora_kv_cache_create(lora_kv_cache_t** out, int num_pages, int page_size, int kv_heads,
                         int head_dim, int max_requests, float k_scale, float v_scale,
                         void* stream_) {
  if (!out) return LORA_EINVAL;
  *out = nullptr;
  int shift = 4;
  while (shift <= 8 && page_size != 1 << shift) ++shift;
  if (shift > 8 || num_pages < 1 || static_cast<long long>(num_pages) * page_size > INT_MAX ||
      kv_heads < 1 || kv_heads > 256 || (head_dim != 64 && head_dim != 128) || max_requests < 1 ||
      max_requests > kMaxRequests || !(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) ||
      !std::isfinite(v_scale))
    return LORA_EINVAL;
  lora_kv_cache* c = new (std::nothrow) lora_kv_cache;
  if (!c) return LORA_ENOMEM;
  if (cudaGetDevice(&c->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess) {
    delete c;
    return LORA_ECUDA;
  }
  c->pages = KvPages{nullptr, num_pages, shift, kv_heads, head_dim};
  c->bytes = c->pages.block(num_pages, 0, 0);
  c->max_requests = max_requests;
  c->k_scale = k_scale;
  c->v_scale = v_scale;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const size_t floats = kv_attend_workspace_floats(c->num_sms, head_dim);
  int rc = LORA_OK;
  if (cudaMalloc(&c->pages.base, c->bytes) != cudaSuccess ||
      cudaMalloc(&c->pieces, floats * sizeof(float)) != cudaSuccess ||
      cudaMalloc(&c->prompt_pieces, kv_prompt_workspace_floats(c->num_sms, head_dim) *
                                        sizeof(float)) != cudaSuccess ||
      cudaMalloc(&c->arrivals, 2 * kKvMaxCtas * sizeof(int32_t)) != cudaSuccess ||
      cudaMalloc(&c->err, sizeof(int32_t)) != cudaSuccess) {
    cudaGetLastError();
    rc = LORA_ENOMEM;
  } else if (cudaMemsetAsync(c->pages.base, 0, c->bytes, stream) != cudaSuccess ||
             cudaMemsetAsync(c->arrivals, 0, 2 * kKvMaxCtas * sizeof(int32_t), stream) != cudaSuccess ||
             cudaMemsetAsync(c->err, 0, sizeof(int32_t), stream) != cudaSuccess ||
             cudaStreamSynchronize(stream) != cudaSuccess) {
    rc = LORA_ECUDA;
  }
  if (rc != LORA_OK) {
    free_all(c);
    delete c;
    return rc;
  }
  *out = c;
  return LORA_OK;
}

int lora_kv_append(lora_kv_cache_t* c, const void* k, int ldk, const void* v, int ldv,
                   const int32_t* slots, int T, void* stream) {
  if (!c) return LORA_EINVAL;
  const int width = c->pages.heads * c->pages.D;
  if (T < 0 || T > kMaxTokens) return fail(c, LORA_EINVAL, "T=%d", T);
  if (ldk < width || ldv < width || ldk % 8 || ldv % 8)
    return fail(c, LORA_EINVAL, "row distances %d, %d: multiples of 8 from %d up", ldk, ldv, width);
  if (T == 0) return LORA_OK;
  if (!k || !v || !slots || !aligned16(k) || !aligned16(v))
    return fail(c, LORA_EINVAL, "k, v and kv_slot must be given, k and v 16-byte aligned");
  const long long n = 2LL * T * (width / kKvGroup);
  kv_append_kernel<<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0,
                     static_cast<cudaStream_t>(stream)>>>(
      c->pages, static_cast<const __nv_bfloat16*>(k), ldk, static_cast<const __nv_bfloat16*>(v), ldv,
      slots, T, c->k_scale, c->v_scale, c->err);
  KV_CUDA(c, cudaGetLastError());
  return LORA_OK;
}

int lora_kv_read(lora_kv_cache_t* c, const int32_t* slots, int T, void* k_out, void* v_out,
                 void* stream) {
  if (!c) return LORA_EINVAL;
  if (T < 0 || T > kMaxTokens) return fail(c, LORA_EINVAL, "T=%d", T);
  if (T == 0) return LORA_OK;
  if (!slots || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
    return fail(c, LORA_EINVAL, "kv_slot and outputs must be given, outputs 16-byte aligned");
  const long long n = 2LL * T * (c->pages.heads * c->pages.D / kKvGroup);
  kv_read_kernel<<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0,
                   static_cast<cudaStream_t>(stream)>>>(
      c->pages, slots, T, c->k_scale, c->v_scale, static_cast<__nv_bfloat16*>(k_out),
      static_cast<__nv_bfloat16*>(v_out), c->err);
  KV_CUDA(c, cudaGetLastError());
  return LORA_OK;
}

int lora_kv_attend(lora_kv_cache_t* c, const void* q, int ldq, int q_heads, const int32_t* q_offsets,
                   const int32_t* kv_len, const int32_t* block_table, int max_blocks, int B, int T,
                   int max_q, float scale, void* out, int ldo, void* stream) {
  if (!c) return LORA_EINVAL;
  const int heads = c->pages.heads, D = c->pages.D;
  if (T < 0 || T > kMaxTokens) return fail(c, LORA_EINVAL, "T=%d", T);
  if (B < 1 || B > c->max_requests)
    return fail(c, LORA_EINVAL, "B=%d outside [1, max_requests=%d]", B, c->max_requests);
  if (q_heads < heads || q_heads % heads || q_heads / heads > 64)
    return fail(c, LORA_EINVAL, "q_heads=%d over %d cache heads", q_heads, heads);
  if (max_q < 1 || max_blocks < 1 ||
      (static_cast<long long>(max_blocks) << c->pages.page_shift) > INT_MAX ||
      static_cast<long long>(B) * max_blocks > INT_MAX || !std::isfinite(scale))
    return fail(c, LORA_EINVAL, "max_q=%d, max_blocks=%d, scale=%g", max_q, max_blocks, scale);
  if (ldq < q_heads * D || ldo < q_heads * D || ldq % 8 || ldo % 8)
    return fail(c, LORA_EINVAL, "row distances %d, %d: multiples of 8 from %d up", ldq, ldo,
                q_heads * D);
  if (T == 0) return LORA_OK;
  if (!q || !q_offsets || !kv_len || !block_table || !out || !aligned16(q) || !aligned16(out))
    return fail(c, LORA_EINVAL, "null argument, or q or out not 16-byte aligned");
  const char *qb = static_cast<const char*>(q), *ob = static_cast<const char*>(out);
  const size_t qn = (static_cast<size_t>(T - 1) * ldq + q_heads * D) * 2;
  const size_t on = (static_cast<size_t>(T - 1) * ldo + q_heads * D) * 2;
  if (qb < ob + on && ob < qb + qn) return fail(c, LORA_EINVAL, "q and out overlap");
  KvAttendArgs a;
  a.pages = c->pages;
  a.q = q;
  a.ldq = ldq;
  a.q_heads = q_heads;
  a.q_offsets = q_offsets;
  a.kv_len = kv_len;
  a.table = block_table;
  a.max_blocks = max_blocks;
  a.B = B;
  a.T = T;
  a.max_q = max_q;
  a.group = q_heads / heads;
  a.group_magic = static_cast<uint32_t>((1ull << 32) / a.group + 1);
  a.scale_log2 = scale * c->k_scale * 1.44269504088896341f;
  a.v_scale = c->v_scale;
  a.out = out;
  a.ldo = ldo;
  a.pieces = c->pieces;
  a.arrivals = c->arrivals;
  a.few_rows = kFewRows;
  a.prompt_pieces = c->prompt_pieces;
  a.prompt_arrivals = c->arrivals + kKvMaxCtas;
  a.err = c->err;
  a.num_sms = c->num_sms;
  KV_CUDA(c, launch_kv_attend(a, static_cast<cudaStream_t>(stream)));
  if (static_cast<long long>(max_q) * (q_heads / heads) > kFewRows)
    KV_CUDA(c, launch_kv_prompt(a, static_cast<cudaStream_t>(stream)));
  return LORA_OK;
}

int lora_kv_get_status(lora_kv_cache_t* c, void* stream_) {
  if (!c) return LORA_EINVAL;
  int32_t flags = 0;
  KV_CUDA(c, cudaStreamSynchronize(static_cast<cudaStream_t>(stream_)));
  KV_CUDA(c, cudaMemcpy(&flags, c->err, 4, cudaMemcpyDeviceToHost));
  KV_CUDA(c, cudaMemset(c->err, 0, 4));
  if (flags & LORA_ERRF_TIMEOUT)
    return fail(c, LORA_ETIMEOUT, "a kernel wait timed out (flags=%d)", flags);
  if (flags)
    return fail(c, LORA_EID, "a slot, page id, length or offset out of range (flags=%d)", flags);
  return LORA_OK;
}

int64_t lora_kv_cache_bytes(const lora_kv_cache_t* c) {
  return c ? static_cast<int64_t>(c->bytes) : 0;
}

const char* lora_kv_last_error(const lora_kv_cache_t* c) { return c ? c->last_error : "null cache"; }

void lora_kv_cache_destroy(lora_kv_cache_t* c) {
  if (!c) return;
  int cur = c->device;
  if (cudaGetDevice(&cur) == cudaSuccess && cur != c->device) cudaSetDevice(c->device);
  cudaDeviceSynchronize();
  free_all(c);
  delete c;
  if (cur != c->device) cudaSetDevice(cur);
}

}  // extern "C"
