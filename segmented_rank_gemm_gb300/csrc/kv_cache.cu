// kv_cache.cu -- the 4-bit key/value cache object, its write and its read-back, and the
// argument checks of the attention over it (include/lora_kv.h).
#include <cuda_bf16.h>
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
#include "kv_decode.cuh"
#include "kv_kernels.h"

namespace lora {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float e4m3_value(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// A group of 16 dimensions of one token and head, of K and of V, a thread: twice 32 bytes of
// values, 8 of codes and one scale.  Threads run along the token's row, so both directions move
// whole lines.
struct Group {
  unsigned t;    // token
  int hg;        // group of the token's row
  int slot;
  bool there;    // the slot is one of the cache's
  uint8_t *k, *v, *k_scale, *v_scale;  // codes and scales
};
__device__ __forceinline__ Group locate(const KvPages& pg, const int32_t* slots, unsigned i,
                                        unsigned groups) {
  Group x;
  x.t = i / groups;
  x.hg = static_cast<int>(i - x.t * groups);
  x.slot = load_in_order(slots + x.t);
  x.there = static_cast<unsigned>(x.slot) < static_cast<unsigned>(pg.num_pages) << pg.page_shift;
  const int per_log2 = pg.D == 128 ? 3 : 2;  // groups of a head
  const int head = x.hg >> per_log2, group = x.hg & ((1 << per_log2) - 1);
  const int pos = x.slot & ((1 << pg.page_shift) - 1), token = pos & (kKvBlock - 1);
  uint8_t* blk = pg.base + pg.block(x.slot >> pg.page_shift, head, pos / kKvBlock);
  x.k = blk + kv_k_code_at(pg.D, token, group * 8);
  x.v = blk + kv_v_code_at(pg.D, token, group * 8);
  x.k_scale = blk + kv_k_scale_at(pg.D, token, group);
  x.v_scale = blk + kv_v_scale_at(pg.D, token, group);
  return x;
}

// Codes of 16 values whose quotients by s round to -7 .. 7, y = 1 / s correctly rounded.  The
// quotient is Markstein's: q = x y is corrected twice by its remainder, x - q s, exact in one
// fused multiply-add once q is within one unit in the last place, which makes the last result the
// correctly rounded x / s -- as a division, with one reciprocal for the group.  Adding
// 1.5 2^23 rounds to an integer, ties to even, and leaves it in the low bits; a shifted add
// puts it in its nibble, and what the sums carry besides is one constant.
template <bool IS_V>
__device__ __forceinline__ uint2 codes_of(const uint32_t (&w)[8], float s, float y) {
  const float2 y2 = make_float2(y, y), minus_s = make_float2(-s, -s);
  const float2 magic = make_float2(12582912.f, 12582912.f);
  uint32_t code[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    code[h] = 0x11111111u * (8u - 0x4B400000u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = make_float2(bf16_lo(w[4 * h + j]), bf16_hi(w[4 * h + j]));
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

// Writes the group at src, of a cache of scale g.
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
  const uint8_t sb = static_cast<uint8_t>(
      __nv_cvt_float_to_fp8(__fdiv_rn(top, 7.f * g), __NV_SATFINITE, __NV_E4M3));
  const float s = e4m3_value(sb) * g;
  const float y = __frcp_rn(s);
  uint2 code;
  // (the range keeps every product and remainder of a quotient from a half up a normal number)
  if (!nan && s > 0x1p-60f && s < 0x1p60f && top * y < 7.49f) {
    code = codes_of<IS_V>(w, s, y);
  } else {  // zeros, saturated scales, the smallest scales, NaN: division and clamp by element
    code = make_uint2(0u, 0u);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
      float q = s > 0.f ? rintf(__fdiv_rn(x, s)) : 0.f;
      q = q != q ? 0.f : fminf(fmaxf(q, -7.f), 7.f);
      (j < 8 ? code.x : code.y) |= static_cast<uint32_t>(static_cast<int>(q) + 8)
                                   << (4 * kv_nibble(IS_V, j & 7));
    }
  }
  *reinterpret_cast<uint2*>(codes) = code;
  *scale = sb;
}

// Bound: for large batches the instructions (about 14 a value, a third of them the quotient)
// beside the bytes, for small ones the launch.  Measured with 8 heads of 128: 8192 tokens 9.5 us (43
// MB, 4.5 TB/s; under a profiler it issues in 66% of its cycles) and 16.6 with the read-back, where 16
// divisions a group, K and V in separate threads, took 32.4; 512 tokens 2.1 us.
// The kernel behind may start at once: what it reads of the cache it reads behind its own wait.
__global__ void __launch_bounds__(kThreads)
    kv_append_kernel(KvPages pg, const __nv_bfloat16* k, int ldk, const __nv_bfloat16* v, int ldv,
                     const int32_t* slots, int T, float k_scale, float v_scale, int32_t* err) {
  griddep_wait();
  griddep_launch_dependents();
  const unsigned groups = pg.heads * pg.D / kKvGroup;  // of a token's row
  const unsigned i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= T * groups) return;
  const Group at = locate(pg, slots, i, groups);
  const uint4* ks =
      reinterpret_cast<const uint4*>(k + static_cast<size_t>(at.t) * ldk + at.hg * kKvGroup);
  const uint4* vs =
      reinterpret_cast<const uint4*>(v + static_cast<size_t>(at.t) * ldv + at.hg * kKvGroup);
  const uint4 k0 = load_in_order(ks), k1 = load_in_order(ks + 1);
  const uint4 v0 = load_in_order(vs), v1 = load_in_order(vs + 1);
  if (!at.there) {
    if (at.slot != -1 && at.hg == 0) atomicOr(err, LORA_ERRF_BAD_ID);
    return;
  }
  write_group<false>(k0, k1, k_scale, at.k, at.k_scale);
  write_group<true>(v0, v1, v_scale, at.v, at.v_scale);
}

// The read-back.  Bound: bytes (8192 tokens of 8 heads of 128 6.8 us, 6.3 TB/s).  The pair of lanes that swap halves: a lane that stored its own 32
// bytes wrote half sectors twice, 2.5 million sector writes for 8192 tokens instead of 1.6.
// Values n s g of a group: n s is exact in bf16 (kv_decode.cuh), so a cache of scale 1 gives it
// as it is.
template <bool IS_V>
__device__ __forceinline__ void values_of(uint2 c, uint32_t sb, float g, uint32_t (&out)[8]) {
  const DecodeBf16 dec = decode_scale_bf16(sb, 0, 0x7B807B80u);  // 2^120
  uint32_t lo[4], hi[4];  // pairs of nibbles i and i + 4
  decode4(c.x, dec, lo);
  decode4(c.y, dec, hi);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (IS_V) {  // dimensions i and i + 4
      out[j] = prmt(lo[2 * (j & 1)], lo[2 * (j & 1) + 1], j < 2 ? 0x5410 : 0x7632);
      out[4 + j] = prmt(hi[2 * (j & 1)], hi[2 * (j & 1) + 1], j < 2 ? 0x5410 : 0x7632);
    } else {  // dimensions 2 i and 2 i + 1
      out[j] = lo[j];
      out[4 + j] = hi[j];
    }
  }
  if (g != 1.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = pack_bf16x2(bf16_lo(out[j]) * g, bf16_hi(out[j]) * g);
  }
}

// Stores the 32 bytes of group i and, by the neighbour lane, of group i ^ 1, so that a store
// covers whole sectors: the lanes of a pair exchange halves, and write first the even lane's
// group, then the odd one's.
__device__ __forceinline__ void store_pair(uint4* rows, unsigned i, unsigned n,
                                           const uint32_t (&x)[8]) {
  const bool odd = i & 1;
  uint32_t give[4], first[4], second[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) give[j] = __shfl_xor_sync(0xffffffffu, odd ? x[j] : x[4 + j], 1);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    first[j] = odd ? give[j] : x[j];
    second[j] = odd ? x[4 + j] : give[j];
  }
  const unsigned even = i & ~1u;
  uint4* dst = rows + static_cast<size_t>(even) * 2 + odd;
  if (even < n) dst[0] = make_uint4(first[0], first[1], first[2], first[3]);
  if (even + 1 < n) dst[2] = make_uint4(second[0], second[1], second[2], second[3]);
}

__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(KvPages pg, const int32_t* slots, int T, float k_scale, float v_scale,
                   __nv_bfloat16* k, __nv_bfloat16* v, int32_t* err) {
  griddep_wait();
  const unsigned groups = pg.heads * pg.D / kKvGroup;
  const unsigned i = blockIdx.x * kThreads + threadIdx.x, n = T * groups;
  uint32_t kv[8] = {}, vv[8] = {};
  if (i < n) {
    const Group at = locate(pg, slots, i, groups);
    if (at.there) {
      const uint2 kc = load_in_order(reinterpret_cast<const uint2*>(at.k));
      const uint2 vc = load_in_order(reinterpret_cast<const uint2*>(at.v));
      const uint32_t ks = load_in_order(at.k_scale), vs = load_in_order(at.v_scale);
      values_of<false>(kc, ks, k_scale, kv);
      values_of<true>(vc, vs, v_scale, vv);
    } else if (at.slot != -1 && at.hg == 0) {
      atomicOr(err, LORA_ERRF_BAD_ID);
    }
  }
  store_pair(reinterpret_cast<uint4*>(k), i, n, kv);
  store_pair(reinterpret_cast<uint4*>(v), i, n, vv);
}

// What an attention call leaves whose wait gave up: the flag, and counts of CTAs that joined a group
// others of which never arrived (include/lora_kv.h: lora_kv_wait_selftest).
__global__ void kv_wait_selftest_kernel(int32_t* arrivals, int n, int32_t* err) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
    mbar_wait(&bar, 0u, err);  // (phase 0 completes only on an arrival)
  }
  for (int i = threadIdx.x; i < n; i += blockDim.x) arrivals[i] = 1;
}

// Blocks over the groups of T rows.
dim3 rows_grid(const KvPages& pg, int T) {
  const long long n = static_cast<long long>(T) * (pg.heads * pg.D / kKvGroup);
  return dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads));
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

// both attention kernels' arrival counts, groups claimed and CTAs done claiming
constexpr size_t kArrivalsBytes = (2 * kKvMaxCtas + 2) * sizeof(int32_t);
constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxRequests = 16384;
// Rows a cache head (query rows times q_heads / kv_heads) up to which a request's attention runs
// in the kernel for few rows, which costs by 8 rows what the one for many costs by 256.  Measured
// over 8 heads of 128 (us, few / many): 64 requests of 1024 positions, 16 rows 50 / 67, 24 rows
// 66 / 67, 32 rows 82 / 67; 8 of 4096, 39 / 42 at 24 and 45 / 42 at 32; 256 of 300, 79 / 97 and 89 / 97.
constexpr int kFewRows = 24;

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

// Whether the cache is the current device's: kernels are launched there.
bool here(const lora_kv_cache* c) {
  int device = -1;
  return cudaGetDevice(&device) == cudaSuccess && device == c->device;
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
      max_requests > kMaxRequests || !(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(7.f * k_scale) ||
      !std::isfinite(7.f * v_scale))
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
      cudaMalloc(&c->arrivals, kArrivalsBytes) != cudaSuccess ||
      cudaMalloc(&c->err, sizeof(int32_t)) != cudaSuccess) {
    cudaGetLastError();
    rc = LORA_ENOMEM;
  } else if (cudaMemsetAsync(c->pages.base, 0, c->bytes, stream) != cudaSuccess ||
             cudaMemsetAsync(c->arrivals, 0, kArrivalsBytes, stream) != cudaSuccess ||
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
  if (!here(c)) return fail(c, LORA_EINVAL, "the cache is on device %d", c->device);
  const int width = c->pages.heads * c->pages.D;
  if (T < 0 || T > kMaxTokens) return fail(c, LORA_EINVAL, "T=%d", T);
  if (ldk < width || ldv < width || ldk % 8 || ldv % 8)
    return fail(c, LORA_EINVAL, "row distances %d, %d: multiples of 8 from %d up", ldk, ldv, width);
  if (T == 0) return LORA_OK;
  if (!k || !v || !slots || !aligned16(k) || !aligned16(v))
    return fail(c, LORA_EINVAL, "k, v and kv_slot must be given, k and v 16-byte aligned");
  KV_CUDA(c, launch_dependent(kv_append_kernel, rows_grid(c->pages, T), kThreads, 0,
                              static_cast<cudaStream_t>(stream), c->pages,
                              static_cast<const __nv_bfloat16*>(k), ldk,
                              static_cast<const __nv_bfloat16*>(v), ldv, slots, T, c->k_scale,
                              c->v_scale, c->err));
  return LORA_OK;
}

int lora_kv_read(lora_kv_cache_t* c, const int32_t* slots, int T, void* k_out, void* v_out,
                 void* stream) {
  if (!c) return LORA_EINVAL;
  if (!here(c)) return fail(c, LORA_EINVAL, "the cache is on device %d", c->device);
  if (T < 0 || T > kMaxTokens) return fail(c, LORA_EINVAL, "T=%d", T);
  if (T == 0) return LORA_OK;
  if (!slots || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
    return fail(c, LORA_EINVAL, "kv_slot and outputs must be given, outputs 16-byte aligned");
  KV_CUDA(c, launch_dependent(kv_read_kernel, rows_grid(c->pages, T), kThreads, 0,
                              static_cast<cudaStream_t>(stream), c->pages, slots, T, c->k_scale,
                              c->v_scale, static_cast<__nv_bfloat16*>(k_out),
                              static_cast<__nv_bfloat16*>(v_out), c->err));
  return LORA_OK;
}

int lora_kv_attend(lora_kv_cache_t* c, const void* q, int ldq, int q_heads, const int32_t* q_offsets,
                   const int32_t* kv_len, const int32_t* block_table, int max_blocks, int B, int T,
                   int max_q, float scale, void* out, int ldo, void* stream) {
  if (!c) return LORA_EINVAL;
  if (!here(c)) return fail(c, LORA_EINVAL, "the cache is on device %d", c->device);
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
  // from products with the keys to scores in units of log2(e); the kernel for
  // few rows multiplies it by kKvUnit
  const float scale_log2 = scale * c->k_scale * 1.44269504088896341f;
  if (!std::isfinite(scale_log2 * kKvUnit))
    return fail(c, LORA_EINVAL, "scale=%g times k_scale=%g is too large", scale, c->k_scale);
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
  a.scale_log2 = scale_log2;
  a.v_scale = c->v_scale;
  a.out = out;
  a.ldo = ldo;
  a.pieces = c->pieces;
  a.arrivals = c->arrivals;
  a.few_rows = kFewRows;
  a.prompt_pieces = c->prompt_pieces;
  a.prompt_arrivals = c->arrivals + kKvMaxCtas;
  a.prompt_claim = c->arrivals + 2 * kKvMaxCtas;
  a.err = c->err;
  a.num_sms = c->num_sms;
  a.many_follow = static_cast<long long>(max_q) * a.group > kFewRows;
  KV_CUDA(c, launch_kv_attend(a, static_cast<cudaStream_t>(stream)));
  if (a.many_follow)
    KV_CUDA(c, launch_kv_prompt(a, static_cast<cudaStream_t>(stream)));
  return LORA_OK;
}

int lora_kv_get_status(lora_kv_cache_t* c, void* stream_) {
  if (!c) return LORA_EINVAL;
  if (!here(c)) return fail(c, LORA_EINVAL, "the cache is on device %d", c->device);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int32_t flags = 0;
  KV_CUDA(c, cudaMemcpyAsync(&flags, c->err, sizeof(flags), cudaMemcpyDeviceToHost, stream));
  KV_CUDA(c, cudaStreamSynchronize(stream));
  if (!flags) return LORA_OK;
  // On the caller's stream, ahead of the calls that follow there.  CTAs that gave up did not arrive
  // where others had: those counts would have later calls join pieces that are not written yet.
  KV_CUDA(c, cudaMemsetAsync(c->err, 0, sizeof(flags), stream));
  if (flags & LORA_ERRF_TIMEOUT)
    KV_CUDA(c, cudaMemsetAsync(c->arrivals, 0, kArrivalsBytes, stream));
  KV_CUDA(c, cudaStreamSynchronize(stream));
  if (flags & LORA_ERRF_TIMEOUT)
    return fail(c, LORA_ETIMEOUT, "a kernel wait timed out (flags=%d)", flags);
  return fail(c, LORA_EID, "a slot, page id, length or offset out of range (flags=%d)", flags);
}

int lora_kv_wait_selftest(lora_kv_cache_t* c, void* stream) {
  if (!c) return LORA_EINVAL;
  if (!here(c)) return fail(c, LORA_EINVAL, "the cache is on device %d", c->device);
  kv_wait_selftest_kernel<<<1, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      c->arrivals, 2 * kKvMaxCtas, c->err);
  KV_CUDA(c, cudaGetLastError());
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
