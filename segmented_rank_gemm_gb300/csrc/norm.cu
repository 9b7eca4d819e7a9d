// norm.cu -- root-mean-square norm with the residual's addition, and an e4m3 copy with row
// scales (include/lora_norm.h: lora_rms_norm).
//
//     h = x + r,   y = (h w) rstd,   rstd = 1 / sqrt(mean h^2 + eps)
//     sx = max|y| / 448,   xq = e4m3(y / sx)
// Rounding is monotone, so max|y| = max|h w| rstd: the sum of h^2 and the maximum of |h w|
// come out of one reduction, and a row needs one pass over memory, held in registers
// between its load and its stores.
//
// Bound: DRAM bytes (x, r, w in; h, y, xq, sx out).  A row is shared by TPR threads with VEC
// 16-byte vectors each, all loaded before the reduction; rows of up to 4 vectors a warp lane
// stay within a warp and need no barrier.  Measured: 8192 rows of 4096 in bf16 with everything
// written 47.0 us, 6.4 TB/s; 512 rows 4.1 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "e4m3_row.cuh"
#include "lora_common.cuh"
#include "lora_kernels.h"
#include "lora_norm.h"

namespace lora {
namespace {

constexpr int kMaxWidth = 32768;
constexpr int kMaxRows = 1 << 20;

struct NormArgs {
  const void *x, *res, *w;
  long long ldx, ldr, ldh;
  float eps;
  int T, K;
  void *h, *y;
  uint8_t* xq;
  float* sx;
};

// VW consecutive elements (16 bytes, or one element) as fp32.
template <typename T, int VW>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16, 8> {
  static __device__ __forceinline__ void load(const void* p, size_t i, float (&f)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16_lo(w[j]);
      f[2 * j + 1] = bf16_hi(w[j]);
    }
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[8]) {
    uint4 v;
    v.x = pack_bf16x2(f[0], f[1]);
    v.y = pack_bf16x2(f[2], f[3]);
    v.z = pack_bf16x2(f[4], f[5]);
    v.w = pack_bf16x2(f[6], f[7]);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = v;
  }
};
template <>
struct Chunk<float, 4> {
  static __device__ __forceinline__ void load(const void* p, size_t i, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[4]) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Chunk<__nv_bfloat16, 2> {
  static __device__ __forceinline__ void load(const void* p, size_t i, float (&f)[2]) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p) + i);
    f[0] = bf16_lo(v);
    f[1] = bf16_hi(v);
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[2]) {
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p) + i) = pack_bf16x2(f[0], f[1]);
  }
};
template <>
struct Chunk<__nv_bfloat16, 1> {
  static __device__ __forceinline__ void load(const void* p, size_t i, float (&f)[1]) {
    f[0] = __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[1]) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f[0]);
  }
};
template <>
struct Chunk<float, 1> {
  static __device__ __forceinline__ void load(const void* p, size_t i, float (&f)[1]) {
    f[0] = static_cast<const float*>(p)[i];
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[1]) {
    static_cast<float*>(p)[i] = f[0];
  }
};

template <int VW>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&f)[VW], float s, float r,
                                           bool fast) {
  if constexpr (VW == 1) {
    *p = static_cast<uint8_t>(to_e4m3x2(f[0], 0.f, s, r, fast) & 0xff);
  } else if constexpr (VW == 2) {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(to_e4m3x2(f[0], f[1], s, r, fast));
  } else {
    uint32_t q[VW / 4];
#pragma unroll
    for (int j = 0; j < VW / 4; ++j)
      q[j] = to_e4m3x2(f[4 * j], f[4 * j + 1], s, r, fast) |
             to_e4m3x2(f[4 * j + 2], f[4 * j + 3], s, r, fast) << 16;
    if constexpr (VW == 8) *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(p) = q[0];
  }
}

// TPR threads a row, VEC chunks of VW elements a thread (chunk c: elements VW (lane + c TPR)).
template <typename T, int VW, int TPR, int VEC, int NT>
__global__ void __launch_bounds__(NT) rms_norm_kernel(NormArgs a) {
  using C = Chunk<T, VW>;
  static_assert(TPR == 32 || TPR == NT, "a row is a warp's or the CTA's");
  griddep_wait();
  const int lane = threadIdx.x % TPR;
  const int row = blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
  if (TPR == 32 && row >= a.T) return;
  const int n = a.K / VW;
  const size_t x0 = static_cast<size_t>(row) * a.ldx, r0 = static_cast<size_t>(row) * a.ldr;
  const size_t h0 = static_cast<size_t>(row) * a.ldh, y0 = static_cast<size_t>(row) * a.K;

  float h[VEC][VW];  // then h w
  float sum = 0.f, top = 0.f;
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    const int e = lane + c * TPR;
    if (e < n) {
      C::load(a.x, x0 + static_cast<size_t>(e) * VW, h[c]);
    } else {
#pragma unroll
      for (int j = 0; j < VW; ++j) h[c][j] = 0.f;
    }
  }
  if (a.res) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      const int e = lane + c * TPR;
      if (e < n) {
        float r[VW];
        C::load(a.res, r0 + static_cast<size_t>(e) * VW, r);
#pragma unroll
        for (int j = 0; j < VW; ++j) h[c][j] += r[j];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    const int e = lane + c * TPR;
    if (e < n) {
      float w[VW];
      C::load(a.w, static_cast<size_t>(e) * VW, w);
      if (a.h) C::store(a.h, h0 + static_cast<size_t>(e) * VW, h[c]);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        sum += h[c][j] * h[c][j];
        h[c][j] *= w[j];
        top = fmaxf(top, fabsf(h[c][j]));
      }
    }
  }
  if (!a.y && !a.xq) return;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, d);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  }
  if constexpr (TPR > 32) {
    __shared__ float2 part[TPR / 32];
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = make_float2(sum, top);
    __syncthreads();
    sum = top = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) {
      sum += part[i].x;
      top = fmaxf(top, part[i].y);
    }
  }
  const float rstd = 1.f / sqrtf(sum / static_cast<float>(a.K) + a.eps);
  top *= rstd;
  const float s = top > 0.f ? __fdiv_rn(top, kE4m3Max) : 1.f;
  const bool fast = fast_scale(s);
  const float rcp = fast ? __frcp_rn(s) : 0.f;
  if (a.sx && lane == 0) a.sx[row] = s;
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    const int e = lane + c * TPR;
    if (e < n) {
#pragma unroll
      for (int j = 0; j < VW; ++j) h[c][j] *= rstd;  // y
      const size_t at = y0 + static_cast<size_t>(e) * VW;
      if (a.y) C::store(a.y, at, h[c]);
      if (a.xq) store_e4m3<VW>(a.xq + at, h[c], s, rcp, fast);
    }
  }
}

template <typename T, int VW, int TPR, int VEC, int NT>
cudaError_t launch(const NormArgs& a, cudaStream_t stream) {
  const int rows = NT / TPR;
  return launch_dependent(rms_norm_kernel<T, VW, TPR, VEC, NT>, dim3((a.T + rows - 1) / rows), NT, 0,
                          stream, a);
}

// Threads and chunks a row, by its chunks.  Measured with a residual, h and y written (us, 8192
// rows of bf16 unless said): 1024 wide 7.6 with a warp a row, 9.5 with 128 threads of one chunk; 4096
// wide 42.1 with 128 threads of four chunks, 45.2 with 256 of two, 52.0 with 512 of one; 8192
// wide 80.6 with 256 of four, 97.8 with 512 of two; 32768 wide (2048 rows) 100 with 1024 of four,
// 154 with 512 of eight; 4-byte floats, 14336 wide (4096 rows) 157 and 168 with the same.  Rows
// that no 16-byte vector fits (odd widths or distances) go by 4-byte pairs or by elements: 1001
// wide 13.4 us, 4090 wide 46.8, 4095 wide 68.6, where 256 threads of eight and 512 of 16 elements
// took 22.7, 104 and 104.
template <typename T, int VW>
cudaError_t launch_width(const NormArgs& a, cudaStream_t stream) {
  const int n = a.K / VW;  // chunks of a row
  if constexpr (VW > 2) {
    if (n <= 64) return launch<T, VW, 32, 2, 128>(a, stream);
    if (n <= 128) return launch<T, VW, 32, 4, 128>(a, stream);
    if (n <= 256) return launch<T, VW, 128, 2, 128>(a, stream);
    if (n <= 512) return launch<T, VW, 128, 4, 128>(a, stream);
    if (n <= 1024) return launch<T, VW, 256, 4, 256>(a, stream);
    if (n <= 2048) return launch<T, VW, 512, 4, 512>(a, stream);
    if constexpr (kMaxWidth / VW > 4096)
      if (n > 4096) return launch<T, VW, 1024, 8, 1024>(a, stream);
    return launch<T, VW, 1024, 4, 1024>(a, stream);
  } else {
    if (n <= 128) return launch<T, VW, 32, 4, 128>(a, stream);
    if (n <= 512) return launch<T, VW, 32, 16, 128>(a, stream);
    if (n <= 1024) return launch<T, VW, 128, 8, 128>(a, stream);
    if (n <= 2048) return launch<T, VW, 256, 8, 256>(a, stream);
    if (n <= 4096) return launch<T, VW, 512, 8, 512>(a, stream);
    if (n <= 8192) return launch<T, VW, 512, 16, 512>(a, stream);
    if constexpr (kMaxWidth / VW > 16384)
      if (n > 16384) return launch<T, VW, 1024, 32, 1024>(a, stream);
    return launch<T, VW, 1024, 16, 1024>(a, stream);
  }
}

bool aligned(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// `rows` rows of `width` bytes, `pitch` bytes apart.
struct Rows {
  const void* p;
  size_t rows, width, pitch;
};

// Whether two sets of rows share a byte.  Sets of the same pitch may interleave (column ranges
// of one buffer); sets of different pitches count by their whole extents.
bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
  if (p >= q + (b.rows - 1) * b.pitch + b.width || q >= p + (a.rows - 1) * a.pitch + a.width)
    return false;
  if (a.pitch != b.pitch) return true;
  const size_t from_a = p <= q ? (q - p) % a.pitch : (a.pitch - (p - q) % a.pitch) % a.pitch;
  return from_a < a.width || from_a + b.width > a.pitch;  // b's columns, counted from a's
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_rms_norm(const void* x, int ldx, const void* res, int ldr, const void* w,
                             float eps, int T, int K, int dtype, void* h, int ldh, void* y, void* xq,
                             float* sx, void* stream_) {
  if (T < 0 || T > kMaxRows || K < 1 || K > kMaxWidth || !(eps >= 0.f) ||
      (dtype != LORA_BF16 && dtype != LORA_F32) || ldx < K || (res && ldr < K) || (h && ldh < K))
    return LORA_EINVAL;
  if (T == 0) return LORA_OK;
  if (!x || !w || !xq != !sx || (!y && !xq && !h)) return LORA_EINVAL;
  const size_t es = dtype == LORA_BF16 ? 2 : 4;
  for (const void* p : {x, res, w, static_cast<const void*>(h), static_cast<const void*>(y)})
    if (!aligned(p, static_cast<int>(es))) return LORA_EINVAL;
  if (!aligned(sx, 4)) return LORA_EINVAL;
  const size_t t = T, n = K;
  const Rows in[] = {{x, t, n * es, ldx * es}, {res, t, n * es, ldr * es}, {w, 1, n * es, n * es}};
  const Rows out[] = {{y, t, n * es, n * es}, {xq, t, n, n}, {sx, t, 4, 4}, {h, t, n * es, ldh * es}};
  for (int i = 0; i < 4; ++i) {
    for (const Rows& s : in) {
      // h may be the residual or x itself: a chunk is read before it is written
      if (i == 3 && h && s.p == h && s.pitch == ldh * es && (h == res || h == x)) continue;
      if (overlap(out[i], s)) return LORA_EINVAL;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return LORA_EINVAL;
  }
  NormArgs a{x, res, w, ldx, ldr, ldh, eps, T, K, h, y, static_cast<uint8_t*>(xq), sx};
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int vw = 16 / static_cast<int>(es);
  const bool vec = K % vw == 0 && ldx % vw == 0 && (!res || ldr % vw == 0) && (!h || ldh % vw == 0) &&
                   aligned(x, 16) && aligned(res, 16) && aligned(w, 16) && aligned(h, 16) &&
                   aligned(y, 16) && aligned(xq, vw);
  const bool pairs = K % 2 == 0 && ldx % 2 == 0 && (!res || ldr % 2 == 0) && (!h || ldh % 2 == 0) &&
                     aligned(x, 4) && aligned(res, 4) && aligned(w, 4) && aligned(h, 4) &&
                     aligned(y, 4) && aligned(xq, 2);
  cudaError_t e;
  if (dtype == LORA_BF16)
    e = vec ? launch_width<__nv_bfloat16, 8>(a, stream)
        : pairs ? launch_width<__nv_bfloat16, 2>(a, stream) : launch_width<__nv_bfloat16, 1>(a, stream);
  else
    e = vec ? launch_width<float, 4>(a, stream) : launch_width<float, 1>(a, stream);
  return e == cudaSuccess ? LORA_OK : LORA_ECUDA;
}
