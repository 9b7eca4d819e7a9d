// kv_prompt.cu -- attention of many query rows a request over the 4-bit cache
// (include/lora_kv.h: lora_kv_attend), for requests whose rows fill tensor-core tiles.
//
// With G = q_heads / kv_heads, row c of a request and cache head is token c / G, query head
// h G + c % G.  A group is (request, head, 256 rows); over tiles of 64 cached positions, per
// half of 128 rows,
//     S = Q K^T,   P = 2^(S unit - m),   l += sum P,   O += P V
// with a running reference m per row that moves only when a score exceeds it by 2^8 (O / l does
// not depend on m), fp16 operands and fp32 accumulators.  As in the kernel for few rows,
// decoded K and V are exact in fp16, queries are scaled by a power of two a row, and P is rounded
// to fp16 under a sum of its fp32 values.
//
// Bound: the tensor cores, 4 D operations a score.  One CTA per SM, its warps in four roles:
//   warps 0-3, 4-7   softmax of the rows 0..127 and 128..255, one row a thread: S from tensor
//                    memory, P back to it (the PV product takes P from there), O at the end
//   warps 8-11       decode a tile's K and V to shared memory in the 128-byte swizzled K-major
//                    layout (V transposed: its 8 x 8 blocks are transposed while they are decoded, by
//                    pairing two tokens' codes before they are extracted)
//   warp 12          issues the products: PV and the next QK of one half run while the other
//                    half's softmax does
// 256 rows share one decoding.  64 positions a tile leave room in tensor memory for S, P and O of
// both halves side by side (128 + 64 + 256 columns at D = 128), so that no product writes
// what an earlier one may still read.
//
// Work split: the tiles of all groups form one sequence, cut into equal ranges for the CTAs; a cut
// within kSnap of a group's edge (in parts of a range) moves there.  A group that is still cut
// leaves pieces (m, l, O), joined in order by the last CTA to arrive.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_decode.cuh"
#include "kv_kernels.h"
#include "lora_common.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

constexpr int kThreads = 13 * 32;
constexpr int kRows = 256;      // rows of a group, two halves
constexpr int kTile = 64;       // positions of a tile
constexpr int kStages = 3;      // decoded tiles of K, and of V
constexpr int kSetup = 2;       // units a group counts before its tiles
constexpr int kSnap = 12;       // a cut within 1 / kSnap of a range from a group's edge moves there
constexpr float kRef = 6.f;     // P is 2^kRef at the reference
constexpr float kSlack = 8.f;   // how far (in powers of two) a score may exceed the reference
constexpr float kNone = -1.7e38f;
constexpr int kTmemCols = 512;

// Instruction descriptor, kind::f16: D fp32, A and B fp16, both K-major.
constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] * B[smem]^T, kind::f16.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ---- requests, groups and the sequence of tiles ----
struct Request {
  int row0, q_len, kv, rows, parts;  // rows of one head, groups of a head
};

// Request b; one that is not for this kernel has 0 rows.  (Bad ones are reported by the other
// kernel, which runs on every call.)
__device__ __forceinline__ Request load_request(const KvAttendArgs& a, int b) {
  Request r;
  r.row0 = __ldg(a.q_offsets + b);
  const int end = __ldg(a.q_offsets + b + 1);
  r.q_len = end - r.row0;
  const int cap = a.max_blocks << a.pages.page_shift;
  r.kv = min(max(__ldg(a.kv_len + b), 0), cap);
  if (r.row0 < 0 || end > a.T || r.q_len < 0 || r.q_len > a.max_q) r.q_len = 0;
  r.rows = r.q_len * (a.q_heads / a.pages.heads);
  if (r.rows <= a.few_rows) r.rows = 0;
  r.parts = (r.rows + kRows - 1) / kRows;
  return r;
}
// Tiles of a request's group `part`: up to the last position its last row sees.
__device__ __forceinline__ int group_tiles(const KvAttendArgs& a, const Request& r, int part) {
  const int G = a.q_heads / a.pages.heads;
  const int last = r.kv - r.q_len + (min((part + 1) * kRows, r.rows) - 1) / G;
  return max(1, (last + kTile) / kTile);
}
__device__ __forceinline__ long long head_units(const KvAttendArgs& a, const Request& r) {
  long long n = 0;
  for (int part = 0; part < r.parts; ++part) n += group_tiles(a, r, part) + kSetup;
  return n;
}

// A position in the sequence of tiles, and the tile's unit.
struct Cursor {
  Request r;
  int b, head, part, tile, tiles;
  long long unit;
  // The tile at or after unit `at`, the rem-th of request b_; a cut near a group's edge moves
  // there (to the next group's first tile by its unit alone: `total` may be next).
  __device__ __forceinline__ void start(const KvAttendArgs& a, int b_, long long rem, long long at,
                                        int snap) {
    b = b_;
    r = load_request(a, b);
    const long long per = head_units(a, r);
    head = static_cast<int>(quotient(rem, per));
    rem -= head * per;
    part = 0;
    while (true) {
      tiles = group_tiles(a, r, part);
      if (rem < tiles + kSetup) break;
      rem -= tiles + kSetup;
      ++part;
    }
    const int off = static_cast<int>(rem);
    if (off <= kSetup + snap) {
      tile = 0;
      unit = at - off + kSetup;
    } else {
      tile = tiles + kSetup - off <= snap ? tiles : off - kSetup;  // tiles: the group's end
      unit = at - off + kSetup + tile;
    }
  }
  // Moves to the first tile of the next group.  Not past the last group.
  __device__ __forceinline__ void next_group(const KvAttendArgs& a) {
    unit += tiles - tile + kSetup;
    tile = 0;
    if (++part == r.parts) {
      part = 0;
      if (++head == a.pages.heads) {
        head = 0;
        do {
          ++b;
          r = load_request(a, b);
        } while (r.parts == 0);
      }
    }
    tiles = group_tiles(a, r, part);
  }
};

// A CTA's range of the sequence, walked by every role alike, a segment (one group's tiles
// tile .. tile + count - 1) at a time.
struct Walk {
  Cursor at;
  long long end;
  int count;
  __device__ __forceinline__ bool first(const KvAttendArgs& a) {
    if (at.tile == at.tiles) {  // a start moved to its group's end
      if (at.unit + kSetup >= end) return false;
      at.next_group(a);
    }
    if (at.unit >= end) return false;
    count = static_cast<int>(min(static_cast<long long>(at.tiles - at.tile), end - at.unit));
    return true;
  }
  __device__ __forceinline__ bool next(const KvAttendArgs& a) {
    if (at.unit + (at.tiles - at.tile) + kSetup >= end) return false;
    at.next_group(a);
    count = static_cast<int>(min(static_cast<long long>(at.tiles), end - at.unit));
    return true;
  }
  // Half 1 has rows.
  __device__ __forceinline__ bool second_half() const {
    return at.r.rows - at.part * kRows > kRows / 2;
  }
};

// Floats of a piece: m, l [256], O [256][D].
template <int D>
constexpr int piece_floats() {
  return kRows * (D + 2);
}

template <int D>
struct Smem {
  static constexpr int kQHalf = 128 * D * 2;     // one half's queries
  static constexpr int kKv = kTile * D * 2;      // one decoded tile of K or V
  static constexpr int kK = 2 * kQHalf, kV = kK + kStages * kKv;
  static constexpr int kBytes = kV + kStages * kKv + 1024;  // + alignment
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(KvAttendArgs a) {
  using L = Smem<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* const sm = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  __shared__ uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  __shared__ uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  __shared__ uint64_t idle, meet;
  __shared__ uint32_t tmem_holder;
  __shared__ long long scan[kThreads / 32], cut_rem[2];
  __shared__ int cut_b[2];
  __shared__ int last_cta;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = a.pages.heads, G = a.q_heads / heads;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 128);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 128);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(&idle, 1);
    mbar_init(&meet, 256);
    fence_mbar_init();
  }

  // the sequence's length and this CTA's cuts
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += head_units(a, load_request(a, b)) * heads;
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long total = 0, before = incl - mine;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const long long span = max(static_cast<long long>(kSetup + 4), quotient(total + gridDim.x - 1, gridDim.x));
  if (span * blockIdx.x >= total) return;
  const int snap = static_cast<int>(min(span / kSnap, static_cast<long long>(1 << 20)));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const long long at = span * (blockIdx.x + i);
    if (at >= before && at < before + mine) {
      long long rem = at - before;
      int b = b0;
      for (; b < b1 - 1; ++b) {
        const long long n = head_units(a, load_request(a, b)) * heads;
        if (rem < n) break;
        rem -= n;
      }
      cut_b[i] = b;
      cut_rem[i] = rem;
    }
  }
  if (warp == 12) tmem_alloc(&tmem_holder, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  const uint32_t tS = tmem, tP = tmem + 128, tO = tmem + 256;

  Walk walk;
  walk.end = total;
  if (span * (blockIdx.x + 1) < total) {
    Cursor cut;
    cut.start(a, cut_b[1], cut_rem[1], span * (blockIdx.x + 1), snap);
    walk.end = cut.unit;
  }
  walk.at.start(a, cut_b[0], cut_rem[0], span * blockIdx.x, blockIdx.x == 0 ? 0 : snap);
  bool ok = true;  // no wait of this role has run out
  bool some = walk.first(a);

  if (warp < 8) {
    // ---------------- softmax ----------------
    const int half = warp >> 2, row = tid & 127;  // this thread's row of the half
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tS + lanes + half * 64, p_at = tP + lanes + half * 32,
                   o_at = tO + lanes + half * D;
    uint8_t* const q_sm = sm + half * L::kQHalf;
    float unit = 0.f;  // from products to scores in units of log2(e)
    int lim = 0;       // the last position the row sees
    // the row's query: scaled so that its largest element is in [2^9, 2^10), as fp16, in the order
    // (0,4),(1,5),(2,6),(3,7) of each eight dimensions, which is the one K's decoding gives
    auto load_q = [&]() {
      const Request& r = walk.at.r;
      const int c = walk.at.part * kRows + half * 128 + row;
      uint4 v[D / 8];
      float top = 0.f;
      if (c < r.rows) {
        const int token = c / G;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(a.q) + static_cast<size_t>(r.row0 + token) * a.ldq +
            (walk.at.head * G + c - token * G) * D);
#pragma unroll
        for (int w = 0; w < D / 8; ++w) v[w] = __ldg(src + w);
        lim = r.kv - r.q_len + token;
      } else {
#pragma unroll
        for (int w = 0; w < D / 8; ++w) v[w] = make_uint4(0u, 0u, 0u, 0u);
        lim = r.kv - 1;  // (written nowhere)
      }
#pragma unroll
      for (int w = 0; w < D / 8; ++w) {
        const uint32_t x[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(bf16_lo(x[i])), fabsf(bf16_hi(x[i]))));
      }
      const int e = top > 0.f && top < INFINITY
                        ? min(120, 9 + 127 - static_cast<int>(__float_as_uint(top) >> 23))
                        : 0;
      const float up = copysignf(__uint_as_float(static_cast<uint32_t>(e + 127) << 23), a.scale_log2);
      // (never 0, so that a masked score stays -inf)
      unit = fmaxf(kKvUnit * fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23),
                   1e-30f);
#pragma unroll
      for (int w = 0; w < D / 8; ++w) {
        const uint32_t x[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
        const uint4 o = make_uint4(pack_f16x2(bf16_lo(x[0]) * up, bf16_lo(x[2]) * up),
                                   pack_f16x2(bf16_hi(x[0]) * up, bf16_hi(x[2]) * up),
                                   pack_f16x2(bf16_lo(x[1]) * up, bf16_lo(x[3]) * up),
                                   pack_f16x2(bf16_hi(x[1]) * up, bf16_hi(x[3]) * up));
        *reinterpret_cast<uint4*>(q_sm + (w >> 3) * (128 * 128) + row * 128 +
                                  (((w & 7) ^ (row & 7)) << 4)) = o;
      }
      fence_proxy_async_smem();
      mbar_arrive(&q_full[half]);
    };

    // the softmax warps wait for one another, bounded like every wait
    uint32_t meetings = 0;
    auto meet_all = [&]() {
      mbar_arrive(&meet);
      ok = mbar_wait(&meet, meetings++ & 1, a.err);
      ok = __all_sync(0xffffffffu, ok);
    };
    uint32_t tiles_done = 0, groups_done = 0;  // of this half
    bool active = some && (half == 0 || walk.second_half());
    if (active) load_q();
    while (some && ok) {
      const Walk now = walk;
      const int first_pos = now.at.tile * kTile;
      float m = kNone, l = 0.f;
      const float my_unit = unit;
      const int my_lim = lim;
      if (active) {
        for (int j = 0; j < now.count && ok; ++j, ++tiles_done) {
          ok = mbar_wait(&s_full[half], tiles_done & 1, a.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          uint32_t s[2][32];
          tmem_ld_32x32b_x32(s_at, s[0]);
          tmem_ld_32x32b_x32(s_at + 32, s[1]);
          tmem_ld_wait();
          const int left = my_lim - (first_pos + j * kTile);  // the tile's positions 0..left are seen
          if (__any_sync(0xffffffffu, left < kTile - 1)) {
#pragma unroll
            for (int i = 0; i < kTile; ++i)
              if (i > left) s[i >> 5][i & 31] = 0xFF800000u;
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kTile; ++i)
            top[i & 3] = fmaxf(top[i & 3], __uint_as_float(s[i >> 5][i & 31]));
          const float peak = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * my_unit;
          if (__any_sync(0xffffffffu, peak > m + (kRef + kSlack))) {
            const float moved = fmaxf(m, peak - kRef), f = ex2(m - moved);
            m = moved;
            l *= f;
            if (j > 0) {  // O of the tiles before: its products are done, S came after them
#pragma unroll
              for (int d = 0; d < D; d += 32) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(o_at + d, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st_32x32b_x32(o_at + d, o);
              }
            }
          }
          const float2 by = make_float2(my_unit, my_unit), minus = make_float2(-m, -m);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 x =
                fma2(make_float2(__uint_as_float(s[i >> 4][2 * i & 31]), __uint_as_float(s[i >> 4][(2 * i & 31) + 1])),
                     by, minus);
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            sum[i & 1] = add2(sum[i & 1], e);
            p[i] = pack_f16x2(e.x, e.y);
          }
          tmem_st_32x32b_x32(p_at, p);
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[half]);
        }
      }
      if (!ok) break;
      // the next segment's queries, while this one's last product runs
      some = walk.next(a);
      const bool next_active = some && (half == 0 || walk.second_half());
      if (next_active) load_q();

      if (active) {
        ok = mbar_wait(&o_full[half], groups_done & 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++groups_done;
        tc_fence_after();
      }
      const Request& r = now.at.r;
      const int c = now.at.part * kRows + half * 128 + row;
      const long long group = now.at.unit - now.at.tile;
      const bool whole = now.at.tile == 0 && now.count == now.at.tiles;
      // this CTA's piece of a group it shares: 0 began before it, 1 goes on after it
      float* const piece = a.prompt_pieces +
                           static_cast<size_t>(blockIdx.x * 2 + (now.at.tile > 0 ? 0 : 1)) * piece_floats<D>();
      if (active) {
        const int token = c / G;
        const float f = whole ? (l == 0.f ? 0.f : kKvUnit * a.v_scale / l) : 1.f;
        uint4* out = reinterpret_cast<uint4*>(
            static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(r.row0 + token) * a.ldo +
            (now.at.head * G + c - token * G) * D);
        float4* part_out = reinterpret_cast<float4*>(piece + 2 * kRows + (half * 128 + row) * D);
#pragma unroll
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(o_at + d, o);
          tmem_ld_wait();
          if (c < r.rows && whole) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[i] = pack_bf16x2(__uint_as_float(o[8 * w + 2 * i]) * f, __uint_as_float(o[8 * w + 2 * i + 1]) * f);
              out[d / 8 + w] = make_uint4(x[0], x[1], x[2], x[3]);
            }
          } else if (c < r.rows) {
#pragma unroll
            for (int w = 0; w < 8; ++w)
              part_out[d / 4 + w] =
                  make_float4(__uint_as_float(o[4 * w]), __uint_as_float(o[4 * w + 1]),
                              __uint_as_float(o[4 * w + 2]), __uint_as_float(o[4 * w + 3]));
          }
          __syncwarp();
        }
        tc_fence_before();
        if (!whole) {
          piece[half * 128 + row] = m;
          piece[kRows + half * 128 + row] = l;
        }
      }
      if (!whole) {
        // The cuts within the group, as their CTAs see them, and the pieces between them: the
        // first cut's CTA before it (piece 1), then pieces 0.
        const int first_cut = static_cast<int>(quotient(group + snap, span)) + 1;
        const int last_cut = static_cast<int>(quotient(group + now.at.tiles - snap + span - 1, span)) - 1;
        const int n = last_cut - first_cut + 2;
        __threadfence();
        meet_all();
        if (!ok) break;
        if (tid == 0) {
          last_cta = atomicAdd(a.prompt_arrivals + first_cut, 1) == n - 1;
          if (last_cta) a.prompt_arrivals[first_cut] = 0;
          __threadfence();
        }
        meet_all();
        if (!ok) break;
        if (last_cta) {
          const auto piece_of = [&](int i) {
            return a.prompt_pieces +
                   static_cast<size_t>(i == 0 ? (first_cut - 1) * 2 + 1 : (first_cut + i - 1) * 2) * piece_floats<D>();
          };
          const int rows = min(kRows, r.rows - now.at.part * kRows);
          for (int x = warp; x < rows; x += 8) {
            float top = kNone;
            for (int i = lane; i < n; i += 32) top = fmaxf(top, __ldcg(piece_of(i) + x));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            float sum = 0.f, o[D / 32] = {};
            for (int i0 = 0; i0 < n; i0 += 32) {
              float f = 0.f;
              if (i0 + lane < n) {
                f = ex2(__ldcg(piece_of(i0 + lane) + x) - top);
                sum += f * __ldcg(piece_of(i0 + lane) + kRows + x);
              }
              const int some_pieces = min(32, n - i0);
#pragma unroll 4
              for (int k = 0; k < some_pieces; ++k) {
                const float w = __shfl_sync(0xffffffffu, f, k);
                const float* p = piece_of(i0 + k) + 2 * kRows + x * D + lane * (D / 32);
#pragma unroll
                for (int d = 0; d < D / 32; d += 2) {
                  const float2 y = __ldcg(reinterpret_cast<const float2*>(p + d));
                  o[d] += w * y.x;
                  o[d + 1] += w * y.y;
                }
              }
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const float f = sum == 0.f ? 0.f : kKvUnit * a.v_scale / sum;
            const int at = now.at.part * kRows + x, token = at / G;
            uint32_t* out = reinterpret_cast<uint32_t*>(
                static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(r.row0 + token) * a.ldo +
                (now.at.head * G + at - token * G) * D + lane * (D / 32));
#pragma unroll
            for (int d = 0; d < D / 32; d += 2) out[d / 2] = pack_bf16x2(o[d] * f, o[d + 1] * f);
          }
        }
        meet_all();  // last_cta is read
      }
      active = next_active;
    }
  } else if (warp < 12) {
    // ---------------- decoding ----------------
    const int t = tid - 256;                   // 0..127
    const int k_token = t & 63, k_part = t >> 6;  // K: one token's half of the dimensions
    const int v_oct = t & 7, v_dims = t >> 3;  // V: 8 tokens x 8 dimensions
    const bool v_mine = v_dims < D / 8;
    const int shift = a.pages.page_shift;
    uint32_t n = 0;  // tiles decoded
    while (some && ok) {
      const Request& r = walk.at.r;
      const int32_t* row = a.table + static_cast<size_t>(walk.at.b) * a.max_blocks;
      const int last = max(0, (r.kv - 1) >> shift);  // the request's last page
      // the page of position pos (of the last page past the end: masked, and within the cache)
      auto page_of = [&](int pos) {
        int id = r.kv > 0 ? __ldg(row + min(pos >> shift, last)) : 0;
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.pages.num_pages)) {
          atomicOr(a.err, LORA_ERRF_BAD_ID);
          id = 0;
        }
        return id;
      };
      auto block_of = [&](int page, int pos) {
        return a.pages.base +
               a.pages.block(page, walk.at.head, (pos & ((1 << shift) - 1)) / kKvBlock);
      };
      constexpr int KW = D / 16;  // words of K a thread decodes
      uint32_t kw[KW], ks[D / 64 * 2], vw[8], vs[4];
      auto fetch = [&](int j) {
        const int kp = (walk.at.tile + j) * kTile + k_token;
        const uint8_t* blk = block_of(page_of(kp), kp);
        const int kt = kp & 15, fr = kv_token_frag(kt);
        const uint4* src = reinterpret_cast<const uint4*>(blk + kt * (D / 2) + k_part * (D / 4));
#pragma unroll
        for (int w = 0; w < KW / 4; ++w) {
          const uint4 x = __ldg(src + w);
          kw[4 * w] = x.x, kw[4 * w + 1] = x.y, kw[4 * w + 2] = x.z, kw[4 * w + 3] = x.w;
        }
        // scales of the thread's D / 32 groups; see kv_k_scale_at
        if constexpr (D == 128) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(blk + kv_k_scales(D) + (fr & 7) * 16 + k_part * 8));
          ks[0] = x.x >> (16 * (fr >> 3));
          ks[1] = x.y >> (16 * (fr >> 3));
        } else {
          const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(blk + kv_k_scales(D) + (fr & 7) * 8 + k_part * 4));
          ks[0] = x >> (8 * (fr >> 3));  // bytes 0 and 2
        }
        const int vp = (walk.at.tile + j) * kTile + v_oct * 8;
        if (v_mine) {
          const uint8_t* vb = block_of(page_of(vp), vp);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            vw[i] = __ldg(reinterpret_cast<const uint32_t*>(vb + kv_v_code_at(D, (vp & 8) + i, v_dims * 4)));
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(vb + kv_v_scales(D) + (v_dims / 2) * 16));
          const int sh = 16 * ((vp & 8) >> 3);  // bytes 0, 1: tokens with bit 2 clear and set
          vs[0] = x.x >> sh, vs[1] = x.y >> sh, vs[2] = x.z >> sh, vs[3] = x.w >> sh;
        }
      };
      fetch(0);
      for (int j = 0; j < walk.count; ++j, ++n) {
        const int stage = n % kStages, parity = (n / kStages) & 1;
        ok = mbar_wait(&k_empty[stage], parity ^ 1, a.err) && mbar_wait(&v_empty[stage], parity ^ 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // K: rows of tokens
        uint8_t* k_sm = sm + L::kK + stage * L::kKv;
#pragma unroll
        for (int g = 0; g < KW / 2; ++g) {  // scale groups of two words
          uint32_t sc;
          if constexpr (D == 128) {
            const uint32_t two = e4m3x2_to_f16x2(static_cast<uint16_t>(ks[g >> 1]));
            sc = g & 1 ? both_hi(two) : both_lo(two);
          } else {
            sc = both_lo(e4m3x2_to_f16x2(static_cast<uint16_t>(ks[0] >> (16 * g))));
          }
          const Decode dec = decode_scales(sc);
#pragma unroll
          for (int w = 2 * g; w < 2 * g + 2; ++w) {
            uint32_t o[4];
            decode4(kw[w], dec, o);
            const int chunk = k_part * KW + w;  // of 8 dimensions
            *reinterpret_cast<uint4*>(k_sm + (chunk >> 3) * (kTile * 128) + k_token * 128 +
                                      (((chunk & 7) ^ (k_token & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&k_full[stage]);
        // V: rows of dimensions, 8 tokens a chunk
        if (v_mine) {
          uint8_t* v_sm = sm + L::kV + stage * L::kKv;
          Decode dec[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // tokens 2i, 2i + 1: bit 2 is i >> 1, bit 1 is i & 1
            const int b2 = i >> 1, t0 = b2 | (i & 1) << 1, t1 = t0 ^ 1;
            dec[i] = decode_scales(
                e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(vs[t0], vs[t1], b2 ? 0x0051 : 0x0040))));
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {  // dimensions 0..3 and 4..7
            uint32_t o[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              decode4(prmt(vw[2 * i], vw[2 * i + 1], hf ? 0x7632 : 0x5410), dec[i], o[i]);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const int dim = v_dims * 8 + hf * 4 + d;
              *reinterpret_cast<uint4*>(v_sm + dim * 128 + ((v_oct ^ (dim & 7)) << 4)) =
                  make_uint4(o[0][d], o[1][d], o[2][d], o[3][d]);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&v_full[stage]);
        if (j + 1 < walk.count) fetch(j + 1);
      }
      if (!ok) break;
      some = walk.next(a);
    }
  } else {
    // ---------------- products ----------------
    constexpr uint32_t kQkDesc = idesc_f16_f32(128, kTile), kPvDesc = idesc_f16_f32(128, D);
    uint32_t n = 0;                                      // tiles
    uint32_t groups[2] = {0, 0}, halves[2] = {0, 0};     // segments and tiles of each half
    const uint32_t q_addr = smem_u32(sm), k_addr = q_addr + L::kK, v_addr = q_addr + L::kV;
    auto qk = [&](int h, uint32_t stage) {
      if (lane == 0) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_bf16(tS + h * 64,
                      smem_desc_sw128(q_addr + h * L::kQHalf + (ks >> 2) * (128 * 128) + (ks & 3) * 32),
                      smem_desc_sw128(k_addr + stage * L::kKv + (ks >> 2) * (kTile * 128) + (ks & 3) * 32),
                      kQkDesc, ks > 0);
        tc_commit(&s_full[h]);
      }
      __syncwarp();
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = mbar_wait(bar, parity & 1, a.err);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      return ok;
    };
    while (some && ok) {
      const int nh = walk.second_half() ? 2 : 1;
      const int count = walk.count;
      if (!wait(&k_full[n % kStages], n / kStages)) break;
      for (int h = 0; h < nh && ok; ++h) {
        if (!wait(&q_full[h], groups[h]++)) break;
        qk(h, n % kStages);
      }
      if (!ok) break;
      if (lane == 0) tc_commit(&k_empty[n % kStages]);
      __syncwarp();
      for (int j = 0; j < count && ok; ++j, ++n) {
        const uint32_t stage = n % kStages, next = (n + 1) % kStages;
        const bool more = j + 1 < count;
        if (!wait(&v_full[stage], n / kStages)) break;
        for (int h = 0; h < nh; ++h) {
          if (!wait(&p_full[h], halves[h]++)) break;
          if (lane == 0) {
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              tc_mma_f16_ts(tO + h * D, tP + h * 32 + ks * 8,
                            smem_desc_sw128(v_addr + stage * L::kKv + ks * 32), kPvDesc, j > 0 || ks > 0);
            if (h == nh - 1) tc_commit(&v_empty[stage]);
            if (!more) tc_commit(&o_full[h]);
          }
          __syncwarp();
          if (more) {
            if (h == 0 && !wait(&k_full[next], (n + 1) / kStages)) break;
            qk(h, next);
            if (h == nh - 1 && lane == 0) tc_commit(&k_empty[next]);
            __syncwarp();
          }
        }
      }
      if (!ok) break;
      some = walk.next(a);
    }
    // every product issued is done before the CTA's memory goes
    if (lane == 0) tc_commit(&idle);
    mbar_wait(&idle, 0, a.err);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, kTmemCols);
}

template <int D>
cudaError_t launch(const KvAttendArgs& a, cudaStream_t stream) {
  static int limit[kAttrDevices] = {};
  cudaError_t e = ensure_smem_limit(kv_prompt_kernel<D>, Smem<D>::kBytes, limit);
  if (e != cudaSuccess) return e;
  kv_prompt_kernel<D><<<std::min(kKvMaxCtas, a.num_sms), kThreads, Smem<D>::kBytes, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv_prompt_workspace_floats(int num_sms, int D) {
  return static_cast<size_t>(std::min(kKvMaxCtas, num_sms)) * 2 *
         (D == 128 ? piece_floats<128>() : piece_floats<64>());
}

cudaError_t launch_kv_prompt(const KvAttendArgs& a, cudaStream_t stream) {
  return a.pages.D == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace lora
