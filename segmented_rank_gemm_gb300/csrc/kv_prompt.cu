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
//   warps 12, 13     issue the products of a half each: PV and the next QK of one half run while
//                    the other half's softmax does
//   warp 14          fetches packed tiles by bulk copies, kRaw tiles ahead
// 256 rows share one decoding.  Tensor memory holds S of two tiles and O of both halves
// (2 x 2 x 64 + 2 x 128 columns at D = 128), so that the softmax finds the next S done; P takes
// the first columns of its S, and the next S but one waits for the product that reads it.
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

constexpr int kThreads = 16 * 32;  // four warpgroups, which split the registers unevenly
constexpr int kRows = 256;      // rows of a group, two halves
constexpr int kTile = 64;       // positions of a tile
constexpr int kStages = 3;      // decoded tiles of K, and of V
constexpr int kRaw = 4;         // packed tiles
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

// The warpgroups' shares of the registers: 2 x 168 + 112 + 64 = 4 x 128, what the CTA is
// launched with.
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
  r.rows = r.q_len * a.group;
  if (r.rows <= a.few_rows) r.rows = 0;
  r.parts = (r.rows + kRows - 1) / kRows;
  return r;
}
// Tiles of a request's group `part`: up to the last position its last row sees.
__device__ __forceinline__ int group_tiles(const KvAttendArgs& a, const Request& r, int part) {
  const int last = r.kv - r.q_len + a.token_of(min((part + 1) * kRows, r.rows) - 1);
  return max(1, (last + kTile) / kTile);
}
// Units of one head of a request, and of the first parts of it, by the lanes of a warp.
__device__ __forceinline__ int part_units(const KvAttendArgs& a, const Request& r, int part) {
  return part < r.parts ? group_tiles(a, r, part) + kSetup : 0;
}
__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ long long head_units(const KvAttendArgs& a, const Request& r, int lane) {
  long long n = 0;
  for (int part = lane; part < r.parts; part += 32) n += part_units(a, r, part);
  return warp_sum(n);
}

// A position in the sequence of tiles, and the tile's unit.
struct Cursor {
  Request r;
  int b, head, part, tile, tiles;
  long long unit;
  // The tile at or after unit `at`, the rem-th of request b_; a cut near a group's edge moves
  // there (to the group's end by tile = tiles, one past its last).  One warp.
  __device__ __forceinline__ void start(const KvAttendArgs& a, int b_, long long rem, long long at,
                                        int snap, int lane) {
    b = b_;
    r = load_request(a, b);
    const long long per = head_units(a, r, lane);
    head = static_cast<int>(quotient(rem, per));
    rem -= head * per;
    for (part = 0;; part += 32) {
      long long incl = part_units(a, r, part + lane);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      const unsigned beyond = __ballot_sync(0xffffffffu, rem < incl);
      const long long all = __shfl_sync(0xffffffffu, incl, 31);
      if (beyond || part + 32 >= r.parts) {
        const int k = beyond ? __ffs(beyond) - 1 : 0;
        const long long first = __shfl_sync(0xffffffffu, incl, max(k - 1, 0));
        part += k;
        if (k > 0) rem -= first;
        break;
      }
      rem -= all;
    }
    tiles = group_tiles(a, r, part);
    const int off = static_cast<int>(rem);
    if (off <= kSetup + snap) {
      tile = 0;
    } else {
      tile = tiles + kSetup - off <= snap ? tiles : off - kSetup;
    }
    unit = at - off + kSetup + tile;
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
    if (at.tile == at.tiles) {  // the start moved to its group's end
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
  static constexpr int kRawTile = kTile / kKvBlock * kv_block_bytes(D);
  static constexpr int kRaws = kV + kStages * kKv;
  static constexpr int kScratch = kRaws + kRaw * kRawTile;
  static constexpr int kBytes = kScratch + 8 * 2048 + 1024;  // + alignment
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(KvAttendArgs a) {
  using L = Smem<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* const sm = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  // The barriers of a half's tiles alternate: a wait is then for the barrier's latest phase or the
  // one under way, never two phases back.
  __shared__ uint64_t q_full[2], s_full[2][2], p_full[2][2], pv_done[2][2];  // [half][tile parity]
  __shared__ uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  __shared__ uint64_t raw_full[kRaw], raw_empty[kRaw];
  __shared__ uint64_t idle[2], meet;
  __shared__ uint32_t tmem_holder;
  __shared__ long long scan[kThreads / 32], cut_rem[2];
  __shared__ float row_unit[kRows];  // a row's factor from products to scores in units of log2(e)
  __shared__ int cut_b[2];
  __shared__ Cursor cuts[2];
  __shared__ int last_cta;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = a.pages.heads, G = a.group;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 128);
      for (int k = 0; k < 2; ++k) {
        mbar_init(&pv_done[i][k], 1);
        mbar_init(&s_full[i][k], 1);
        mbar_init(&p_full[i][k], 128);
      }
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&k_empty[i], 2);
      mbar_init(&v_full[i], 128);
      mbar_init(&v_empty[i], 2);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 128);
    }
    mbar_init(&idle[0], 1);
    mbar_init(&idle[1], 1);
    mbar_init(&meet, 256);
    fence_mbar_init();
  }

  // The sequence's length and this CTA's cuts.  A thread sums a run of consecutive requests; those
  // with many groups are summed by its warp.
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  const auto request_units = [&](int b, bool mine) {  // of request b (mine), by all lanes
    Request r = {};
    if (mine) r = load_request(a, b);
    long long n = 0;
    if (r.parts <= 4)
      for (int part = 0; part < r.parts; ++part) n += part_units(a, r, part);
    for (unsigned big = __ballot_sync(0xffffffffu, r.parts > 4); big; big &= big - 1) {
      const int k = __ffs(big) - 1;
      Request x;
      x.kv = __shfl_sync(0xffffffffu, r.kv, k);
      x.q_len = __shfl_sync(0xffffffffu, r.q_len, k);
      x.rows = __shfl_sync(0xffffffffu, r.rows, k);
      x.parts = __shfl_sync(0xffffffffu, r.parts, k);
      const long long sum = head_units(a, x, lane);
      if (lane == k) n = sum;
    }
    return n * heads;
  };
  long long mine = 0, last_units = 0;
  for (int i = 0; i < per; ++i) {
    last_units = request_units(b0 + i, b0 + i < b1);
    mine += last_units;
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long total = 0, before = incl - mine;
#pragma unroll
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
    const bool here = at >= before && at < before + mine;
    if (per > 1 && __any_sync(0xffffffffu, here)) {
      long long rem = at - before;
      int b = b0;
      for (int k = 0; k < per - 1; ++k) {  // (the run's last takes what is left)
        const bool go = here && b == b0 + k && b < b1 - 1;
        const long long n = request_units(b0 + k, go);
        if (go && rem >= n) {
          rem -= n;
          ++b;
        }
      }
      if (here) cut_b[i] = b, cut_rem[i] = rem;
    } else if (here) {
      cut_b[i] = b0, cut_rem[i] = at - before;
    }
  }
  if (warp == 12) tmem_alloc(&tmem_holder, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  if (warp < 2) {  // warp 0: where the range starts; warp 1: where it ends
    const long long at = span * (blockIdx.x + warp);
    if (at < total) {
      Cursor cut;
      cut.start(a, cut_b[warp], cut_rem[warp], at, blockIdx.x + warp == 0 ? 0 : snap, lane);
      if (lane == 0) cuts[warp] = cut;
    } else if (lane == 0) {
      cuts[warp].unit = total;
    }
  }
  __syncthreads();
  // S: two tiles of each half, 64 columns each, whose first 32 become P; O behind them
  const uint32_t tS = tmem, tO = tmem + 256;

  Walk walk;
  walk.at = cuts[0];
  walk.end = cuts[1].unit;
  bool ok = true;  // no wait of this role has run out
  bool some = walk.first(a);

  // (one instruction a warpgroup)
  if (warp < 8) setmaxnreg_inc<168>();
  else if (warp < 12) setmaxnreg_dec<112>();
  else setmaxnreg_dec<64>();

  if (warp < 8) {
    // ---------------- softmax ----------------
    const int half = warp >> 2, row = tid & 127;  // this thread's row of the half
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tS + lanes + half * 128, o_at = tO + lanes + half * D;
    uint8_t* const q_sm = sm + half * L::kQHalf;
    uint8_t* const scratch = sm + L::kScratch + warp * 2048;  // 32 rows of 64 bytes
    float unit = 0.f;  // this row's row_unit
    int lim = 0;       // the last position it sees
    // The queries of the warp's 32 rows, a row's 16-byte pieces on consecutive lanes: scaled so that
    // the row's largest element is in [2^9, 2^10), as fp16, in the order (0,4),(1,5),(2,6),(3,7)
    // of each eight dimensions, which is the one K's decoding gives.
    auto load_q = [&]() {
      constexpr int LR = D / 8, RI = 32 / LR;  // lanes a row, rows a step
      const Request& r = walk.at.r;
      const int c0 = walk.at.part * kRows + half * 128;
      const int w = lane % LR, sub = lane / LR;
      uint4 v[32 / RI];
#pragma unroll
      for (int i = 0; i < 32 / RI; ++i) {
        const int c = c0 + (warp & 3) * 32 + i * RI + sub, token = a.token_of(c);
        v[i] = c < r.rows
                   ? __ldg(reinterpret_cast<const uint4*>(
                               static_cast<const __nv_bfloat16*>(a.q) +
                               static_cast<size_t>(r.row0 + token) * a.ldq +
                               (walk.at.head * G + c - token * G) * D) + w)
                   : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < 32 / RI; ++i) {
        const int at = (warp & 3) * 32 + i * RI + sub;
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(bf16_lo(x[k])), fabsf(bf16_hi(x[k]))));
#pragma unroll
        for (int d = LR / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int e = top > 0.f && top < INFINITY
                          ? min(120, 9 + 127 - static_cast<int>(__float_as_uint(top) >> 23))
                          : 0;
        const float up = copysignf(__uint_as_float(static_cast<uint32_t>(e + 127) << 23), a.scale_log2);
        // (never 0, so that a masked score stays -inf)
        if (w == 0)
          row_unit[half * 128 + at] = fmaxf(
              kKvUnit * fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23), 1e-30f);
        *reinterpret_cast<uint4*>(q_sm + (w >> 3) * (128 * 128) + at * 128 + (((w & 7) ^ (at & 7)) << 4)) =
            make_uint4(pack_f16x2(bf16_lo(x[0]) * up, bf16_lo(x[2]) * up),
                       pack_f16x2(bf16_hi(x[0]) * up, bf16_hi(x[2]) * up),
                       pack_f16x2(bf16_lo(x[1]) * up, bf16_lo(x[3]) * up),
                       pack_f16x2(bf16_hi(x[1]) * up, bf16_hi(x[3]) * up));
      }
      fence_proxy_async_smem();
      mbar_arrive(&q_full[half]);
      __syncwarp();
      unit = row_unit[half * 128 + row];
      const int c = c0 + row;  // (a row past the last is written nowhere)
      lim = c < r.rows ? r.kv - r.q_len + a.token_of(c) : r.kv - 1;
    };
    // the softmax warps wait for one another, bounded like every wait
    uint32_t meetings = 0;
    auto meet_all = [&]() {
      mbar_arrive(&meet);
      ok = mbar_wait(&meet, meetings++ & 1, a.err);
      ok = __all_sync(0xffffffffu, ok);
    };
    uint32_t n = 0;  // tiles of this half
    bool active = some && (half == 0 || walk.second_half());
    if (active) load_q();
    while (some && ok) {
      const Walk now = walk;
      const int first_pos = now.at.tile * kTile;
      float m = kNone, l = 0.f;
      const float my_unit = unit;
      const int my_lim = lim;
      if (active) {
        for (int j = 0; j < now.count; ++j, ++n) {
          ok = mbar_wait(&s_full[half][n & 1], n >> 1 & 1, a.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = s_at + (n & 1) * 64;
          uint32_t s[2][32];
          tmem_ld_32x32b_x32(at, s[0]);
          tmem_ld_32x32b_x32(at + 32, s[1]);
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
            if (j > 0) {  // O of the tiles before, once their products are done
              ok = mbar_wait(&pv_done[half][(n - 1) & 1], (n - 1) >> 1 & 1, a.err);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
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
          tmem_st_32x32b_x32(at, p);
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[half][n & 1]);
        }
      }
      if (!ok) break;
      // the next segment's queries, while this one's last products run
      some = walk.next(a);
      const bool next_active = some && (half == 0 || walk.second_half());
      if (next_active) load_q();

      if (active) {
        ok = mbar_wait(&pv_done[half][(n - 1) & 1], (n - 1) >> 1 & 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      const Request& r = now.at.r;
      const int c0 = now.at.part * kRows;
      const long long group = now.at.unit - now.at.tile;
      const bool whole = now.at.tile == 0 && now.count == now.at.tiles;
      // this CTA's piece of a group it shares: 0 began before it, 1 goes on after it
      float* const piece = a.prompt_pieces +
                           static_cast<size_t>(blockIdx.x * 2 + (now.at.tile > 0 ? 0 : 1)) * piece_floats<D>();
      if (active) {
        // 64 bytes of every row at a time, from one row a lane to 4 lanes a row
        const float f = whole ? (l == 0.f ? 0.f : kKvUnit * a.v_scale / l) : 1.f;
        const int step = whole ? 32 : 16;  // dimensions
        const auto at = [&](int x, int k) {  // 16-byte piece k of row x
          return reinterpret_cast<uint4*>(scratch + x * 64 + ((k ^ (x >> 1 & 3)) << 4));
        };
        uint8_t* dst[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = (warp & 3) * 32 + i * 8 + (lane >> 2), c = c0 + half * 128 + x, token = a.token_of(c);
          dst[i] = nullptr;
          if (c < r.rows)
            dst[i] = (whole ? reinterpret_cast<uint8_t*>(static_cast<__nv_bfloat16*>(a.out) +
                                                         static_cast<size_t>(r.row0 + token) * a.ldo +
                                                         (now.at.head * G + c - token * G) * D)
                            : reinterpret_cast<uint8_t*>(piece + 2 * kRows + (half * 128 + x) * D)) +
                     (lane & 3) * 16;
        }
#pragma unroll 1
        for (int d = 0; d < D; d += step) {
          uint32_t o[32];
          if (whole) {
            tmem_ld_32x32b_x32(o_at + d, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * f, __uint_as_float(o[2 * i + 1]) * f);
          } else {
            uint32_t part[16];
            tmem_ld_32x32b_x16(o_at + d, part);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = part[i];
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *at(lane, k) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (dst[i]) {
              *reinterpret_cast<uint4*>(dst[i]) = *at(i * 8 + (lane >> 2), lane & 3);
              dst[i] += 64;
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
            const int at = now.at.part * kRows + x, token = a.token_of(at);
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
    // Lanes are dealt so that the reads of a packed tile, the writes of K's rows and those of V's
    // transposed rows all go to different banks:
    //   K  a thread decodes 32 dimensions (16 bytes) of one token, or of two 32 apart
    //   V  a thread decodes 8 tokens (octet vo) x 8 dimensions (vd); odd octets read each pair of
    //      tokens the other way round, and odd vd decode their upper four dimensions first
    constexpr int KC = D / 32;              // 16-byte pieces of a K row
    constexpr int KT = kTile * KC / 128;    // tokens of a thread, 128 / KC apart
    const int t = tid - 256;                // 0..127
    const int kt = t / KC, kc = t % KC;
    const int w = t >> 5;
    const int vo = (lane & 3) | (w & 1) << 2;
    const int vd = (lane >> 2) | (D == 128 ? ((w >> 1) ^ (lane >> 1 & 1)) << 3 : 0);
    const bool v_mine = D == 128 || w < 2;
    const int v_half = vo & 1;              // token of the octet's block half
    const uint32_t sel_lo = vo & 1 ? 0x1054u : 0x5410u, sel_hi = vo & 1 ? 0x3276u : 0x7632u;
    const uint32_t sel[2] = {vd & 1 ? sel_hi : sel_lo, vd & 1 ? sel_lo : sel_hi};
    const bool swap = D == 128 && kc >= 2;  // these lanes decode their last 16 dimensions first
    uint32_t n = 0;  // tiles decoded
    while (some && ok) {
      for (int j = 0; j < walk.count; ++j, ++n) {
        const int stage = n % kStages, parity = (n / kStages) & 1, slot = n % kRaw;
        ok = mbar_wait(&raw_full[slot], (n / kRaw) & 1, a.err);
        const uint8_t* const tile = sm + L::kRaws + slot * L::kRawTile;
        uint32_t kw[KT][4], ks[KT];  // ks: the two groups' scales as fp16
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          const int token = kt + i * (128 / KC), in = token & 15, fr = kv_token_frag(in);
          const uint8_t* blk = tile + (token >> 4) * kv_block_bytes(D);
          const uint4 x = *reinterpret_cast<const uint4*>(blk + in * (D / 2) + kc * 16);
          kw[i][0] = swap ? x.z : x.x, kw[i][1] = swap ? x.w : x.y;
          kw[i][2] = swap ? x.x : x.z, kw[i][3] = swap ? x.y : x.w;
          if constexpr (D == 128) {
            const uint32_t two = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(
                blk + kv_k_scales(D) + (fr & 7) * 16 + kc * 4 + (fr >> 3) * 2));
            ks[i] = swap ? prmt(two, two, 0x1032) : two;
          } else {
            const uint32_t x4 =
                *reinterpret_cast<const uint32_t*>(blk + kv_k_scales(D) + (fr & 7) * 8 + kc * 4) >>
                (8 * (fr >> 3));
            ks[i] = e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(x4, 0u, 0x4420)));
          }
        }
        uint32_t vw[8], vs[4];
        if (v_mine) {
          const uint8_t* blk = tile + (vo >> 1) * kv_block_bytes(D);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            vw[i] = *reinterpret_cast<const uint32_t*>(blk + kv_v_code_at(D, v_half * 8 + (i ^ v_half), vd * 4));
          const uint4 x = *reinterpret_cast<const uint4*>(blk + kv_v_scales(D) + (vd >> 1) * 16);
          const int sh = 16 * v_half;  // then bytes 0, 1: tokens with bit 2 clear and set
          vs[0] = x.x >> sh, vs[1] = x.y >> sh, vs[2] = x.z >> sh, vs[3] = x.w >> sh;
        }
        mbar_arrive(&raw_empty[slot]);
        ok = ok && mbar_wait(&k_empty[stage], parity ^ 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // K: rows of tokens
        uint8_t* const k_sm = sm + L::kK + stage * L::kKv;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          const int token = kt + i * (128 / KC);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const Decode dec = decode_scales(g ? both_hi(ks[i]) : both_lo(ks[i]));
#pragma unroll
            for (int x = 2 * g; x < 2 * g + 2; ++x) {
              uint32_t o[4];
              decode4(kw[i][x], dec, o);
              const int chunk = kc * 4 + (swap ? x ^ 2 : x);  // of 8 dimensions
              *reinterpret_cast<uint4*>(k_sm + (chunk >> 3) * (kTile * 128) + token * 128 +
                                        (((chunk & 7) ^ (token & 7)) << 4)) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&k_full[stage]);
        // V: rows of dimensions, 8 tokens a chunk
        ok = mbar_wait(&v_empty[stage], parity ^ 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (v_mine) {
          uint8_t* const v_sm = sm + L::kV + stage * L::kKv;
          Decode dec[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // tokens 2i, 2i + 1: bit 2 is i >> 1, bit 1 is i & 1
            const int b2 = i >> 1, t0 = b2 | (i & 1) << 1, t1 = t0 ^ 1;
            dec[i] = decode_scales(
                e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(vs[t0], vs[t1], b2 ? 0x0051 : 0x0040))));
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {  // four dimensions at a time
            uint32_t o[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) decode4(prmt(vw[2 * i], vw[2 * i + 1], sel[hf]), dec[i], o[i]);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const int dim = vd * 8 + ((hf ^ vd) & 1) * 4 + d;
              *reinterpret_cast<uint4*>(v_sm + dim * 128 + ((vo ^ (dim & 7)) << 4)) =
                  make_uint4(o[0][d], o[1][d], o[2][d], o[3][d]);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&v_full[stage]);
      }
      if (!ok) break;
      some = walk.next(a);
    }
  } else if (warp == 14) {
    // ---------------- fetching ----------------
    const int shift = a.pages.page_shift;
    const int step = min(kTile, 1 << shift);          // positions of a copy
    const bool mine = lane * kKvBlock < kTile && lane * kKvBlock % step == 0;
    const uint32_t bytes = step / kKvBlock * kv_block_bytes(D);
    uint32_t n = 0;
    const auto prefetch_q = [&](const Cursor& at) {  // a group's queries to L2
      const int first = a.token_of(at.part * kRows), last = a.token_of(min((at.part + 1) * kRows, at.r.rows) - 1);
      for (int token = first + lane; token <= last; token += 32)
        bulk_prefetch_l2(static_cast<const __nv_bfloat16*>(a.q) + static_cast<size_t>(at.r.row0 + token) * a.ldq +
                             at.head * G * D,
                         G * D * 2);
    };
    while (some && ok) {
      Walk ahead = walk;
      if (ahead.next(a)) prefetch_q(ahead.at);
      const Request& r = walk.at.r;
      const int32_t* row = a.table + static_cast<size_t>(walk.at.b) * a.max_blocks;
      const int last = max(0, (r.kv - 1) >> shift);  // the request's last page
      // the page of position pos (of the last page past the end: masked, and within the cache)
      auto page_of = [&](int j) {
        const int pos = (walk.at.tile + j) * kTile + lane * kKvBlock;
        return mine && r.kv > 0 ? __ldg(row + min(pos >> shift, last)) : 0;
      };
      int id = page_of(0);
      for (int j = 0; j < walk.count; ++j, ++n) {
        const int slot = n % kRaw;
        const int next_id = j + 1 < walk.count ? page_of(j + 1) : 0;
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.pages.num_pages)) {
          atomicOr(a.err, LORA_ERRF_BAD_ID);
          id = 0;
        }
        ok = mbar_wait(&raw_empty[slot], ((n / kRaw) & 1) ^ 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&raw_full[slot], L::kRawTile);
        __syncwarp();
        if (mine) {
          const int pos = (walk.at.tile + j) * kTile + lane * kKvBlock;
          bulk_load_g2s(sm + L::kRaws + slot * L::kRawTile + lane * kv_block_bytes(D),
                        a.pages.base + a.pages.block(id, walk.at.head, (pos & ((1 << shift) - 1)) / kKvBlock),
                        bytes, &raw_full[slot]);
        }
        id = next_id;
      }
      if (!ok) break;
      some = walk.next(a);
    }
    // copies in flight write this CTA's memory: every one issued has landed when its slot's
    // barrier has turned
    for (uint32_t i = n > kRaw ? n - kRaw : 0; i < n; ++i)
      mbar_wait(&raw_full[i % kRaw], (i / kRaw) & 1, a.err);
  } else if (warp < 14 && lane == 0) {
    // ---------------- products ----------------
    // One thread a half, so that one half's waits and commits pass while the other's products
    // run; descriptors advance by constants, 32 bytes (2 units) a 16-wide step.
    constexpr uint32_t kQkDesc = idesc_f16_f32(128, kTile), kPvDesc = idesc_f16_f32(128, D);
    const int half = warp - 12;
    const uint32_t s_at = tS + half * 128, o_at = tO + half * D;
    const uint32_t base = smem_u32(sm);
    const uint64_t q_desc = smem_desc_sw128(base + half * L::kQHalf),
                   k_desc = smem_desc_sw128(base + L::kK), v_desc = smem_desc_sw128(base + L::kV);
    uint32_t k_stage = 0, k_turn = 0, v_stage = 0, v_turn = 0;  // of the next tiles
    uint32_t groups_done = 0, n = 0;                            // groups and PV products of this half
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && mbar_wait(bar, parity & 1, a.err);
      tc_fence_after();
      return ok;
    };
    const auto qk = [&](uint32_t tile) {  // S of the half's tile, whose K is the next stage
      if (!wait(&k_full[k_stage], k_turn)) return;
      uint64_t qd = q_desc, kd = k_desc + k_stage * (L::kKv >> 4);
#pragma unroll
      for (int slab = 0; slab < D / 64; ++slab) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma_bf16(s_at + (tile & 1) * 64, qd + ks * 2, kd + ks * 2, kQkDesc, slab > 0 || ks > 0);
        qd += 128 * 128 >> 4;
        kd += kTile * 128 >> 4;
      }
      tc_commit(&s_full[half][tile & 1]);
      tc_commit(&k_empty[k_stage]);
      if (++k_stage == kStages) k_stage = 0, ++k_turn;
    };
    while (some && ok) {
      const int count = walk.count;
      if (half == 1 && !walk.second_half()) {
        // no rows: the stages pass by
        for (int j = 0; j < count; ++j) {
          if (!wait(&k_full[k_stage], k_turn) || !wait(&v_full[v_stage], v_turn)) break;
          mbar_arrive(&k_empty[k_stage]);
          mbar_arrive(&v_empty[v_stage]);
          if (++k_stage == kStages) k_stage = 0, ++k_turn;
          if (++v_stage == kStages) v_stage = 0, ++v_turn;
        }
      } else {
        // S of two tiles ahead.  S of tile i takes the place of P of tile i - 2, so its product
        // waits until that one's is done.
        if (!wait(&q_full[half], groups_done++)) break;
        if (n > 0 && !wait(&pv_done[half][(n - 1) & 1], (n - 1) >> 1)) break;
        qk(n);
        if (count > 1 && ok) qk(n + 1);
        for (int j = 0; j < count && ok; ++j, ++n) {
          if (!wait(&v_full[v_stage], v_turn) || !wait(&p_full[half][n & 1], n >> 1)) break;
          const uint64_t vd = v_desc + v_stage * (L::kKv >> 4);
          const uint32_t p_at = s_at + (n & 1) * 64;
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            tc_mma_f16_ts(o_at, p_at + ks * 8, vd + ks * 2, kPvDesc, j > 0 || ks > 0);
          tc_commit(&pv_done[half][n & 1]);
          tc_commit(&v_empty[v_stage]);
          if (++v_stage == kStages) v_stage = 0, ++v_turn;
          if (j + 2 < count && wait(&pv_done[half][n & 1], n >> 1)) qk(n + 2);
        }
      }
      if (!ok) break;
      some = walk.next(a);
    }
    // every product issued is done before the CTA's memory goes
    tc_commit(&idle[half]);
    mbar_wait(&idle[half], 0, a.err);
  }
  __syncwarp();
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
