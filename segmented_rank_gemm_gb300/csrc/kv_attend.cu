// kv_attend.cu -- attention of few query rows a request over the 4-bit cache
// (include/lora_kv.h: lora_kv_attend).
//
// For one request and one cache head the query rows are columns: with G = q_heads / kv_heads,
// column c is token c / G, head h G + c % G.  A group is (request, head, 8 NT columns); over its
// cached positions j, in tiles of 32,
//     s_jc = scale <k_j, q_c>,   p_jc = 2^(s_jc - m_c),   l_c = sum_j p_jc,   O_c = sum_j p_jc v_j
// with s in units of log2(e) and m_c a running reference: O_c / l_c does not depend on it, so it
// moves (and O, l are rescaled) only when a score exceeds it by 2^8, not at every new maximum.
//
// Bound: a cached element is 0.56 bytes, so at the memory's rate an SM has 41 elements a cycle
// to decode and multiply with 128 lanes -- three instructions an element.  Decoding is two
// instructions a pair and the products go to the tensor cores (mma.sync 16x8x16: a decode step
// has 1 to 8 columns a group, far from the 128 rows a tcgen05 tile wants, and its operand A comes
// from the registers that decoded it, without a trip through shared or tensor memory):
//   S^T tile = K (16 tokens x 16 dimensions) Q^T,    K and Q in bf16
//   O^T tile = V^T (16 dimensions x 16 tokens) P^T,  V and P in fp16
// K's decoded values n s have at most 7 significant bits, exact in bf16, and q stays as it came.
// V's are exact in fp16 (times 2^-5); p is rounded to fp16 (relative error 2^-11, in 2^-6 .. 2^14
// around the reference 2^6 it is normal down to 2^-20 of the maximum) while l sums the fp32 p.
//
// Decoding, per pair of 4-bit codes n in two halves of a register: n OR the bits of 2^k gives
// 2^k + n, and one fused multiply-add (2^k + n) s - (2^k + 8) s = (n - 8) s, exact because
// (2^k + 8) s has at most 11 (fp16) or 8 (bf16) significant bits.
//
// Work split: the tiles of all groups form one sequence, cut into equal ranges for the CTAs
// and those into equal ranges for their warps, so that one long request fills the GPU and many
// short ones balance.  Each warp is independent: it runs its own ring of bulk copies (a tile of
// one head is one contiguous 4.6 KB, two of them for 16-position pages) and keeps its group's
// state in registers.  A group cut by a range's end leaves (m, l, O) pieces, joined by the CTA
// and, between CTAs, by the last one to arrive, in the order of the pieces: results do not
// depend on timing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_kernels.h"
#include "lora_common.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;    // positions of a tile
constexpr int kStages = 3;   // tiles of a warp's ring
constexpr int kMinTiles = 8; // tiles of a CTA's range, at least
constexpr int kCtasPerSm = 2;
constexpr float kRef = 6.f;    // p is 2^kRef at the reference
constexpr float kSlack = 8.f;  // how far (in powers of two) a score may exceed the reference
constexpr float kNone = -1.7e38f;

// ---- small instructions ----
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---- requests, groups and the sequence of tiles ----
struct Request {
  int row0, q_len, kv, tiles, col_tiles;
};

// Request b, checked: one with bad offsets has q_len 0.
template <int NT>
__device__ __forceinline__ Request load_request(const KvAttendArgs& a, int b, bool report) {
  Request r;
  r.row0 = __ldg(a.q_offsets + b);
  const int end = __ldg(a.q_offsets + b + 1);
  r.kv = __ldg(a.kv_len + b);
  r.q_len = end - r.row0;
  bool bad = false;
  if (r.row0 < 0 || end > a.T || r.q_len < 0 || r.q_len > a.max_q) {
    bad = true;
    r.q_len = 0;
  }
  const int cap = a.max_blocks << a.pages.page_shift;
  if (r.kv < 0 || r.kv > cap) {
    bad = true;
    r.kv = min(max(r.kv, 0), cap);
  }
  if (bad && report) atomicOr(a.err, LORA_ERRF_BAD_ID);
  const int G = a.q_heads / a.pages.heads;
  r.tiles = max(1, (r.kv + kTile - 1) / kTile);
  r.col_tiles = (r.q_len * G + 8 * NT - 1) / (8 * NT);
  return r;
}

__device__ __forceinline__ long long request_tiles(const Request& r, int heads) {
  return static_cast<long long>(r.tiles) * r.col_tiles * heads;
}

// A position in the sequence of tiles: request, head, column tile, tile (fastest last).
template <int NT>
struct Cursor {
  Request r;
  int b, head, col, tile;
  __device__ __forceinline__ void start(const KvAttendArgs& a, int b_, long long rem) {
    b = b_;
    r = load_request<NT>(a, b, false);
    tile = static_cast<int>(rem % r.tiles);
    const long long g = rem / r.tiles;
    col = static_cast<int>(g % r.col_tiles);
    head = static_cast<int>(g / r.col_tiles);
  }
  // Moves to the next tile; true if that begins another group.  Not past the last one.
  __device__ __forceinline__ bool next(const KvAttendArgs& a) {
    if (++tile < r.tiles) return false;
    tile = 0;
    if (++col < r.col_tiles) return true;
    col = 0;
    if (++head < a.pages.heads) return true;
    head = 0;
    do {
      ++b;
      r = load_request<NT>(a, b, false);
    } while (r.col_tiles == 0);
    return true;
  }
};

// ---- partial results ----
// A piece: m [8 NT], l [8 NT], O [8 NT][D].
template <int D, int NT>
constexpr int piece_floats() {
  return 8 * NT * (D + 2);
}

struct PieceInfo {
  long long group;  // first tile of the group in the sequence, -1: none
  int tiles;        // of the group
  int b, head, col;
};

template <int D, int NT>
struct State {
  float o[D / 16][NT][4];  // [dimension pair][column tile][fragment]
  float m[NT][2], l[NT][2];
};

// Columns' rows in q and out: the element offset of column c, or -1.
template <int NT>
__device__ __forceinline__ long long column_offset(const KvAttendArgs& a, const Request& r, int head,
                                                   int col_tile, int c, int ld) {
  const int G = a.q_heads / a.pages.heads;
  const int col = col_tile * 8 * NT + c;
  if (col >= r.q_len * G) return -1;
  const int token = col / G;
  return static_cast<long long>(r.row0 + token) * ld +
         static_cast<long long>(head * G + (col - token * G)) * a.pages.D;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) kv_attend_kernel(KvAttendArgs a) {
  constexpr int kBlock = kv_block_bytes(D), kTileBytes = 2 * kBlock;
  constexpr int KT = D / 16;         // 16-wide steps of D
  constexpr int KW = D / 32;         // 32-bit words of K a lane reads of a token
  constexpr int VW = D / 64;         // of V
  constexpr int LD = D / 8;          // dimensions of V a lane owns
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ long long scan[kWarps];
  __shared__ long long start_rem[kWarps];
  __shared__ int start_b[kWarps];
  __shared__ PieceInfo info[kWarps * 2];
  __shared__ int last_cta;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int heads = a.pages.heads;

  // rows of no request
  {
    const int lo = max(0, min(__ldg(a.q_offsets), a.T)), hi = max(0, min(__ldg(a.q_offsets + a.B), a.T));
    const int words = a.q_heads * D / 8;  // 16-byte words of a row
    const long long n = static_cast<long long>(lo + a.T - hi) * words;
    for (long long i = blockIdx.x * kThreads + tid; i < n; i += gridDim.x * kThreads) {
      int row = static_cast<int>(i / words);
      if (row >= lo) row += hi - lo;
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(row) * a.ldo)[
          i % words] = make_uint4(0u, 0u, 0u, 0u);
    }
  }

  // the sequence's length and this CTA's range; where each warp starts
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b)
    mine += request_tiles(load_request<NT>(a, b, blockIdx.x == 0), heads);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  if (tid < kWarps * 2) info[tid].group = -1;
  if (tid < kWarps * kStages) mbar_init(&full[0][0] + tid, 1);
  fence_mbar_init();
  __syncthreads();
  long long total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const long long span = max(static_cast<long long>(kMinTiles), (total + gridDim.x - 1) / gridDim.x);
  const long long cta_lo = span * blockIdx.x, cta_hi = min(total, cta_lo + span);
  if (cta_lo >= total) return;
  const long long wspan = (cta_hi - cta_lo + kWarps - 1) / kWarps;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const long long at = cta_lo + w * wspan;
    if (at < cta_hi && at >= before && at < before + mine) {
      long long rem = at - before;
      int b = b0;
      for (;; ++b) {
        const long long n = request_tiles(load_request<NT>(a, b, false), heads);
        if (rem < n) break;
        rem -= n;
      }
      start_b[w] = b;
      start_rem[w] = rem;
    }
  }
  __syncthreads();

  const long long w_lo = cta_lo + warp * wspan, w_hi = min(cta_hi, w_lo + wspan);
  float* const warp_pieces =
      a.pieces + static_cast<size_t>(gridDim.x) * 2 * piece_floats<D, NT>() +
      static_cast<size_t>(blockIdx.x * kWarps + warp) * 2 * piece_floats<D, NT>();

  if (w_lo < w_hi) {
    uint8_t* const my_ring = ring + warp * kStages * kTileBytes;
    uint64_t* const bar = full[warp];
    Cursor<NT> in, at;
    in.start(a, start_b[warp], start_rem[warp]);
    at = in;
    const int n = static_cast<int>(w_hi - w_lo);
    const int shift = a.pages.page_shift;

    // page ids of 32 consecutive tiles of the request being fetched, one tile a lane
    int ids_b = -1, ids_tile = 0, id0 = 0, id1 = 0;
    bool dead = false;
    auto fetch_ids = [&]() {
      ids_b = in.b;
      ids_tile = in.tile & ~31;
      const int last = max(0, (in.r.kv - 1) >> shift);  // the request's last page
      const int32_t* row = a.table + static_cast<size_t>(in.b) * a.max_blocks;
      const int pos = (ids_tile + lane) * kTile;
      const int i0 = min(pos >> shift, last), i1 = min((pos + kKvBlock) >> shift, last);
      const bool some = in.r.kv > 0;
      id0 = some ? __ldg(row + i0) : 0;
      id1 = some ? __ldg(row + i1) : 0;
      if (static_cast<unsigned>(id0) >= static_cast<unsigned>(a.pages.num_pages) ||
          static_cast<unsigned>(id1) >= static_cast<unsigned>(a.pages.num_pages)) {
        atomicOr(a.err, LORA_ERRF_BAD_ID);
        if (static_cast<unsigned>(id0) >= static_cast<unsigned>(a.pages.num_pages)) id0 = 0;
        if (static_cast<unsigned>(id1) >= static_cast<unsigned>(a.pages.num_pages)) id1 = 0;
      }
    };
    auto issue = [&](int u) {  // fetch tile `in` as the warp's u-th
      if (in.b != ids_b || (in.tile & ~31) != ids_tile) fetch_ids();
      const int p0 = __shfl_sync(0xffffffffu, id0, in.tile & 31);
      const int p1 = __shfl_sync(0xffffffffu, id1, in.tile & 31);
      if (lane == 0) {
        uint8_t* dst = my_ring + (u % kStages) * kTileBytes;
        uint64_t* b = bar + u % kStages;
        mbar_arrive_expect_tx(b, kTileBytes);
        const int blk = (in.tile * kTile & ((1 << shift) - 1)) / kKvBlock;
        if (shift > 4) {
          bulk_load_g2s(dst, a.pages.base + a.pages.block(p0, in.head, blk), kTileBytes, b);
        } else {
          bulk_load_g2s(dst, a.pages.base + a.pages.block(p0, in.head, 0), kBlock, b);
          bulk_load_g2s(dst + kBlock, a.pages.base + a.pages.block(p1, in.head, 0), kBlock, b);
        }
      }
    };

    int issued = 0;
    for (; issued < kStages && issued < n; ++issued) {
      if (issued) in.next(a);
      issue(issued);
    }

    uint32_t qf[KT][NT][2];
    int lim[NT][2], lim_lo = 0, lim_hi = 0;
    State<D, NT> st;
    const int ta = kv_frag_token(g);  // tokens of fragment rows g and g + 8: ta, ta + 8
    const int tv = ((t & 1) | (t >> 1) << 1);
    bool fresh = true;
    long long group = w_lo - at.tile;

    for (int u = 0; u < n; ++u) {
      if (fresh) {
        // the group's queries, the last position each column sees, and an empty state
        const int G = a.q_heads / heads;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const long long off = column_offset<NT>(a, at.r, at.head, at.col, nt * 8 + g, a.ldq);
          const uint4* src =
              reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + off + t * (D / 4));
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            const uint4 v = off >= 0 ? __ldg(src + w) : make_uint4(0u, 0u, 0u, 0u);
            qf[2 * w][nt][0] = prmt(v.x, v.z, 0x5410);
            qf[2 * w][nt][1] = prmt(v.x, v.z, 0x7632);
            qf[2 * w + 1][nt][0] = prmt(v.y, v.w, 0x5410);
            qf[2 * w + 1][nt][1] = prmt(v.y, v.w, 0x7632);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // (a column past the last has zero queries and is not written: any limit does)
            const int c = at.col * 8 * NT + nt * 8 + 2 * t + j;
            lim[nt][j] = at.r.kv - at.r.q_len + min(c / G, at.r.q_len - 1);
            st.m[nt][j] = kNone;
            st.l[nt][j] = 0.f;
          }
        }
        lim_lo = at.r.kv - at.r.q_len + at.col * 8 * NT / G;
        lim_hi = at.r.kv - at.r.q_len + min(at.r.q_len * G - 1, at.col * 8 * NT + 8 * NT - 1) / G;
#pragma unroll
        for (int m = 0; m < KT; ++m)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) st.o[m][nt][j] = 0.f;
        fresh = false;
      }

      if (!dead && !mbar_wait(bar + u % kStages, (u / kStages) & 1, a.err)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      const int pos0 = at.tile * kTile;
      if (pos0 <= lim_hi) {
        const uint8_t* tile = my_ring + (u % kStages) * kTileBytes;
        float s[2][NT][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint8_t* blk = tile + k * kBlock;
          uint32_t kw[2][KW], sc[2][KW / 2];
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(blk + ta * 64 + 16 * t);
            const uint4 y = *reinterpret_cast<const uint4*>(blk + (ta + 8) * 64 + 16 * t);
            kw[0][0] = x.x, kw[0][1] = x.y, kw[0][2] = x.z, kw[0][3] = x.w;
            kw[1][0] = y.x, kw[1][1] = y.y, kw[1][2] = y.z, kw[1][3] = y.w;
            const uint32_t b4 = *reinterpret_cast<const uint32_t*>(blk + kv_k_scales(D) + lane * 4);
            sc[0][0] = prmt(b4, 0u, 0x4040) << 4;
            sc[0][1] = prmt(b4, 0u, 0x4141) << 4;
            sc[1][0] = prmt(b4, 0u, 0x4242) << 4;
            sc[1][1] = prmt(b4, 0u, 0x4343) << 4;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(blk + ta * 32 + 8 * t);
            const uint2 y = *reinterpret_cast<const uint2*>(blk + (ta + 8) * 32 + 8 * t);
            kw[0][0] = x.x, kw[0][1] = x.y;
            kw[1][0] = y.x, kw[1][1] = y.y;
            const uint32_t b2 = *reinterpret_cast<const uint16_t*>(blk + kv_k_scales(D) + lane * 2);
            sc[0][0] = prmt(b2, 0u, 0x4040) << 4;
            sc[1][0] = prmt(b2, 0u, 0x4141) << 4;
          }
          uint32_t bias[2][KW / 2];
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int p = 0; p < KW / 2; ++p) {
              // e4m3's exponent and mantissa as bf16's, rescaled by 2^120: exact
              sc[r][p] = mul_bf16x2(sc[r][p], 0x7B807B80u);
              bias[r][p] = mul_bf16x2(sc[r][p], 0xC308C308u);  // -136 s
            }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[k][nt][j] = 0.f;
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            uint32_t v[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[r][i] = fma_bf16x2((kw[r][w] >> (4 * i) & 0x000F000Fu) | 0x43004300u, sc[r][w / 2],
                                     bias[r][w / 2]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_bf16(s[k][nt], v[0][0], v[1][0], v[0][1], v[1][1], qf[2 * w][nt][0],
                       qf[2 * w][nt][1]);
              mma_bf16(s[k][nt], v[0][2], v[1][2], v[0][3], v[1][3], qf[2 * w + 1][nt][0],
                       qf[2 * w + 1][nt][1]);
            }
          }
        }

        // scores in units of log2(e); positions a column does not see
        bool over = false;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[k][nt][j] *= a.scale_log2;
        if (pos0 + kTile - 1 > lim_lo) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (pos0 + k * kKvBlock + ta + (j >> 1) * 8 > lim[nt][j & 1])
                  s[k][nt][j] = -INFINITY;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float top = fmaxf(fmaxf(s[0][nt][j], s[0][nt][j + 2]),
                                    fmaxf(s[1][nt][j], s[1][nt][j + 2]));
            over |= top > st.m[nt][j] + (kRef + kSlack);
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float top = fmaxf(fmaxf(s[0][nt][j], s[0][nt][j + 2]),
                                fmaxf(s[1][nt][j], s[1][nt][j + 2]));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              const float m = fmaxf(st.m[nt][j], top - kRef);
              const float f = ex2(st.m[nt][j] - m);
              st.m[nt][j] = m;
              st.l[nt][j] *= f;
#pragma unroll
              for (int d = 0; d < KT; ++d) {
                st.o[d][nt][j] *= f;
                st.o[d][nt][j + 2] *= f;
              }
            }
        }

#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint8_t* blk = tile + k * kBlock;
          uint32_t pf[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              p[j] = ex2(s[k][nt][j] - st.m[nt][j & 1]);
              st.l[nt][j & 1] += p[j];
            }
            pf[nt][0] = transpose_8x8(pack_f16x2(p[0], p[1]));
            pf[nt][1] = transpose_8x8(pack_f16x2(p[2], p[3]));
          }
          // V: lane group t's four tokens, this lane's LD dimensions
          uint32_t vw[4][VW], vs;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int token = (tv ^ (i & 1)) | (i & 1) << 2 | (i >> 1) << 3;
            if constexpr (D == 128) {
              const uint2 x = *reinterpret_cast<const uint2*>(blk + kv_v_codes(D) + token * 64 +
                                                              ((8 * g) ^ ((t >> 1) << 5)));
              vw[i][0] = x.x, vw[i][1] = x.y;
            } else {
              vw[i][0] = *reinterpret_cast<const uint32_t*>(blk + kv_v_codes(D) + token * 32 + 4 * g);
            }
          }
          vs = *reinterpret_cast<const uint32_t*>(blk + kv_v_scales(D) +
                                                  ((D == 128 ? g : g >> 1) * 4 + t) * 4);
          uint32_t v[2][LD];  // [token pair][dimension]
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            const uint32_t s0 = mul_f16x2(e4m3x2_to_f16x2(static_cast<uint16_t>(vs >> (16 * pr))),
                                          0x28002800u);        // s 2^-5
            const uint32_t c0 = mul_f16x2(s0, 0xE408E408u);    // -1032 s 2^-5
            const uint32_t s1 = mul_f16x2(s0, 0x2C002C00u);    // s 2^-9
            const uint32_t c1 = mul_f16x2(s0, 0xD480D480u);    // -72 s 2^-5
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const uint32_t y = prmt(vw[2 * pr][w], vw[2 * pr + 1][w], hf ? 0x7632 : 0x5410);
                const uint32_t y8 = y >> 8;
                uint32_t* o = v[pr] + w * 8 + hf * 4;
                o[0] = fma_f16x2((y & 0x000F000Fu) | 0x64006400u, s0, c0);
                o[1] = fma_f16x2((y & 0x00F000F0u) | 0x64006400u, s1, c1);
                o[2] = fma_f16x2((y8 & 0x000F000Fu) | 0x64006400u, s0, c0);
                o[3] = fma_f16x2((y8 & 0x00F000F0u) | 0x64006400u, s1, c1);
              }
          }
#pragma unroll
          for (int m = 0; m < KT; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(st.o[m][nt], v[0][2 * m], v[0][2 * m + 1], v[1][2 * m], v[1][2 * m + 1],
                      pf[nt][0], pf[nt][1]);
        }
      }

      // the stage is free: every lane has read it
      __syncwarp();
      if (issued < n && !dead) {
        in.next(a);
        issue(issued);
        ++issued;
      }

      const bool group_ends = at.tile == at.r.tiles - 1;
      if (group_ends || u == n - 1) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float l = st.l[nt][j];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            st.l[nt][j] = l;
          }
        if (group_ends && group >= w_lo) {
          const float unit = 32.f * a.v_scale;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const long long off =
                  column_offset<NT>(a, at.r, at.head, at.col, nt * 8 + 2 * t + j, a.ldo);
              if (off < 0) continue;
              const float f = st.l[nt][j] == 0.f ? 0.f : unit / st.l[nt][j];
              uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + off + g * LD);
#pragma unroll
              for (int w = 0; w < LD / 8; ++w) {
                uint32_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  x[i] = pack_bf16x2(st.o[4 * w + i][nt][j] * f, st.o[4 * w + i][nt][j + 2] * f);
                dst[w] = make_uint4(x[0], x[1], x[2], x[3]);
              }
            }
        } else {
          // a piece: slot 0 began before this warp's range, slot 1 goes on after it
          const int slot = group < w_lo ? 0 : 1;
          float* piece = warp_pieces + slot * piece_floats<D, NT>();
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int c = nt * 8 + 2 * t + j;
              if (g == 0) {
                piece[c] = st.m[nt][j];
                piece[8 * NT + c] = st.l[nt][j];
              }
              float* o = piece + 16 * NT + c * D + g * LD;
#pragma unroll
              for (int m = 0; m < KT; m += 2)
                *reinterpret_cast<float4*>(o + 2 * m) =
                    make_float4(st.o[m][nt][j], st.o[m][nt][j + 2], st.o[m + 1][nt][j],
                                st.o[m + 1][nt][j + 2]);
            }
          if (lane == 0) info[warp * 2 + slot] = PieceInfo{group, at.r.tiles, at.b, at.head, at.col};
        }
      }
      if (u + 1 < n && at.next(a)) {
        fresh = true;
        group = w_lo + u + 1;
      }
    }
    if (dead)  // copies still in flight write this CTA's shared memory: let them land
      for (int i = 0; i < kStages; ++i) mbar_wait(bar + i, ((issued - 1) / kStages) & 1, a.err);
  }
  __syncthreads();

  // Join the pieces, in the order of the sequence.  dst: the CTA's piece (then O, m and l), or
  // the output.
  auto join = [&](auto piece_of, int n, const PieceInfo& gi, float* dst) {
    Request r = load_request<NT>(a, gi.b, false);
    const float unit = 32.f * a.v_scale;
    for (int e = tid; e < 8 * NT * (D / 4); e += kThreads) {
      const int c = e / (D / 4), d = e % (D / 4) * 4;
      const long long off = column_offset<NT>(a, r, gi.head, gi.col, c, a.ldo);
      if (off < 0) continue;
      float m = kNone;
      for (int i = 0; i < n; ++i) m = fmaxf(m, __ldcg(piece_of(i) + c));
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < n; ++i) {
        const float* p = piece_of(i);
        const float f = ex2(__ldcg(p + c) - m);
        l += f * __ldcg(p + 8 * NT + c);
        const float4 x = __ldcg(reinterpret_cast<const float4*>(p + 16 * NT + c * D + d));
        o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
      }
      if (dst) {
        if (d == 0) {
          dst[c] = m;
          dst[8 * NT + c] = l;
        }
        *reinterpret_cast<float4*>(dst + 16 * NT + c * D + d) = o;
      } else {
        const float f = l == 0.f ? 0.f : unit / l;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + off + d) =
            make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
      }
    }
  };
  constexpr int kPiece = piece_floats<D, NT>();
  float* const cta_warp_pieces = a.pieces + static_cast<size_t>(gridDim.x) * 2 * kPiece +
                                 static_cast<size_t>(blockIdx.x) * kWarps * 2 * kPiece;
  for (int i = 0; i < kWarps * 2;) {
    const PieceInfo gi = info[i];
    if (gi.group < 0) {
      ++i;
      continue;
    }
    int idx[kWarps * 2], n = 0, j = i;
    for (; j < kWarps * 2; ++j) {
      if (info[j].group < 0) continue;
      if (info[j].group != gi.group) break;
      idx[n++] = j;
    }
    i = j;
    const auto warp_piece = [&](int k) { return cta_warp_pieces + idx[k] * kPiece; };
    const long long end = gi.group + gi.tiles;
    if (gi.group >= cta_lo && end <= cta_hi) {
      join(warp_piece, n, gi, nullptr);
      continue;
    }
    const int first = static_cast<int>(gi.group / span), last = static_cast<int>((end - 1) / span);
    join(warp_piece, n, gi, a.pieces + (blockIdx.x * 2 + (gi.group < cta_lo ? 0 : 1)) * static_cast<size_t>(kPiece));
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      const int seen = atomicAdd(a.arrivals + first, 1);
      last_cta = seen == last - first;
      if (last_cta) a.arrivals[first] = 0;
      __threadfence();
    }
    __syncthreads();
    if (last_cta)
      join([&](int k) { return a.pieces + (k == 0 ? first * 2 + 1 : (first + k) * 2) * static_cast<size_t>(kPiece); },
           last - first + 1, gi, nullptr);
    __syncthreads();
  }
}

template <int D, int NT>
cudaError_t launch(const KvAttendArgs& a, cudaStream_t stream) {
  constexpr int smem = kWarps * kStages * 2 * kv_block_bytes(D);
  static int limit[kAttrDevices] = {};
  cudaError_t e = ensure_smem_limit(kv_attend_kernel<D, NT>, smem, limit);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(kKvMaxCtas, a.num_sms * kCtasPerSm);
  kv_attend_kernel<D, NT><<<ctas, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv_attend_workspace_floats(int num_sms, int D) {
  const size_t ctas = std::min(kKvMaxCtas, num_sms * kCtasPerSm);
  return ctas * 2 * (1 + kWarps) * (D == 128 ? piece_floats<128, 1>() : piece_floats<64, 1>());
}

cudaError_t launch_kv_attend(const KvAttendArgs& a, cudaStream_t stream) {
  return a.pages.D == 128 ? launch<128, 1>(a, stream) : launch<64, 1>(a, stream);
}

}  // namespace lora
