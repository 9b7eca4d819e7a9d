// kv_attend.cu -- attention of few query rows a request over the 4-bit cache
// (include/lora_kv.h: lora_kv_attend).
//
// For one request and one cache head the query rows are columns: with G = q_heads / kv_heads,
// column c is token c / G, head h G + c % G.  A group is (request, head, 8 columns); over its
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
//   S^T tile = K (16 tokens x 16 dimensions) Q^T
//   O^T tile = V^T (16 dimensions x 16 tokens) P^T
// in fp16 with fp32 accumulation.  K's and V's decoded values n s 2^-5 are exact in fp16.  A query
// row is scaled by the power of two that brings its largest element to 2^9 .. 2^10, which its 8
// significant bits survive down to 2^-23 of that (2^-19 in the dimensions whose keys are decoded
// sixteen times as large, and whose queries are that much smaller).  p is rounded to fp16 (relative error 2^-11;
// with the reference at 2^6 it is a normal number down to 2^-20 of the maximum) while l sums
// the fp32 p.
//
// Work split: the tiles of all groups form one sequence, cut into equal ranges for the CTAs
// and those into equal ranges for their warps, so that one long request fills the GPU and many
// short ones balance.  A group counts kSetup units besides its tiles, about what its queries'
// load and its output cost, and a cut near a group's edge moves there.  Each warp is independent:
// it runs its own ring of bulk copies (a tile of one head is one contiguous 4.6 KB, two copies for
// 16-position pages) and keeps its group's state in registers.  A group cut by a range's end leaves
// (m, l, O) pieces (a warp's last one in its ring, which is free by then), joined by the CTA and,
// between CTAs, by the last one to arrive, in the order of the pieces: results do not depend on
// timing.
//
// Measured (32 query heads over 8 of 128): 3 contexts of 91 to 107 thousand positions 82 us, 350
// MB at 4.3 TB/s; 512 single tokens over 1 to 2048 positions 63 us; one over 1000 12.8 us.  What
// bounds it: a tile is 617 instructions, half of them the decoding, of which a scheduler's four warps issue
// three in four cycles in the main loop (the tiles stream at 5.7 TB/s there); before it lie 4.5 us of
// launch, scan and first loads, and behind it the spread of the warps and the joins, 10 to 15 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kv_decode.cuh"
#include "kv_kernels.h"
#include "kv_span.cuh"
#include "lora_common.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;    // positions of a tile
constexpr int kCols = 8;     // columns of a group
constexpr int kStages = 3;   // tiles of a warp's ring
// Units a group counts before its tiles (512 single tokens: 63.5 us with 2, 64.4 with 3, 67.2 with
// 4), and units of a CTA's range, at least (one request of 1000 positions: 12.8 us with 4, 12.7 with
// 8, 14.1 with 16; 4 requests of 512 over one head 11.8, 12.6, 14.2).
constexpr int kSetup = 2;
constexpr int kMinSpan = 4;
constexpr int kCtasPerSm = 2;
constexpr float kRef = 6.f;    // p is 2^kRef at the reference
constexpr float kSlack = 8.f;  // how far (in powers of two) a score may exceed the reference
constexpr float kNone = -1.7e38f;

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first of a sum.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// ---- requests, groups and the sequence of tiles ----
// The tiles start at position `first`, and the positions of a request's queries' limits count from
// there: token t sees see + slope t (a span's; a whole causal request: 0, kv - q_len and 1).
struct Request {
  int row0, q_len, kv, tiles, col_tiles;
  int first, see, slope, table_row;
  SpanKind kind;
  template <Spans SPANS>
  __device__ __forceinline__ int last_seen(int token) const {
    if (SPANS == kShared) return see + slope * token;
    return SPANS == kEncoder ? kv - 1 : kv - q_len + token;  // (held anyway: fewer registers)
  }
};

__device__ __forceinline__ int tiles_of(int positions) {  // (up to 2^31 - 1 of them)
  return max(1u, (static_cast<unsigned>(positions) + kTile - 1) / kTile);
}

// Request b, checked: one with bad offsets has q_len 0.  (Loads in order: the kernel's wait for the
// one before stands ahead of them.)
template <Spans SPANS>
__device__ __forceinline__ Request load_request(const KvAttendArgs& a, int b, bool report) {
  Request r;
  const int G = a.group;
  if constexpr (SPANS != kRequests) {
    const Span s = load_span<SPANS>(a, b, report);
    r = Request{s.row0, s.q_len, s.kv, 0, 0, s.first, s.see, s.slope, s.table_row, s.kind};
    r.tiles = tiles_of(r.kv - r.first);
    r.col_tiles = span_is_few(a, s) ? (r.q_len * G + kCols - 1) / kCols : 0;
    return r;
  }
  r.row0 = load_in_order(a.q_offsets + b);
  const int end = load_in_order(a.q_offsets + b + 1);
  r.kv = load_in_order(a.kv_len + b);
  // (in this order: the difference of any two offsets need not be an int)
  bool bad = r.row0 < 0 || end < r.row0 || end > a.T || end - r.row0 > a.max_q;
  r.q_len = bad ? 0 : end - r.row0;
  const int cap = a.max_blocks << a.pages.page_shift;
  if (r.kv < 0 || r.kv > cap) {
    bad = true;
    r.kv = min(max(r.kv, 0), cap);
  }
  if (bad && report) atomicOr(a.err, LORA_ERRF_BAD_ID);
  r.first = 0;
  r.see = r.kv - r.q_len;
  r.slope = 1;
  r.table_row = b;
  r.kind = kSpanWhole;
  r.tiles = tiles_of(r.kv);
  r.col_tiles = r.q_len * G > a.few_rows ? 0 : (r.q_len * G + kCols - 1) / kCols;
  return r;
}

__device__ __forceinline__ long long request_units(const Request& r, int heads) {
  return static_cast<long long>(r.tiles + kSetup) * r.col_tiles * heads;
}

// A position in the sequence of tiles: request, head, column tile, tile (fastest last), and
// the tile's unit: a group's tiles come after its kSetup units.
template <Spans SPANS>
struct Cursor {
  Request r;
  int b, head, col, tile;
  long long unit;
  // The first tile at or after unit `at`, the rem-th of request b_; a cut within snap of a group's
  // edge moves there (to its end by tile = tiles, one past the last).
  __device__ __forceinline__ void start(const KvAttendArgs& a, int b_, long long rem, long long at,
                                        int snap) {
    b = b_;
    r = load_request<SPANS>(a, b, false);
    const int per = r.tiles + kSetup;
    const long long group = quotient(rem, per);
    const int off = static_cast<int>(rem - group * per);
    tile = off <= kSetup + snap ? 0 : per - off <= snap ? r.tiles : off - kSetup;
    unit = at - off + kSetup + tile;
    head = static_cast<int>(quotient(group, r.col_tiles));
    col = static_cast<int>(group - static_cast<long long>(head) * r.col_tiles);
  }
  // Moves to the next group.  Not past the last one.
  __device__ __forceinline__ void next_group(const KvAttendArgs& a) {
    unit += r.tiles - tile + kSetup;
    tile = 0;
    if (++col < r.col_tiles) return;
    col = 0;
    if (++head < a.pages.heads) return;
    head = 0;
    do {
      ++b;
      r = load_request<SPANS>(a, b, false);
    } while (r.col_tiles == 0);
  }
};

// ---- partial results ----
// A piece: m [8], l [8], O [8][D].
template <int D>
constexpr int piece_floats() {
  return kCols * (D + 2);
}

struct PieceInfo {
  long long group;  // unit of the group's first tile, -1: none
  int tiles;        // of the group
  int cols;         // its columns
  int row0, head, first_col;
  SpanKind kind;
  const float* at;
};

template <int D>
struct State {
  float o[D / 16][4];  // [dimension pair][fragment]
  float2 minus, l;     // -m and l of the fragment's two columns
};

// Columns' rows in q and out: the element offset of column c, or -1.
__device__ __forceinline__ long long column_offset(const KvAttendArgs& a, const Request& r, int head,
                                                   int col_tile, int c, int ld) {
  const int G = a.group;
  const int col = col_tile * kCols + c;
  if (col >= r.q_len * G) return -1;
  const int token = a.token_of(col);
  return static_cast<long long>(r.row0 + token) * ld +
         static_cast<long long>(head * G + (col - token * G)) * a.pages.D;
}

// A bulk copy, or two one behind the other, counted on `bar` and asked for by the one lane with `mine`.
__device__ __forceinline__ void fetch_one(uint32_t mine, uint32_t dst, const uint8_t* src,
                                          uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %0, 0;\n\t"
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%4], %3;\n\t"
      "@p cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%2], %3, [%4];\n\t}" ::"r"(mine),
      "r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void fetch_two(uint32_t mine, uint32_t dst, const uint8_t* src0,
                                          const uint8_t* src1, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %0, 0;\n\t"
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%5], %6;\n\t"
      "@p cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%2], %4, [%5];\n\t"
      "@p cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%7], [%3], %4, [%5];\n\t}" ::"r"(mine),
      "r"(dst), "l"(src0), "l"(src1), "r"(bytes), "r"(bar), "r"(2 * bytes), "r"(dst + bytes)
      : "memory");
}

template <int D, Spans SPANS>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv_attend_kernel(KvAttendArgs a) {
  constexpr int kBlock = kv_block_bytes(D), kTileBytes = 2 * kBlock;
  constexpr int KT = D / 16;         // 16-wide steps of D
  constexpr int KW = D / 32;         // 32-bit words of K a lane reads of a token
  constexpr int VW = D / 64;         // of V
  constexpr int LD = D / 8;          // dimensions of V a lane owns
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ long long scan[kWarps];
  __shared__ long long start_rem[kWarps + 1], cut_unit[kWarps + 1];  // of the warps' cuts
  __shared__ int start_b[kWarps + 1];
  __shared__ PieceInfo info[kWarps * 2];
  __shared__ int last_cta[2];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int heads = a.pages.heads;

  if (tid < kWarps * 2) info[tid].group = -1;
  if (tid < kWarps * kStages) mbar_init(&full[0][0] + tid, 1);
  fence_mbar_init();
  // The kernel ahead may have written anything that is read below, the lengths among it (the maps of
  // the batch do).  The kernel for many rows needs nothing of this one's: it may start now, on what came
  // before both, and waits for this one at its end.
  griddep_wait();
  if (a.many_follow) griddep_launch_dependents();

  // the sequence's length and this CTA's range; where each warp starts
  const int count_b = SPANS == kShared ? a.B + a.groups : a.B;
  const int per = (count_b + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, count_b), b1 = min(b0 + per, count_b);
  long long mine = 0;
  for (int b = b0; b < b1; ++b)
    mine += request_units(load_request<SPANS>(a, b, blockIdx.x == 0), heads);
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
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const long long span = max(static_cast<long long>(kMinSpan), quotient(total + gridDim.x - 1, gridDim.x));

  // rows of no request
  {
    const int lo = max(0, min(load_in_order(a.q_offsets), a.T));
    const int hi = max(0, min(load_in_order(a.q_offsets + a.B), a.T));
    const int words = a.q_heads * D / 8;  // 16-byte words of a row
    const long long n = static_cast<long long>(lo + a.T - hi) * words;
    for (long long i = blockIdx.x * kThreads + tid; i < n; i += gridDim.x * kThreads) {
      int row = static_cast<int>(i / words);
      if (row >= lo) row += hi - lo;
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(row) * a.ldo)[
          i % words] = make_uint4(0u, 0u, 0u, 0u);
    }
  }

  if (SPANS == kAlone && blockIdx.x == gridDim.x - 1) {  // (else done by what reads and joins the parts)
    for (int b = tid; b < a.B; b += kThreads) check_group_of(a, b);
    for (int v = 0; v < a.groups; ++v) check_prefix_pages(a, v, tid, kThreads);
  }
  if (span * blockIdx.x >= total) return;
  const long long raw_lo = span * blockIdx.x, raw_hi = min(total, raw_lo + span);
  // A cut within snap of a group's edge moves there, which spares two pieces (512 tokens beside 8
  // prompts: 85.9 us without, 84.0 with; 512 tokens alone 62.8 and 63.2, 65.0 for wspan / 4; 256
  // requests of 2 tokens over 300 positions 48.6 and 44.9).
  const int wspan = static_cast<int>((span + kWarps - 1) / kWarps), snap = min(wspan / 4, 2);
#pragma unroll
  for (int w = 0; w <= kWarps; ++w) {
    const long long at = min(raw_hi, raw_lo + static_cast<long long>(w) * wspan);
    if (at >= before && at < before + mine) {
      long long rem = at - before;
      int b = b0;
      for (; b < b1 - 1; ++b) {  // (the run's last takes what is left)
        const long long n = request_units(load_request<SPANS>(a, b, false), heads);
        if (rem < n) break;
        rem -= n;
      }
      start_b[w] = b;
      start_rem[w] = rem;
    }
  }
  __syncthreads();
  Cursor<SPANS> in;
#pragma unroll 1
  for (int w = kWarps + warp; w >= 0; w -= kWarps) {  // this warp's first tile; warp 0: the CTA's end too
    if (w > kWarps) continue;
    const long long at = min(raw_hi, raw_lo + static_cast<long long>(w) * wspan);
    in.unit = total;
    if (at < total) in.start(a, start_b[w], start_rem[w], at, at == 0 ? 0 : snap);
    if (lane == 0) cut_unit[w] = in.unit;
  }
  __syncthreads();
  const long long w_lo = cut_unit[warp], w_hi = cut_unit[warp + 1];
  const long long cta_lo = cut_unit[0], cta_hi = cut_unit[kWarps];
  float* const warp_pieces =
      a.pieces + static_cast<size_t>(gridDim.x) * 2 * piece_floats<D>() +
      static_cast<size_t>(blockIdx.x * kWarps + warp) * 2 * piece_floats<D>();
  if (w_lo < w_hi && in.tile == in.r.tiles) {  // the cut moved to its group's end
    if (w_lo + kSetup < w_hi) in.next_group(a);
    else in.unit = w_hi;
  }

  if (w_lo < w_hi && in.unit < w_hi) {
    uint8_t* const my_ring = ring + warp * kStages * kTileBytes;
    uint64_t* const bar = full[warp];
    Cursor<SPANS> at = in;
    const int shift = a.pages.page_shift;
    const uint32_t page_bytes = static_cast<uint32_t>(kBlock) << (shift - 4);  // of one head
    const size_t page_stride = static_cast<size_t>(page_bytes) * heads;
    const int in_page = max(0, (1 << shift) / kTile - 1);  // mask of a tile's place in its page

    // Where 32 consecutive tiles of the request and head being fetched are, one tile a lane, which
    // asks for it (two pages a tile where a page is half of one).
    int src_b = -1, src_tile = 0, src_head = 0;
    const uint8_t *src0 = nullptr, *src1 = nullptr;
    auto aim = [&]() {
      if (in.b == src_b && (in.tile & ~31) == src_tile) {  // another head's
        const ptrdiff_t by = static_cast<ptrdiff_t>(in.head - src_head) * page_bytes;
        src0 += by;
        src1 += by;
      } else {
        src_b = in.b;
        src_tile = in.tile & ~31;
        const unsigned last = max(0, (in.r.kv - 1) >> shift);  // the request's last page
        const int32_t* row = a.table + static_cast<size_t>(SPANS == kShared ? in.r.table_row : in.b) * a.max_blocks;
        const unsigned pos = in.r.first + (src_tile + lane) * static_cast<unsigned>(kTile);  // (past 2^31, maybe)
        const bool some = in.r.kv > in.r.first;
        int id0 = some ? __ldg(row + min(pos >> shift, last)) : 0;
        int id1 = some ? __ldg(row + min((pos + kKvBlock) >> shift, last)) : 0;
        const unsigned pages = a.pages.num_pages;
        if (static_cast<unsigned>(id0) >= pages || static_cast<unsigned>(id1) >= pages) {
          atomicOr(a.err, LORA_ERRF_BAD_ID);
          if (static_cast<unsigned>(id0) >= pages) id0 = 0;
          if (static_cast<unsigned>(id1) >= pages) id1 = 0;
        }
        const uint8_t* base = a.pages.base + static_cast<size_t>(in.head) * page_bytes;
        src0 = base + id0 * page_stride + ((src_tile + lane) & in_page) * kTileBytes;
        src1 = base + id1 * page_stride;
      }
      src_head = in.head;
    };
    bool dead = false;
    // Fetch tile `in` into a stage, if there is one left, and move on; in.unit is its group's first
    // tile's.
    int in_left = static_cast<int>(min(static_cast<long long>(in.r.tiles - in.tile), w_hi - in.unit));
    in.unit -= in.tile;
    const uint32_t ring_at = smem_u32(my_ring), bar_at = smem_u32(bar);
    auto fetch = [&](int stage) {
      if (in_left == 0) return;
      const uint32_t mine = lane == (in.tile & 31);
      if (shift > 4)
        fetch_one(mine, ring_at + stage * kTileBytes, src0, kTileBytes, bar_at + stage * 8);
      else
        fetch_two(mine, ring_at + stage * kTileBytes, src0, src1, kBlock, bar_at + stage * 8);
      ++in.tile;
      if (--in_left > 0) {
        if ((in.tile & 31) == 0) aim();
      } else if (in.tile == in.r.tiles) {
        in.unit += in.tile;
        if (in.unit + kSetup < w_hi) {
          in.next_group(a);
          aim();
          in_left = static_cast<int>(min(static_cast<long long>(in.r.tiles), w_hi - in.unit));
        }
      }
    };
    aim();
    for (int i = 0; i < kStages; ++i) fetch(i);

    uint32_t qf[KT][2];
    int lim[2];
    float2 unit;  // from products to scores in units of log2(e)
    State<D> st;
    const int ta = kv_frag_token(g);  // tokens of fragment rows g and g + 8: ta, ta + 8
    const int tv = (t & 1) | (t >> 1) << 1;
    const int G = a.group;
    int stage = 0;
    uint32_t phase = 0;
    bool there = false;  // the stage's tile has been seen to be there

    while (at.unit < w_hi) {
      // the group's queries, the last position each column sees, and an empty state
      const long long group = at.unit - at.tile;
      const long long off = column_offset(a, at.r, at.head, at.col, g, a.ldq);
      const uint4* src =
          reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + off + t * (D / 4));
      uint4 v[KW];
      float top = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        v[w] = off >= 0 ? load_in_order(src + w) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t x[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(bf16_lo(x[i])), fabsf(bf16_hi(x[i]))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e with top 2^e in [2^9, 2^10); rows of zeros, infinities or tiny values keep e in range
      const int e = top > 0.f && top < INFINITY
                        ? min(120, 9 + 127 - static_cast<int>(__float_as_uint(top) >> 23))
                        : 0;
      const float up = copysignf(__uint_as_float(static_cast<uint32_t>(e + 127) << 23), a.scale_log2);
      const float up16 = up * 0x1p-4f;  // of the dimensions whose keys come sixteen times as large
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const uint32_t x[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qf[2 * w + (i >> 1)][i & 1] =
              i & 1 ? pack_f16x2(bf16_lo(x[i]) * up16, bf16_hi(x[i]) * up16)
                    : pack_f16x2(bf16_lo(x[i]) * up, bf16_hi(x[i]) * up);
      }
      // (never 0, so that a masked score stays -inf)
      const float down =
          fmaxf(kKvUnit * fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23), 1e-30f);
      unit.x = __shfl_sync(0xffffffffu, down, 8 * t);
      unit.y = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // (a column past the last has zero queries and is not written: any limit does)
        const int c = at.col * kCols + 2 * t + j;
        lim[j] = at.r.template last_seen<SPANS>(min(a.token_of(c), at.r.q_len - 1));
      }
      st.minus = make_float2(-kNone, -kNone);
      st.l = make_float2(0.f, 0.f);
      const int lim_lo = at.r.template last_seen<SPANS>(a.token_of(at.col * kCols));
      const int lim_hi =
          at.r.template last_seen<SPANS>(a.token_of(min(at.r.q_len * G - 1, at.col * kCols + kCols - 1)));
#pragma unroll
      for (int m = 0; m < KT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) st.o[m][j] = 0.f;

      const int count = static_cast<int>(min(static_cast<long long>(at.r.tiles - at.tile), w_hi - at.unit));
      for (int i = 0; i < count; ++i) {
        if (!there && !dead) dead = __any_sync(0xffffffffu, !mbar_wait(bar + stage, phase, a.err));
        const int next_stage = stage == kStages - 1 ? 0 : stage + 1;
        const uint32_t next_phase = next_stage ? phase : phase ^ 1;
        there = __all_sync(0xffffffffu, mbar_peek(bar + next_stage, next_phase));
        const int pos0 = (at.tile + i) * kTile;
        if (pos0 <= lim_hi) {
          const uint8_t* tile = my_ring + stage * kTileBytes;
          float2 s[2][2];  // [block][row g, row g + 8]
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint8_t* blk = tile + k * kBlock;
            uint32_t kw[2][KW], sc[2];  // sc: the row's scales as fp16
            if constexpr (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(blk + ta * 64 + 16 * t);
              const uint4 y = *reinterpret_cast<const uint4*>(blk + (ta + 8) * 64 + 16 * t);
              kw[0][0] = x.x, kw[0][1] = x.y, kw[0][2] = x.z, kw[0][3] = x.w;
              kw[1][0] = y.x, kw[1][1] = y.y, kw[1][2] = y.z, kw[1][3] = y.w;
              const uint32_t b4 = *reinterpret_cast<const uint32_t*>(blk + kv_k_scales(D) + lane * 4);
              sc[0] = e4m3x2_to_f16x2(static_cast<uint16_t>(b4));
              sc[1] = e4m3x2_to_f16x2(static_cast<uint16_t>(b4 >> 16));
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(blk + ta * 32 + 8 * t);
              const uint2 y = *reinterpret_cast<const uint2*>(blk + (ta + 8) * 32 + 8 * t);
              kw[0][0] = x.x, kw[0][1] = x.y;
              kw[1][0] = y.x, kw[1][1] = y.y;
              const uint32_t both = e4m3x2_to_f16x2(
                  *reinterpret_cast<const uint16_t*>(blk + kv_k_scales(D) + lane * 2));
              sc[0] = both_lo(both);
              sc[1] = both_hi(both);
            }
            float acc[4];
#pragma unroll
            for (int p = 0; p < KW / 2; ++p) {  // the lane's scale groups
              Decode16 dec[2];
#pragma unroll
              for (int r = 0; r < 2; ++r)
                dec[r] = decode_scales16(D == 128 ? (p ? both_hi(sc[r]) : both_lo(sc[r])) : sc[r]);
#pragma unroll
              for (int w = 2 * p; w < 2 * p + 2; ++w) {
                uint32_t v[2][4];
                decode4(kw[0][w], dec[0], v[0]);
                decode4(kw[1][w], dec[1], v[1]);
                if (w == 0)
                  mma_f16_first(acc, v[0][0], v[1][0], v[0][1], v[1][1], qf[0][0], qf[0][1]);
                else
                  mma_f16(acc, v[0][0], v[1][0], v[0][1], v[1][1], qf[2 * w][0], qf[2 * w][1]);
                mma_f16(acc, v[0][2], v[1][2], v[0][3], v[1][3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
              }
            }
            s[k][0] = make_float2(acc[0], acc[1]);
            s[k][1] = make_float2(acc[2], acc[3]);
          }

          if (pos0 + kTile - 1 > lim_lo) {  // positions a column does not see
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int pos = pos0 + k * kKvBlock + ta + r * 8;
                if (pos > lim[0]) s[k][r].x = -INFINITY;
                if (pos > lim[1]) s[k][r].y = -INFINITY;
              }
          }
          float2 top;
          top.x = fmaxf(fmaxf(s[0][0].x, s[0][1].x), fmaxf(s[1][0].x, s[1][1].x));
          top.y = fmaxf(fmaxf(s[0][0].y, s[0][1].y), fmaxf(s[1][0].y, s[1][1].y));
          const bool over = fmaf(top.x, unit.x, st.minus.x) > kRef + kSlack ||
                            fmaf(top.y, unit.y, st.minus.y) > kRef + kSlack;
          if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
              top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, d));
              top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, d));
            }
            const float2 minus = make_float2(fminf(st.minus.x, kRef - top.x * unit.x),
                                             fminf(st.minus.y, kRef - top.y * unit.y));
            const float fx = ex2(minus.x - st.minus.x), fy = ex2(minus.y - st.minus.y);
            st.minus = minus;
            st.l.x *= fx;
            st.l.y *= fy;
#pragma unroll
            for (int d = 0; d < KT; ++d) {
              st.o[d][0] *= fx;
              st.o[d][1] *= fy;
              st.o[d][2] *= fx;
              st.o[d][3] *= fy;
            }
          }

#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint8_t* blk = tile + k * kBlock;
            uint32_t pf[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float2 x = fma2(s[k][r], unit, st.minus);
              const float2 p = make_float2(ex2(x.x), ex2(x.y));
              st.l = add2(st.l, p);
              pf[r] = transpose_8x8(pack_f16x2(p.x, p.y));
            }
            // V: lane group t's four tokens, this lane's LD dimensions
            uint32_t vw[4][VW], vs;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int token = (tv ^ (r & 1)) | (r & 1) << 2 | (r >> 1) << 3;
              if constexpr (D == 128) {
                const uint2 x = *reinterpret_cast<const uint2*>(blk + kv_v_codes(D) + token * 64 +
                                                                ((8 * g) ^ ((t >> 1) << 5)));
                vw[r][0] = x.x, vw[r][1] = x.y;
              } else {
                vw[r][0] = *reinterpret_cast<const uint32_t*>(blk + kv_v_codes(D) + token * 32 + 4 * g);
              }
            }
            vs = *reinterpret_cast<const uint32_t*>(blk + kv_v_scales(D) +
                                                    ((D == 128 ? g : g >> 1) * 4 + t) * 4);
            const Decode16 dec[2] = {
                decode_scales16(e4m3x2_to_f16x2(static_cast<uint16_t>(vs))),
                decode_scales16(e4m3x2_to_f16x2(static_cast<uint16_t>(vs >> 16)))};
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {  // 4 of the word's dimensions
                uint32_t v[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r)
                  decode4(prmt(vw[2 * r][w], vw[2 * r + 1][w], hf ? 0x7632 : 0x5410), dec[r], v[r]);
                const int m = w * 4 + hf * 2;
                mma_f16(st.o[m], v[0][0], v[0][1], v[1][0], v[1][1], pf[0], pf[1]);
                mma_f16(st.o[m + 1], v[0][2], v[0][3], v[1][2], v[1][3], pf[0], pf[1]);
              }
          }
        }

        // the stage is free: every lane has read it
        __syncwarp();
        if (!dead) fetch(stage);
        stage = next_stage;
        phase = next_phase;
      }
      const bool whole = at.tile + count == at.r.tiles && group >= w_lo;

#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) {
        st.l.x += __shfl_xor_sync(0xffffffffu, st.l.x, d);
        st.l.y += __shfl_xor_sync(0xffffffffu, st.l.y, d);
      }
      if (SPANS == kShared && whole) {  // to be joined with the other part of its rows
        const PartRows to(a, at.r.kind);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const long long row = column_offset(a, at.r, at.head, at.col, 2 * t + j, a.q_heads * D);
          if (row < 0) continue;
          if (g == 0) to.put(a, row / D, -(j ? st.minus.y : st.minus.x), j ? st.l.y : st.l.x);
          float* o = to.o + row + g * LD;
#pragma unroll
          for (int m = 0; m < KT; m += 2)
            *reinterpret_cast<float4*>(o + 2 * m) =
                make_float4(st.o[m][j], st.o[m][j + 2] * 0x1p-4f, st.o[m + 1][j], st.o[m + 1][j + 2] * 0x1p-4f);
        }
      } else if (whole) {
        const float back = kKvUnit * a.v_scale;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const long long off = column_offset(a, at.r, at.head, at.col, 2 * t + j, a.ldo);
          if (off < 0) continue;
          const float l = j ? st.l.y : st.l.x;
          const float f = l == 0.f ? 0.f : back / l, f16 = f * 0x1p-4f;
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + off + g * LD);
#pragma unroll
          for (int w = 0; w < LD / 8; ++w) {
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[i] = pack_bf16x2(st.o[4 * w + i][j] * f, st.o[4 * w + i][j + 2] * f16);
            dst[w] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      } else {
        // a piece: slot 0 began before this warp's range, slot 1 goes on after it
        const int slot = group < w_lo ? 0 : 1;
        const bool last = at.unit + (at.r.tiles - at.tile) + kSetup >= w_hi;
        float* piece = last ? reinterpret_cast<float*>(my_ring) : warp_pieces + slot * piece_floats<D>();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = 2 * t + j;
          if (g == 0) {
            piece[c] = -(j ? st.minus.y : st.minus.x);
            piece[kCols + c] = j ? st.l.y : st.l.x;
          }
          float* o = piece + 2 * kCols + c * D + g * LD;
#pragma unroll
          for (int m = 0; m < KT; m += 2)
            *reinterpret_cast<float4*>(o + 2 * m) =
                make_float4(st.o[m][j], st.o[m][j + 2] * 0x1p-4f, st.o[m + 1][j], st.o[m + 1][j + 2] * 0x1p-4f);
        }
        if (lane == 0)
          info[warp * 2 + slot] =
              PieceInfo{group, at.r.tiles, min(kCols, at.r.q_len * G - at.col * kCols), at.r.row0,
                        at.head, at.col * kCols, SPANS == kShared ? at.r.kind : kSpanWhole, piece};
      }
      if (at.unit + (at.r.tiles - at.tile) + kSetup >= w_hi) break;
      at.next_group(a);
    }
    if (dead)  // copies still in flight write this CTA's shared memory: let them land
      for (int i = 0; i < kStages; ++i) mbar_wait(bar + i, phase, a.err);
  }
  __syncthreads();

  // Join column c of n pieces, in the order of the sequence, into dst (a piece) or the output:
  // one warp, the weights 2^(m_i - max m) one piece a lane, then the weighted sum, whose loads
  // do not wait for one another.
  constexpr int kPiece = piece_floats<D>(), VL = D / 32, kAhead = 4;
  const auto join_column = [&](auto piece_of, auto load, int n, const PieceInfo& gi, int c, float* dst) {
    using Vec = std::conditional_t<VL == 4, float4, float2>;
    float o[VL] = {};
    const auto ask = [&](int k) {
      return load(reinterpret_cast<const Vec*>(piece_of(k) + 2 * kCols + c * D + lane * VL));
    };
    const auto add = [&](float w, const Vec& x) {
      o[0] += w * x.x, o[1] += w * x.y;
      if constexpr (VL == 4) o[2] += w * x.z, o[3] += w * x.w;
    };
    Vec ahead[kAhead];  // the first pieces', asked for with the maxima
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (k < n) ahead[k] = ask(k);
    float m = kNone;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, load(piece_of(i) + c));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float l = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
      float f = 0.f;
      if (i0 + lane < n) {
        const float* p = piece_of(i0 + lane);
        f = ex2(load(p + c) - m);
        l += f * load(p + kCols + c);
      }
      const int some = min(32, n - i0);
      if (i0 == 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (k < n) add(__shfl_sync(0xffffffffu, f, k), ahead[k]);
      }
#pragma unroll 8
      for (int k = i0 == 0 ? kAhead : 0; k < some; ++k) add(__shfl_sync(0xffffffffu, f, k), ask(i0 + k));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (dst) {
      if (lane == 0) {
        dst[c] = m;
        dst[kCols + c] = l;
      }
#pragma unroll
      for (int i = 0; i < VL; i += 2)
        *reinterpret_cast<float2*>(dst + 2 * kCols + c * D + lane * VL + i) = make_float2(o[i], o[i + 1]);
    } else if (SPANS == kShared) {
      const int G = a.group, token = a.token_of(gi.first_col + c);
      const PartRows to(a, gi.kind);
      const size_t row = static_cast<size_t>(gi.row0 + token) * a.q_heads + gi.head * G + gi.first_col + c - token * G;
      if (lane == 0) to.put(a, row, m, l);
#pragma unroll
      for (int i = 0; i < VL; i += 2)
        *reinterpret_cast<float2*>(to.o + row * D + lane * VL + i) = make_float2(o[i], o[i + 1]);
    } else {
      const int G = a.group, token = a.token_of(gi.first_col + c);
      const float f = l == 0.f ? 0.f : kKvUnit * a.v_scale / l;
      uint32_t* out = reinterpret_cast<uint32_t*>(
          static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(gi.row0 + token) * a.ldo +
          (gi.head * G + gi.first_col + c - token * G) * D + lane * VL);
#pragma unroll
      for (int i = 0; i < VL; i += 2) out[i / 2] = pack_bf16x2(o[i] * f, o[i + 1] * f);
    }
  };
  // The groups that several warps share, their columns dealt to the warps.  Those that other
  // CTAs share too become pieces of this CTA: 0 began before it, 1 goes on after it.
  const auto load_own = [](const auto* p) { return *p; };           // of this CTA's pieces
  const auto load_other = [](const auto* p) { return __ldcg(p); };  // of other CTAs'
  int shared_group[2] = {-1, -1}, item = 0;
  for (int i = 0; i < kWarps * 2;) {
    if (info[i].group < 0) {
      ++i;
      continue;
    }
    // its pieces: slot 0 or 1 of this warp, and slot 0 of the warps after it
    const PieceInfo gi = info[i];
    const int piece0 = i;
    int n = 1;
    while ((piece0 & ~1) + 2 * n < kWarps * 2 && info[(piece0 & ~1) + 2 * n].group == gi.group) ++n;
    i = (n == 1 ? piece0 : (piece0 & ~1) + 2 * (n - 1)) + 1;
    float* dst = nullptr;
    if (gi.group < cta_lo || gi.group + gi.tiles > cta_hi) {
      const int k = gi.group < cta_lo ? 0 : 1;
      shared_group[k] = piece0;
      dst = a.pieces + static_cast<size_t>(blockIdx.x * 2 + k) * kPiece;
    }
    for (int c = 0; c < gi.cols; ++c, ++item)
      if (item % kWarps == warp)
        join_column([&](int k) { return info[k == 0 ? piece0 : (piece0 & ~1) + 2 * k].at; }, load_own, n, gi,
                    c, dst);
  }
  if (shared_group[0] < 0 && shared_group[1] < 0) return;
  // The last CTA to arrive joins the CTAs' pieces: piece 1 of the CTA before the first of the CTAs'
  // cuts within the group, then pieces 0 of those behind them.
  const auto first_cut = [&](const PieceInfo& gi) {
    return static_cast<int>(quotient(gi.group + snap, span)) + 1;
  };
  const auto last_cut = [&](const PieceInfo& gi) {
    return static_cast<int>(quotient(gi.group + gi.tiles - snap + span - 1, span)) - 1;
  };
  __threadfence();
  __syncthreads();
  if (tid < 2 && shared_group[tid] >= 0) {
    const PieceInfo gi = info[shared_group[tid]];
    const int first = first_cut(gi), others = last_cut(gi) - first + 1;
    last_cta[tid] = atomicAdd(a.arrivals + first, 1) == others;
    if (last_cta[tid]) a.arrivals[first] = 0;
    __threadfence();
  }
  __syncthreads();
  item = 0;
  for (int k = 0; k < 2; ++k) {
    if (shared_group[k] < 0 || !last_cta[k]) continue;
    const PieceInfo gi = info[shared_group[k]];
    const int first = first_cut(gi), n = last_cut(gi) - first + 2;
    for (int c = 0; c < gi.cols; ++c, ++item)
      if (item % kWarps == warp)
        join_column([&](int x) { return a.pieces + static_cast<size_t>((first + x) * 2 - (x == 0 ? 1 : 2)) * kPiece; },
                    load_other, n, gi, c, nullptr);
  }
}

template <int D, Spans SPANS>
cudaError_t launch(const KvAttendArgs& a, cudaStream_t stream) {
  constexpr int smem = kWarps * kStages * 2 * kv_block_bytes(D);
  static int limit[kAttrDevices] = {};
  cudaError_t e = ensure_smem_limit(kv_attend_kernel<D, SPANS>, smem, limit);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(kKvMaxCtas, a.num_sms * kCtasPerSm);
  return launch_dependent(kv_attend_kernel<D, SPANS>, dim3(ctas), kThreads, smem, stream, a);
}

}  // namespace

size_t kv_attend_workspace_floats(int num_sms, int D) {
  const size_t ctas = std::min(kKvMaxCtas, num_sms * kCtasPerSm);
  return ctas * 2 * (1 + kWarps) * (D == 128 ? piece_floats<128>() : piece_floats<64>());
}

template <int D>
static cudaError_t launch_spans(const KvAttendArgs& a, cudaStream_t stream) {
  if (a.alone) return launch<D, kAlone>(a, stream);
  if (a.groups) return launch<D, kShared>(a, stream);
  return a.causal ? launch<D, kRequests>(a, stream) : launch<D, kEncoder>(a, stream);
}
cudaError_t launch_kv_attend(const KvAttendArgs& a, cudaStream_t stream) {
  return a.pages.D == 128 ? launch_spans<128>(a, stream) : launch_spans<64>(a, stream);
}

}  // namespace lora
