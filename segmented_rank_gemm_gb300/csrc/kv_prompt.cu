// kv_prompt.cu -- attention of many query rows a request over the 4-bit cache
// (include/lora_kv.h: lora_kv_attend), for requests whose rows fill tensor-core tiles.
//
// With G = q_heads / kv_heads, row c of a request and cache head is token c / G, query head
// h G + c % G.  A group is (request, head, 256 rows); over tiles of 64 cached positions, per
// half of 128 rows,
//     S = Q K^T,   P = 2^(S unit - m),   l += sum P,   O += P V
// with a running reference m per row that moves only when a score exceeds it by 2^8 (O / l does
// not depend on m) and fp32 accumulators.  K is decoded to bf16 and V to fp16, both exactly; the
// queries stay as they came, in bf16, and P is rounded to fp16 under a sum of its fp32 values (2^-11 of
// it, an eighth of the output's own rounding; 32-bit operands would halve the products' rate at least).
//
// Bound: the tensor cores, 4 D operations a score.  One CTA per SM, its warps in roles that meet
// at barriers in shared memory:
//   warps 0-3, 4-7   softmax of the rows 0..127 and 128..255, one row a thread: S from tensor
//                    memory, P back to it (the PV product takes P from there), O at the end
//   warps 8-11       decode a tile's K and V to shared memory in the 128-byte swizzled K-major
//                    layout (V transposed: its 8 x 8 blocks are transposed while they are decoded, by
//                    pairing two tokens' codes before they are extracted), and load the queries
//   warps 12, 13     issue the PV products of a half each
//   warp 14          issues the QK products, the halves in turn
//   warp 15          walks the CTA's work, announces it to the others a segment at a time, and fetches
//                    packed tiles by bulk copies, kRaw tiles ahead
// 256 rows share one decoding.  Tensor memory holds three tiles of S (the halves take them in turn),
// P and O of both halves: 192 + 64 + 256 columns at D = 128.  What costs time here are the hops
// between roles, 300 to 500 cycles each from a commit to the waiting thread's next instruction: a
// product takes 256 (PV) or 384 (QK).  With three S, the next one is under way when a softmax has
// read its own, and with P beside S rather than in its place no QK waits for a PV.
//
// Work split: a CTA claims a group at a time, larger ones first, which leaves the CTAs within about
// a small group of one another whatever the lengths are, and every group to one CTA: results do not
// depend on the order.  Where the largest group alone would outlast that (few groups, long
// contexts), the tiles of all groups form one sequence instead, cut into equal ranges for the CTAs; a
// cut near a group's edge moves there.  A group that is still cut leaves pieces (m, l, O), joined in
// order by the last CTA to arrive.
//
// Measured (32 query heads over 8 of 128): 8 prompts of 1024 tokens at up to 2048 positions 129 us,
// 110 GFLOP at 0.85 PFLOP/s, the tensor pipe at work in 40% of the cycles; cut into equal ranges
// instead of whole groups 153 us, with natural instead of falling sizes 12% more by the model.  A
// tile takes 1780 cycles, of which its products are 1365 (QK and PV of both halves from three
// warps, measured alone); a quarter of the time goes to the changes of groups, where the
// output of one, the queries of the next and its first products follow one another.
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

constexpr int kThreads = 16 * 32;  // four warpgroups, which split the registers unevenly
constexpr int kRows = 256;      // rows of a group, two halves
constexpr int kTile = 64;       // positions of a tile
constexpr int kStages = 3;      // decoded tiles of K, and of V
constexpr int kRaw = 3;         // packed tiles
// Units (a tile's time, 1780 cycles) a group counts before its tiles, what its change costs (9500
// cycles measured), and units that the pieces of a group cut in two cost (13000 each).
constexpr int kSetup = 6;
constexpr int kPieces = 15;
// The same where pieces are joined by a kernel of their own (kv_share.cu), rows of all groups at once,
// and cost what writing them does.
constexpr int kPiecesLater = 2;
// A cut this near to a group's edge moves there: a group cut in two costs its CTAs about as much as
// this many tiles, as long as that is little of a range.
__device__ __forceinline__ int snap_of(long long span, bool later) {
  return static_cast<int>(later ? min(span / 4, 2ll) : min(max(span / 12, 8ll), min(span / 4, 1ll << 20)));
}
constexpr float kRef = 6.f;     // P is 2^kRef at the reference
constexpr float kSlack = 8.f;   // how far (in powers of two) a score may exceed the reference
constexpr float kNone = -1.7e38f;
constexpr int kTmemCols = 512;
constexpr int kSerialParts = 24;

// Instruction descriptor, kind::f16: D fp32, A and B fp16 (idesc_bf16_f32: bf16), both K-major.
constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Products and commits for a whole warp to call, in convergent code, with `leader` set in one lane,
// which issues: descriptors then stay in uniform registers (a branch around them would cost a
// move to one for every operand of every product).
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one;
}
// D[tmem] (+)= A * B[smem]^T, kind::f16, A in shared memory (descriptor) or tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(leader)
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
// The tiles start at position `first`, and limits count from there: token t sees see + slope t (a
// whole causal request: 0, kv - q_len and 1).
struct Request {
  int row0, q_len, kv, rows, parts;  // rows of one head, groups of a head
  int first, see, slope, table_row;
  SpanKind kind;
};

// Request b; one that is not for this kernel has 0 rows.  (Bad ones are reported by the other
// kernel, which runs on every call.)
template <Spans SPANS>
__device__ __forceinline__ Request load_request(const KvAttendArgs& a, int b) {
  Request r;
  if constexpr (SPANS != kRequests) {
    const Span s = load_span<SPANS>(a, b, false);
    r = Request{s.row0, s.q_len, s.kv, s.q_len * a.group, 0, s.first, s.see, s.slope, s.table_row, s.kind};
    if (span_is_few(a, s)) r.rows = 0;
    r.parts = (r.rows + kRows - 1) / kRows;
    return r;
  }
  r.row0 = __ldg(a.q_offsets + b);
  const int end = __ldg(a.q_offsets + b + 1);
  // (in this order: the difference of any two offsets need not be an int)
  const bool bad = r.row0 < 0 || end < r.row0 || end > a.T || end - r.row0 > a.max_q;
  r.q_len = bad ? 0 : end - r.row0;
  const int cap = a.max_blocks << a.pages.page_shift;
  r.kv = min(max(__ldg(a.kv_len + b), 0), cap);
  r.rows = r.q_len * a.group;
  if (r.rows <= a.few_rows) r.rows = 0;
  r.parts = (r.rows + kRows - 1) / kRows;
  r.first = 0;
  r.see = r.kv - r.q_len;
  r.slope = 1;
  r.table_row = b;
  r.kind = kSpanWhole;
  return r;
}
// Tiles of a request's group `part`: up to the last position its last row sees.
__device__ __forceinline__ int group_tiles(const KvAttendArgs& a, const Request& r, int part) {
  const int last = r.see + r.slope * a.token_of(min((part + 1) * kRows, r.rows) - 1);
  return max(last, 0) / kTile + 1;  // (last may be next to 2^31)
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

// The first of a request's groups (their tiles grow with the part) of at least `tiles` tiles;
// r.parts if there is none.
__device__ __forceinline__ int first_part(const KvAttendArgs& a, const Request& r, int tiles) {
  if (tiles <= 1) return 0;
  // its last row's token sees position kTile (tiles - 1)
  const long long token = static_cast<long long>(kTile) * (tiles - 1) - r.see;
  if (token <= 0) return 0;
  if (token >= r.q_len || r.slope == 0) return r.parts;
  return static_cast<int>(token) * a.group / kRows;
}
// Groups are dealt whole in kBuckets classes of size, the largest first: the least tiles of class i
// when the largest group has `most`.
constexpr int kBuckets = 4;
__device__ __forceinline__ int bucket_least(int most, int i) {
  return i == kBuckets - 1 ? 1 : (most * (kBuckets - 1 - i) + kBuckets - 1) / kBuckets;
}
// Parts [lo, hi) of a request are in class i.
__device__ __forceinline__ int2 bucket_parts(const KvAttendArgs& a, const Request& r, int most, int i) {
  return make_int2(first_part(a, r, bucket_least(most, i)),
                   i == 0 ? r.parts : first_part(a, r, bucket_least(most, i - 1)));
}

// A position in the sequence of tiles, and the tile's unit.
template <Spans SPANS>
struct Cursor {
  Request r;
  int b, head, part, tile, tiles;
  long long unit;
  // The tile at or after unit `at`, the rem-th of request b_; a cut near a group's edge moves
  // there (to the group's end by tile = tiles, one past its last).  One warp.
  __device__ __forceinline__ void start(const KvAttendArgs& a, int b_, long long rem, long long at,
                                        int snap, int lane) {
    b = b_;
    r = load_request<SPANS>(a, b);
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
          r = load_request<SPANS>(a, b);
        } while (r.parts == 0);
      }
    }
    tiles = group_tiles(a, r, part);
  }
};

// A CTA's range of the sequence, walked a segment (one group's tiles tile .. tile + count - 1) at a
// time.
template <Spans SPANS>
struct Walk {
  Cursor<SPANS> at;
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
};
// A segment as the roles see it.
struct Segment {
  int count;      // tiles; 0: there is no more
  int tile;       // the first, in the group
  int tiles;      // of the group
  int rows;       // of the group, at most 256
  int first_row;  // its first row in the request
  int row0;       // the request's first row in q and out
  int see, slope;  // token t of the request sees positions 0 .. see + slope t, from its first on
  int head;
  SpanKind kind;
  long long unit;  // of the group's first tile
};

// Floats of a piece: m, l [256], O [256][D].
template <int D>
constexpr int piece_floats() {
  return kv_prompt_piece_floats(D);
}
static_assert(kRows == kKvPromptRows, "the rows of a piece");

constexpr int kScratchWarp = 4096;  // a softmax warp's 32 rows of 128 bytes, on their way out
template <int D>
struct Smem {
  static constexpr int kQHalf = 128 * D * 2;     // one half's queries
  static constexpr int kKv = kTile * D * 2;      // one decoded tile of K or V
  static constexpr int kK = 2 * kQHalf, kV = kK + kStages * kKv;
  static constexpr int kRawTile = kTile / kKvBlock * kv_block_bytes(D);
  static constexpr int kRaws = kV + kStages * kKv;
  static constexpr int kScratch = kRaws + kRaw * kRawTile;
  static constexpr int kBytes = kScratch + 8 * kScratchWarp + 1024;  // + alignment
};
constexpr int kSegments = 4;       // announced ahead
constexpr int kSegmentReaders = 15;  // warps

// The barriers; [phase] of a ring or of a half's tiles.  (arrivals)
struct Barriers {
  uint64_t seg_full[kSegments], seg_empty[kSegments];  // (1) (kSegmentReaders)
  uint64_t raw_full[kRaw], raw_empty[kRaw];            // (bytes) (128)
  uint64_t k_full[kStages], k_empty[kStages];          // (128) (commit)
  uint64_t v_full[kStages], v_empty[kStages];          // (128) (2: a commit a half)
  uint64_t q_full[2], q_free;                          // (128) (commit of a segment's last QK)
  // S: full by a half's own tiles (a half without rows in a segment would lose count of a place's
  // phases), of which up to three are ahead of its softmax; read by place.
  uint64_t s_full[2][3], s_read[3];                    // (commit) (128)
  uint64_t p_full[2], pv_done[2];                      // (128) (commit)
  uint64_t meet, idle[3];                              // (256) (commit)
};

template <int D, Spans SPANS>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(KvAttendArgs a) {
  using L = Smem<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* const sm = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  __shared__ Barriers bar;
  __shared__ Segment segments[kSegments];
  __shared__ uint32_t tmem_holder;
  __shared__ long long scan[kThreads / 32], cut_rem[2];
  __shared__ int cut_b[2];
  __shared__ int warp_most[kThreads / 32], bucket_count[kBuckets][kThreads / 32];
  __shared__ int last_cta;
  __shared__ float2 row_join[kRows];  // of a shared group's rows: max m, factor of O

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = a.pages.heads, G = a.group;

  int job = 0;  // the first group to claim, asked for early
  if (warp == 15 && lane == 0) job = atomicAdd(a.prompt_claim, 1);
  if (warp == 12) tmem_alloc(&tmem_holder, kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < kSegments; ++i) mbar_init(&bar.seg_full[i], 1), mbar_init(&bar.seg_empty[i], kSegmentReaders);
    for (int i = 0; i < kRaw; ++i) mbar_init(&bar.raw_full[i], 1), mbar_init(&bar.raw_empty[i], 128);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.k_full[i], 128), mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_full[i], 128), mbar_init(&bar.v_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i)
      mbar_init(&bar.q_full[i], 128), mbar_init(&bar.p_full[i], 128), mbar_init(&bar.pv_done[i], 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bar.s_full[0][i], 1), mbar_init(&bar.s_full[1][i], 1);
      mbar_init(&bar.s_read[i], 128), mbar_init(&bar.idle[i], 1);
    }
    mbar_init(&bar.q_free, 1);
    mbar_init(&bar.meet, 256);
    fence_mbar_init();
  }

  // The sequence's length and this CTA's cuts.  A thread sums a run of consecutive requests; those
  // with many groups are summed by its warp, one after the other (16 requests of 7 groups each, which
  // are one warp's, took 4 us longer when a thread summed 4 groups at most).
  const int count_b = SPANS == kShared ? a.B + a.groups : a.B;
  const int per = (count_b + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, count_b), b1 = min(b0 + per, count_b);
  int most = 0;  // tiles of the largest group
  const auto request_units = [&](int b, bool mine) {  // of request b (mine), by all lanes
    Request r = {};
    if (mine) r = load_request<SPANS>(a, b);
    if (r.parts) most = max(most, group_tiles(a, r, r.parts - 1));
    long long n = 0;
    if (r.parts <= kSerialParts)
      for (int part = 0; part < r.parts; ++part) n += part_units(a, r, part);
    for (unsigned big = __ballot_sync(0xffffffffu, r.parts > kSerialParts); big; big &= big - 1) {
      const int k = __ffs(big) - 1;
      Request x;
      x.see = __shfl_sync(0xffffffffu, r.see, k);
      x.slope = SPANS != kRequests ? __shfl_sync(0xffffffffu, r.slope, k) : 1;
      x.rows = __shfl_sync(0xffffffffu, r.rows, k);
      x.parts = __shfl_sync(0xffffffffu, r.parts, k);
      const long long sum = head_units(a, x, lane);
      if (lane == k) n = sum;
    }
    return n * heads;
  };
  long long mine = 0;
  for (int i = 0; i < per; ++i) mine += request_units(b0 + i, b0 + i < b1);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) warp_most[warp] = most;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  long long total = 0, before = incl - mine;
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
    most = max(most, warp_most[w]);
  }
  const long long span = max(static_cast<long long>(kSetup + 4), quotient(total + gridDim.x - 1, gridDim.x));
  const bool later = SPANS == kShared;  // pieces of rows in two parts are joined with those
  const int snap = snap_of(span, later);
  // Whole groups, claimed one by one, unless the largest would outlast the rest by more than its
  // cutting costs.
  const bool whole = most + kSetup <= span + (later ? kPiecesLater : kPieces);
  if (whole) {
#pragma unroll 1
    for (int i = 0; i < kBuckets; ++i) {
      int n = 0;
      for (int b = b0; b < b1; ++b) {
        const int2 parts = bucket_parts(a, load_request<SPANS>(a, b), most, i);
        n += (parts.y - parts.x) * heads;
      }
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) bucket_count[i][warp] = n;
    }
  }
#pragma unroll 1
  for (int i = 0; i < (whole ? 0 : 2); ++i) {
    const long long at = span * (blockIdx.x + i);
    const bool here = at >= before && at < before + mine;
    if (!__any_sync(0xffffffffu, here)) continue;
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
  }
  __syncthreads();
  const uint32_t tS = tmem, tP = tmem + 192, tO = tmem + 256;
  bool ok = true;  // no wait of this role has run out

  // (one instruction a warpgroup)
  if (warp < 8) setmaxnreg_inc<168>();
  else if (warp < 12) setmaxnreg_dec<112>();
  else setmaxnreg_dec<64>();

  // The next segment, as this warp's seg-th; its place is given back.
  uint32_t seg = 0;
  const auto next_segment = [&](Segment& s) {
    if (!ok) return false;
    const uint32_t at = seg % kSegments;
    ok = mbar_wait(&bar.seg_full[at], seg / kSegments & 1, a.err);
    ok = __all_sync(0xffffffffu, ok);
    s = segments[at];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.seg_empty[at]);
    ++seg;
    return ok && s.count > 0;
  };

  if (warp < 8) {
    // ---------------- softmax ----------------
    const int half = warp >> 2, row = tid & 127;  // this thread's row of the half
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t p_at = tP + lanes + half * 32, o_at = tO + lanes + half * D;
    uint8_t* const scratch = sm + L::kScratch + warp * kScratchWarp;
    // from products to scores in units of log2(e); never 0, so that a masked score stays -inf (with
    // a scale of 0 the keys are decoded to zeros)
    const float unit = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
    // the softmax warps wait for one another, bounded like every wait
    uint32_t meetings = 0;
    auto meet_all = [&]() {
      mbar_arrive(&bar.meet);
      ok = mbar_wait(&bar.meet, meetings++ & 1, a.err);
      ok = __all_sync(0xffffffffu, ok);
    };
    uint32_t step = 0, n = 0;  // S tiles of both halves, tiles of this half
    Segment g = {};
    while (next_segment(g)) {
      const int halves = g.rows > 128 ? 2 : 1;
      const bool active = half < halves;
      float m = kNone, l = 0.f;
      if (active) {
        // the last position this row sees, from the segment's first tile on (a row past the
        // last is written nowhere)
        const int lim = g.see + (SPANS != kRequests ? g.slope : 1) * a.token_of(g.first_row + min(half * 128 + row, g.rows - 1)) -
                        g.tile * kTile;
        uint32_t at = (step + half) % 3;  // S's place
        for (int j = 0; j < g.count; ++j, ++n) {
          uint32_t pv_there = 1;  // the product before has been seen to be done
          ok = mbar_wait(&bar.s_full[half][n % 3], n / 3 & 1, a.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          uint32_t s[2][32];
          tmem_ld_32x32b_x32(tS + lanes + at * 64, s[0]);
          tmem_ld_32x32b_x32(tS + lanes + at * 64 + 32, s[1]);
          tmem_ld_wait();
          tc_fence_before();
          mbar_arrive(&bar.s_read[at]);
          at += halves;
          if (at >= 3) at -= 3;
          const int left = lim - j * kTile;  // the tile's positions 0..left are seen
          if (__any_sync(0xffffffffu, left < kTile - 1)) {
#pragma unroll
            for (int i = 0; i < kTile; ++i)
              if (i > left) s[i >> 5][i & 31] = 0xFF800000u;
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kTile; ++i)
            top[i & 3] = fmaxf(top[i & 3], __uint_as_float(s[i >> 5][i & 31]));
          const float peak = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * unit;
          const bool move = __any_sync(0xffffffffu, peak > m + (kRef + kSlack));
          float f = 1.f;
          if (move) {
            const float moved = fmaxf(m, peak - kRef);
            f = ex2(m - moved);
            m = moved;
            l *= f;
          }
          const float2 by = make_float2(unit, unit), minus = make_float2(-m, -m);
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
            // (as late as spares the wait: at the tile's start it is not done yet)
            if (i == 23 && n > 0) pv_there = mbar_peek(&bar.pv_done[half], (n - 1) & 1);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          // the product before is done: P's place is free, and O may be rescaled
          if (!pv_there) {
            ok = mbar_wait(&bar.pv_done[half], (n - 1) & 1, a.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          tc_fence_after();
          tmem_st_32x32b_x32(p_at, p);
          if (move && j > 0) {
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
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&bar.p_full[half]);
        }
      }
      if (!ok) break;
      step += g.count * halves;

      if (active) {
        ok = mbar_wait(&bar.pv_done[half], (n - 1) & 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      const bool whole = g.tile == 0 && g.count == g.tiles;
      // this CTA's piece of a group it shares: 0 began before it, 1 goes on after it
      float* const piece = a.prompt_pieces +
                           static_cast<size_t>(blockIdx.x * 2 + (g.tile > 0 ? 0 : 1)) * piece_floats<D>();
      if (active) {
        // 128 bytes of every row at a time, from one row a lane to 8 lanes a row
        // (raw: fp32 as it is, to a piece or to be joined with the other part of its rows)
        const bool part = SPANS == kShared && whole, raw = SPANS == kShared || !whole;
        const float f = raw ? 1.f : l == 0.f ? 0.f : kKvUnit * a.v_scale / l;
        const float2 by = make_float2(f, f), none = make_float2(0.f, 0.f);
        const auto at = [&](int x, int k) {  // 16-byte piece k of row x
          return reinterpret_cast<uint4*>(scratch + x * 128 + ((k ^ (x & 7)) << 4));
        };
        // where they go: from the group's first token (or row of the piece) on, in bytes
        const int first_token = a.token_of(g.first_row);
        const PartRows to(a, g.kind);
        const size_t first_row = static_cast<size_t>(g.row0 + first_token) * a.q_heads + g.head * G;  // of the parts
        uint8_t* const base =
            part     ? reinterpret_cast<uint8_t*>(to.o + first_row * D)
            : whole ? reinterpret_cast<uint8_t*>(static_cast<__nv_bfloat16*>(a.out) +
                                                 static_cast<size_t>(g.row0 + first_token) * a.ldo + g.head * G * D)
                    : reinterpret_cast<uint8_t*>(piece + 2 * kRows);
        const int x0 = half * 128 + (warp & 3) * 32;
        const bool all = x0 + 32 <= g.rows;
        uint8_t* dst[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t x = x0 + i * 4 + (lane >> 3), c = g.first_row + x, token = a.token_of(c);
          const uint32_t row_bytes = part ? a.q_heads * (D * 4u) : whole ? static_cast<uint32_t>(a.ldo) * 2 : 0;
          const uint32_t in_row = whole ? (c - token * G) * (part ? D * 4 : D * 2) : x * (D * 4);
          dst[i] = base + static_cast<uint64_t>(token - first_token) * row_bytes + in_row + (lane & 7) * 16;
        }
        const auto put = [&](const uint32_t (&o)[32], int off) {  // 32 words of this lane's row
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *at(lane, k) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          __syncwarp();
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = *at(i * 4 + (lane >> 3), lane & 7);
          if (all) {
#pragma unroll
            for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dst[i] + off) = v[i];
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (x0 + i * 4 + (lane >> 3) < g.rows) *reinterpret_cast<uint4*>(dst[i] + off) = v[i];
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int d = 0; d < D; d += 64) {
          uint32_t o[2][32];
          tmem_ld_32x32b_x32(o_at + d, o[0]);
          tmem_ld_32x32b_x32(o_at + d + 32, o[1]);
          tmem_ld_wait();
          if (!raw) {
            uint32_t x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float2 y = fma2(make_float2(__uint_as_float(o[i >> 4][2 * i & 31]),
                                                __uint_as_float(o[i >> 4][(2 * i & 31) + 1])),
                                    by, none);
              x[i] = pack_bf16x2(y.x, y.y);
            }
            put(x, d * 2);
          } else {
            put(o[0], d * 4);
            put(o[1], d * 4 + 128);
          }
        }
        tc_fence_before();
        if (!whole) {
          piece[half * 128 + row] = m;
          piece[kRows + half * 128 + row] = l;
        }
        // (a group that is cut names its pieces for each of its rows, in the CTA with the first one)
        if (SPANS == kShared && (whole || g.tile == 0) && half * 128 + row < g.rows) {
          const int c = g.first_row + half * 128 + row, token = a.token_of(c);
          const int first_cut = whole ? 0 : static_cast<int>(quotient(g.unit + snap, span)) + 1;
          const int last_cut = whole ? 0 : static_cast<int>(quotient(g.unit + g.tiles - snap + span - 1, span)) - 1;
          const size_t at_row = first_row + static_cast<size_t>(token - first_token) * a.q_heads + c - token * G;
          if (whole) to.put(a, at_row, m, l);
          else to.ml[at_row] = KvPieces(first_cut, last_cut - first_cut + 2, half * 128 + row).packed(to.all);
        }
      }
      if (SPANS != kShared && !whole) {
        // The cuts within the group, as their CTAs see them, and the pieces between them: the
        // first cut's CTA before it (piece 1), then pieces 0.
        const int first_cut = static_cast<int>(quotient(g.unit + snap, span)) + 1;
        const int last_cut = static_cast<int>(quotient(g.unit + g.tiles - snap + span - 1, span)) - 1;
        const int pieces = last_cut - first_cut + 2;
        __threadfence();
        meet_all();
        if (!ok) break;
        if (tid == 0) {
          last_cta = atomicAdd(a.prompt_arrivals + first_cut, 1) == pieces - 1;
          if (last_cta) a.prompt_arrivals[first_cut] = 0;
          __threadfence();
        }
        meet_all();
        if (!ok) break;
        if (last_cta) {
          const auto piece_of = [&](int i) {
            return a.prompt_pieces +
                   static_cast<size_t>(kv_prompt_piece(first_cut, i)) * piece_floats<D>();
          };
          // a row's maximum and the factor of its sum first, one row a thread
          if (tid < g.rows) {
            float top = kNone, sum = 0.f;
#pragma unroll 4
            for (int i = 0; i < pieces; ++i) top = fmaxf(top, __ldcg(piece_of(i) + tid));
#pragma unroll 4
            for (int i = 0; i < pieces; ++i)
              sum += ex2(__ldcg(piece_of(i) + tid) - top) * __ldcg(piece_of(i) + kRows + tid);
            row_join[tid] = make_float2(top, sum == 0.f ? 0.f : kKvUnit * a.v_scale / sum);
          }
          meet_all();
          if (!ok) break;
          // then a row a warp, four at a time
#pragma unroll 1
          for (int x0 = warp; x0 < g.rows; x0 += 32) {
            float o[4][D / 32] = {};
            for (int i = 0; i < pieces; ++i) {
              const float* const piece_i = piece_of(i);
              float w[4];
              float2 y[4][D / 64];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int x = min(x0 + k * 8, g.rows - 1);
                w[k] = __ldcg(piece_i + x);
#pragma unroll
                for (int d = 0; d < D / 64; ++d)
                  y[k][d] = __ldcg(reinterpret_cast<const float2*>(piece_i + 2 * kRows + x * D) + d * 32 + lane);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float f = ex2(w[k] - row_join[min(x0 + k * 8, g.rows - 1)].x);
#pragma unroll
                for (int d = 0; d < D / 64; ++d) {
                  o[k][2 * d] += f * y[k][d].x;
                  o[k][2 * d + 1] += f * y[k][d].y;
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int x = x0 + k * 8;
              if (x >= g.rows) break;
              const float f = row_join[x].y;
              const int c = g.first_row + x, token = a.token_of(c);
              uint32_t* out = reinterpret_cast<uint32_t*>(
                  static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(g.row0 + token) * a.ldo +
                  (g.head * G + c - token * G) * D);
#pragma unroll
              for (int d = 0; d < D / 64; ++d)
                out[d * 32 + lane] = pack_bf16x2(o[k][2 * d] * f, o[k][2 * d + 1] * f);
            }
          }
        }
        meet_all();  // last_cta is read
        if (!ok) break;
      }
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
    const int v_half = vo & 1;              // the octet's half of its block
    const uint32_t sel_lo = vo & 1 ? 0x1054u : 0x5410u, sel_hi = vo & 1 ? 0x3276u : 0x7632u;
    const uint32_t sel[2] = {vd & 1 ? sel_hi : sel_lo, vd & 1 ? sel_lo : sel_hi};
    const bool swap = D == 128 && kc >= 2;  // these lanes decode their last 16 dimensions first
    // 2^120, with the sign of the softmax's scale (whose size the scores are multiplied by); 0 for 0
    const uint32_t k_unit = a.scale_log2 < 0.f ? 0xFB80FB80u : a.scale_log2 > 0.f ? 0x7B807B80u : 0u;
    uint32_t n = 0;  // tiles decoded
    Segment g = {};
    // A segment's queries, copied a row's 16-byte pieces on consecutive lanes (rows past the last are
    // zero), in two steps: asked for, and handed over.
    const auto ask_q = [&]() {
      constexpr int LR = D / 8, RI = 128 / LR;  // lanes a row, rows a step
      const int x0 = t / LR, p = t % LR;
      if (seg > 1) ok = mbar_wait(&bar.q_free, seg & 1, a.err);  // of the segment before
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const __nv_bfloat16* const q = static_cast<const __nv_bfloat16*>(a.q) +
                                     static_cast<size_t>(g.row0) * a.ldq + g.head * G * D + p * 8;
      uint8_t* const dst = sm + (p >> 3) * (128 * 128) + x0 * 128 + (((p & 7) ^ (x0 & 7)) << 4);
      const int rows = g.rows > 128 ? 256 : 128;
#pragma unroll 4
      for (int i = 0; i < rows / RI; ++i) {
        const int x = i * RI + x0, c = min(g.first_row + x, g.first_row + g.rows - 1), token = a.token_of(c);
        cp_async_16_zfill(dst + (x >> 7) * L::kQHalf + (i * RI & 127) * 128,
                          q + static_cast<size_t>(token) * a.ldq + (c - token * G) * D, x < g.rows ? 16 : 0);
      }
    };
    const auto hand_q = [&]() {
      cp_async_wait_all();
      fence_proxy_async_smem();
      mbar_arrive(&bar.q_full[0]);
      if (g.rows > 128) mbar_arrive(&bar.q_full[1]);
    };
    while (next_segment(g)) {
      // The queries: asked for as soon as the products with those before are seen to be done, and
      // behind two tiles at the latest (which need no product with them: three tiles fit the
      // stages); handed over a tile later.
      const int q_last = seg == 1 ? 0 : min(2, g.count);
      bool asked = false, handed = false;
      const auto hand_once = [&]() {
        if (asked && !handed) hand_q();
        handed = asked;
      };
      for (int j = 0; j <= g.count; ++j) {
        hand_once();
        if (!asked && (j == q_last || __any_sync(0xffffffffu, mbar_peek(&bar.q_free, seg & 1)))) {
          ask_q();
          asked = true;
        }
        if (!ok) break;
        if (j == g.count) {
          hand_once();
          break;
        }
        const int stage = n % kStages, parity = (n / kStages) & 1, slot = n % kRaw;
        const uint32_t raw_there = mbar_peek(&bar.raw_full[slot], (n / kRaw) & 1),
                       k_free = mbar_peek(&bar.k_empty[stage], parity ^ 1),
                       v_free = mbar_peek(&bar.v_empty[stage], parity ^ 1);
        if (!raw_there) ok = mbar_wait(&bar.raw_full[slot], (n / kRaw) & 1, a.err);
        const uint8_t* const tile = sm + L::kRaws + slot * L::kRawTile;
        uint32_t kw[KT][4], ks[KT];  // ks: the two groups' scales in bytes 0 and 1
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          const int token = kt + i * (128 / KC), in = token & 15, fr = kv_token_frag(in);
          const uint8_t* blk = tile + (token >> 4) * kv_block_bytes(D);
          const uint4 x = *reinterpret_cast<const uint4*>(blk + in * (D / 2) + kc * 16);
          kw[i][0] = swap ? x.z : x.x, kw[i][1] = swap ? x.w : x.y;
          kw[i][2] = swap ? x.x : x.z, kw[i][3] = swap ? x.y : x.w;
          if constexpr (D == 128) {
            const uint32_t two = *reinterpret_cast<const uint16_t*>(
                blk + kv_k_scales(D) + (fr & 7) * 16 + kc * 4 + (fr >> 3) * 2);
            ks[i] = swap ? prmt(two, 0u, 0x4401) : two;
          } else {
            ks[i] = prmt(*reinterpret_cast<const uint32_t*>(blk + kv_k_scales(D) + (fr & 7) * 8 + kc * 4),
                         0u, fr >> 3 ? 0x4431 : 0x4420);
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
        mbar_arrive(&bar.raw_empty[slot]);
        if (!k_free) ok = ok && mbar_wait(&bar.k_empty[stage], parity ^ 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // K: rows of tokens
        uint8_t* const k_sm = sm + L::kK + stage * L::kKv;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          const int token = kt + i * (128 / KC);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const DecodeBf16 dec = decode_scale_bf16(ks[i], half, k_unit);
#pragma unroll
            for (int x = 2 * half; x < 2 * half + 2; ++x) {
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
        mbar_arrive(&bar.k_full[stage]);
        // V: rows of dimensions, 8 tokens a chunk
        if (!v_free) ok = mbar_wait(&bar.v_empty[stage], parity ^ 1, a.err);
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
        mbar_arrive(&bar.v_full[stage]);
        ++n;
      }
    }
  } else if (warp < 14) {
    // ---------------- PV products ----------------
    // Descriptors advance by constants, 32 bytes (2 units) a 16-wide step.
    constexpr uint32_t kDesc = idesc_f16_f32(128, D);
    const uint32_t leader = elect_leader();
    const int half = warp - 12;
    const uint32_t p_at = tP + half * 32, o_at = tO + half * D;
    const uint64_t v_desc = smem_desc_sw128(smem_u32(sm) + L::kV);
    uint32_t stage = 0, turn = 0, n = 0;  // of the next tile; tiles of this half
    Segment g = {};
    while (next_segment(g)) {
      const bool active = half == 0 || g.rows > 128;
      for (int j = 0; j < g.count; ++j) {
        const uint32_t v_there = mbar_peek(&bar.v_full[stage], turn);
        if (active) ok = mbar_wait(&bar.p_full[half], n & 1, a.err);
        if (!v_there) ok = ok && mbar_wait(&bar.v_full[stage], turn, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (active) {
          tc_fence_after();
          const uint64_t vd = v_desc + stage * (L::kKv >> 4);
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            mma_ts(o_at, p_at + ks * 8, vd + ks * 2, kDesc, ks > 0 ? 1 : j, leader);
          commit(&bar.pv_done[half], leader);
          commit(&bar.v_empty[stage], leader);
          ++n;
        } else if (leader) {
          mbar_arrive(&bar.v_empty[stage]);  // no rows: the stages pass by
        }
        if (++stage == kStages) stage = 0, turn ^= 1;
      }
    }
    // every product issued is done before the CTA's memory goes
    commit(&bar.idle[half], leader);
    mbar_wait(&bar.idle[half], 0, a.err);
  } else if (warp == 14) {
    // ---------------- QK products ----------------
    constexpr uint32_t kDesc = idesc_bf16_f32(128, kTile);
    const uint32_t leader = elect_leader();
    const uint64_t q_desc = smem_desc_sw128(smem_u32(sm)), k_desc = smem_desc_sw128(smem_u32(sm) + L::kK);
    uint32_t stage = 0, turn = 0;           // of the next tile of K
    uint32_t at = 0, phase = 0;             // of the next S's place
    uint32_t n[2] = {0, 0}, groups1 = 0;    // the halves' next s_full; groups of half 1
    bool used = false;                      // S's places have been used
    Segment g = {};
    while (next_segment(g)) {
      const int halves = g.rows > 128 ? 2 : 1;
      ok = mbar_wait(&bar.q_full[0], (seg - 1) & 1, a.err);
      if (halves == 2) ok = ok && mbar_wait(&bar.q_full[1], groups1++ & 1, a.err);
      ok = __all_sync(0xffffffffu, ok);
      uint32_t k_there = 0, free = 0;  // what was seen ahead
      for (int j = 0; j < g.count && ok; ++j) {
        if (!k_there) ok = mbar_wait(&bar.k_full[stage], turn, a.err);
        const uint32_t k_stage = stage;
        if (++stage == kStages) stage = 0, turn ^= 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= halves) break;
          if (used && !free) ok = ok && mbar_wait(&bar.s_read[at], phase ^ 1, a.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t s_at = tS + at * 64;
          if (++at == 3) at = 0, phase ^= 1, used = true;
          free = used ? mbar_peek(&bar.s_read[at], phase ^ 1) : 1;
          if (h == halves - 1) k_there = mbar_peek(&bar.k_full[stage], turn);
          uint64_t qd = q_desc + h * (L::kQHalf >> 4), kd = k_desc + k_stage * (L::kKv >> 4);
#pragma unroll
          for (int slab = 0; slab < D / 64; ++slab) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) mma_ss(s_at, qd + ks * 2, kd + ks * 2, kDesc, slab > 0 || ks > 0, leader);
            qd += 128 * 128 >> 4;
            kd += kTile * 128 >> 4;
          }
          commit(&bar.s_full[h][n[h]], leader);
          if (++n[h] == 3) n[h] = 0;
        }
        commit(&bar.k_empty[k_stage], leader);
      }
      commit(&bar.q_free, leader);
    }
    commit(&bar.idle[2], leader);
    mbar_wait(&bar.idle[2], 0, a.err);
  } else {
    // ---------------- the walk and the packed tiles ----------------
    const int shift = a.pages.page_shift;
    const int step = min(kTile, 1 << shift);          // positions of a copy
    const bool copies = lane * kKvBlock < kTile && lane * kKvBlock % step == 0;
    const uint32_t bytes = step / kKvBlock * kv_block_bytes(D);
    Walk<SPANS> walk;
    bool some = false;
    // Whole groups: a lane's two counts of a warp's requests in a class, classes first, and the
    // groups up to them.
    static_assert(kBuckets * (kThreads / 32) == 64, "two counts a lane");
    const int* const counts = &bucket_count[0][0];
    const int count0 = whole ? counts[2 * lane] : 0, count1 = whole ? counts[2 * lane + 1] : 0;
    const auto scan_lanes = [&](int v) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += x;
      }
      return v;
    };
    const int upto = scan_lanes(count0 + count1);
    // The job-th group, for every lane.
    const auto take = [&]() {
      job = __shfl_sync(0xffffffffu, job, 0);
      unsigned beyond = __ballot_sync(0xffffffffu, job < upto);
      if (!beyond) return false;
      int k = __ffs(beyond) - 1;
      int rem = job - __shfl_sync(0xffffffffu, upto - count0 - count1, k);
      const int c0 = __shfl_sync(0xffffffffu, count0, k);
      int entry = 2 * k;
      if (rem >= c0) rem -= c0, ++entry;
      const int bucket = entry / (kThreads / 32), first = entry % (kThreads / 32) * 32;
      // the thread of that warp whose requests have it, then the request
      const int x0 = min((first + lane) * per, count_b), x1 = min(x0 + per, count_b);
      int n = 0;
      for (int b = x0; b < x1; ++b) {
        const int2 parts = bucket_parts(a, load_request<SPANS>(a, b), most, bucket);
        n += (parts.y - parts.x) * heads;
      }
      const int incl = scan_lanes(n);
      k = __ffs(__ballot_sync(0xffffffffu, rem < incl)) - 1;
      rem -= __shfl_sync(0xffffffffu, incl - n, k);
      Cursor<SPANS>& c = walk.at;
      int2 parts;
      for (c.b = (first + k) * per;; ++c.b) {
        c.r = load_request<SPANS>(a, c.b);
        parts = bucket_parts(a, c.r, most, bucket);
        n = (parts.y - parts.x) * heads;
        if (rem < n) break;
        rem -= n;
      }
      c.head = rem / (parts.y - parts.x);
      c.part = parts.y - 1 - (rem - c.head * (parts.y - parts.x));
      c.tile = 0;
      c.unit = 0;
      c.tiles = walk.count = group_tiles(a, c.r, c.part);
      return true;
    };
    if (whole) {
      some = take();
    } else if (span * blockIdx.x < total) {
      walk.end = total;
      if (span * (blockIdx.x + 1) < total) {
        walk.at.start(a, cut_b[1], cut_rem[1], span * (blockIdx.x + 1), snap, lane);
        walk.end = walk.at.unit;
      }
      walk.at.start(a, cut_b[0], cut_rem[0], span * blockIdx.x, blockIdx.x == 0 ? 0 : snap, lane);
      some = walk.first(a);
    }
    uint32_t n = 0;
    while (ok) {
      // announce the segment, or the end
      const uint32_t place = seg % kSegments;
      ok = mbar_wait(&bar.seg_empty[place], (seg / kSegments & 1) ^ 1, a.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const Cursor<SPANS>& c = walk.at;
      const int rows = some ? min(kRows, c.r.rows - c.part * kRows) : 0;
      if (lane == 0) {
        segments[place] = some ? Segment{walk.count, c.tile, c.tiles, rows, c.part * kRows, c.r.row0,
                                         c.r.see, c.r.slope, c.head, c.r.kind, c.unit - c.tile}
                               : Segment{};
        mbar_arrive(&bar.seg_full[place]);
      }
      __syncwarp();
      ++seg;
      if (!some) break;
      if (seg > 1) {  // its queries to L2: they are read behind the segment before
        const int last = a.token_of(c.part * kRows + rows - 1);
        for (int token = a.token_of(c.part * kRows) + lane; token <= last; token += 32)
          bulk_prefetch_l2(static_cast<const __nv_bfloat16*>(a.q) +
                               static_cast<size_t>(c.r.row0 + token) * a.ldq + c.head * G * D,
                           G * D * 2);
      }
      const int32_t* const pages = a.table + static_cast<size_t>(c.r.table_row) * a.max_blocks;
      const unsigned last_page = max(0, (c.r.kv - 1) >> shift);  // the request's
      // the page of a tile's position (of the last page past the end: masked, and within the cache)
      const auto page_of = [&](int j) {
        const unsigned pos = c.r.first + (c.tile + j) * kTile + lane * static_cast<unsigned>(kKvBlock);
        return copies && c.r.kv > c.r.first ? __ldg(pages + min(pos >> shift, last_page)) : 0;
      };
      int id = page_of(0);
      for (int j = 0; j < walk.count; ++j, ++n) {
        const int slot = n % kRaw;
        const int next_id = j + 1 < walk.count ? page_of(j + 1) : 0;
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.pages.num_pages)) {
          atomicOr(a.err, LORA_ERRF_BAD_ID);
          id = 0;
        }
        ok = mbar_wait(&bar.raw_empty[slot], ((n / kRaw) & 1) ^ 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar.raw_full[slot], L::kRawTile);
        __syncwarp();
        if (copies) {
          const int pos = (c.tile + j) * kTile + lane * kKvBlock;
          bulk_load_g2s(sm + L::kRaws + slot * L::kRawTile + lane * kv_block_bytes(D),
                        a.pages.base + a.pages.block(id, c.head, (pos & ((1 << shift) - 1)) / kKvBlock),
                        bytes, &bar.raw_full[slot]);
        }
        id = next_id;
      }
      if (!ok) break;
      if (whole) {
        if (lane == 0) job = atomicAdd(a.prompt_claim, 1);
        some = take();
      } else {
        some = walk.next(a);
      }
    }
    // the last CTA to have claimed sets the counts back
    if (lane == 0) {
      __threadfence();
      if (atomicAdd(a.prompt_claim + 1, 1) == static_cast<int>(gridDim.x) - 1) {
        a.prompt_claim[0] = 0;
        a.prompt_claim[1] = 0;
      }
    }
    // copies in flight write this CTA's memory: every one issued has landed when its slot's
    // barrier has turned
    for (uint32_t i = n > kRaw ? n - kRaw : 0; i < n; ++i)
      mbar_wait(&bar.raw_full[i % kRaw], (i / kRaw) & 1, a.err);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, kTmemCols);
  // the kernel for few rows, ahead of this one, may still be at work: what follows in the stream
  // waits for this one alone
  griddep_wait();
}

template <int D, Spans SPANS>
cudaError_t launch(const KvAttendArgs& a, cudaStream_t stream) {
  static int limit[kAttrDevices] = {};
  cudaError_t e = ensure_smem_limit(kv_prompt_kernel<D, SPANS>, Smem<D>::kBytes, limit);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv_prompt_kernel<D, SPANS>, dim3(std::min(kKvMaxCtas, a.num_sms)), kThreads,
                          Smem<D>::kBytes, stream, a);
}

}  // namespace

size_t kv_prompt_workspace_floats(int num_sms, int D) {
  return static_cast<size_t>(std::min(kKvMaxCtas, num_sms)) * 2 *
         (D == 128 ? piece_floats<128>() : piece_floats<64>());
}

template <int D>
static cudaError_t launch_spans(const KvAttendArgs& a, cudaStream_t stream) {
  if (a.groups) return launch<D, kShared>(a, stream);
  return a.causal ? launch<D, kRequests>(a, stream) : launch<D, kEncoder>(a, stream);
}
cudaError_t launch_kv_prompt(const KvAttendArgs& a, cudaStream_t stream) {
  return a.pages.D == 128 ? launch_spans<128>(a, stream) : launch_spans<64>(a, stream);
}

}  // namespace lora
