// kv_span.cuh -- what the attention kernels' span variants run over (include/lora_kv.h:
// lora_kv_attend_shared, lora_kv_attend_cross).
//
// A span is a run of consecutive query rows and a run of cached positions from a page's start on.  A
// call's spans are its groups' prefixes (the rows of all members, which see all of it) and then its
// requests (their rows, over what lies behind the prefix).  Where a request has no prefix, its span
// gives its output; else the two spans' results meet in kv_share.cu, by the rule for a softmax
// over two sets of positions: with p = 2^(s - m), o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kv_decode.cuh"
#include "kv_kernels.h"
#include "lora_kernels.h"

namespace lora {

// What a variant of the attention kernels runs over.
enum Spans {
  kRequests = 0,  // whole causal requests
  kEncoder = 1,   // requests whose rows see all of them
  kShared = 2,    // groups' prefixes and requests, whose results are joined
  kAlone = 3      // whole causal requests, with groups that are checked but not used
};
enum SpanKind { kSpanWhole = 0, kSpanTail = 1, kSpanPrefix = 2 };

struct Span {
  int row0, q_len;  // its rows; one with bad offsets has none
  int first, kv;    // positions first .. kv - 1, of the request in row `table_row` of the table
  int see, slope;   // its token t sees positions first .. first + see + slope t
  int table_row;
  SpanKind kind;
};

// Span v of a call's groups + B (or B), checked.
template <Spans S>
__device__ __forceinline__ Span load_span(const KvAttendArgs& a, int v, bool report) {
  Span s;
  const int cap = a.max_blocks << a.pages.page_shift, in_page = (1 << a.pages.page_shift) - 1;
  bool bad;
  if (S == kShared && v < a.groups) {
    int from = load_in_order(a.group_offsets + v), to = load_in_order(a.group_offsets + v + 1);
    bad = from < 0 || to < from || to > a.B;
    s.table_row = load_in_order(a.prefix_row + v);
    s.kv = load_in_order(a.prefix_len + v);
    bad = bad || s.table_row < 0 || s.table_row >= a.B || s.kv < 0 || s.kv > cap || (s.kv & in_page);
    if (bad) from = to = 0;
    s.row0 = load_in_order(a.q_offsets + from);
    const int end = load_in_order(a.q_offsets + to);
    bad = bad || s.row0 < 0 || end < s.row0 || end > a.T;
    s.q_len = bad || s.kv == 0 ? 0 : end - s.row0;
    if (bad) s.kv = s.table_row = 0;
    s.first = 0;
    s.see = s.kv - 1;
    s.slope = 0;
    s.kind = kSpanPrefix;
  } else {
    const int b = S == kShared ? v - a.groups : v;
    s.row0 = load_in_order(a.q_offsets + b);
    const int end = load_in_order(a.q_offsets + b + 1);
    s.kv = load_in_order(a.kv_len + b);
    const int share = S != kEncoder ? load_in_order(a.shared + b) : 0;
    // (in this order: the difference of any two offsets need not be an int)
    bad = s.row0 < 0 || end < s.row0 || end > a.T || end - s.row0 > a.max_q;
    s.q_len = bad ? 0 : end - s.row0;
    if (s.kv < 0 || s.kv > cap) {
      bad = true;
      s.kv = min(max(s.kv, 0), cap);
    }
    // every row of a request sees all of its group's prefix, whose pages are whole
    bad = bad || (s.q_len > 0 && (share < 0 || (share & in_page) || share > max(0, s.kv - s.q_len)));
    s.first = S == kAlone ? 0 : min(max(share, 0), s.kv) & ~in_page;
    s.see = (S != kEncoder ? s.kv - s.q_len : s.kv - 1) - s.first;
    s.slope = S != kEncoder ? 1 : 0;
    s.table_row = b;
    s.kind = s.first > 0 ? kSpanTail : kSpanWhole;
  }
  if (bad && report) atomicOr(a.err, LORA_ERRF_BAD_ID);
  return s;
}

// Whether a span is the kernel for few rows' (kv_attend.cu) or the one for many's (kv_prompt.cu): by rows, as
// the requests of lora_kv_attend are.  (Parts of rows with two spans to the former also with up to 64 rows where
// they are short spare the latter changes of groups, but fill the former: 61 requests of 4 to 7 tokens behind
// shared prefixes 67.2 us so and 72.8 by rows, but 64 requests of 7 tokens over 384 positions of their own 91 and
// 62, and 40 batches drawn with 2 to 49 requests of 4 to 7 tokens 12% longer by their mean.)
__device__ __forceinline__ bool span_is_few(const KvAttendArgs& a, const Span& s) {
  return s.q_len * a.group <= a.few_rows;
}

// The groups agree with their requests: one with a prefix is a member, and has its group's.
__device__ __forceinline__ void check_group_of(const KvAttendArgs& a, int b) {
  if (load_in_order(a.q_offsets + b + 1) <= load_in_order(a.q_offsets + b)) return;
  const int share = load_in_order(a.shared + b);
  if (share <= 0) return;
  int lo = 0, hi = a.groups;  // the last group that starts at b or before
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (load_in_order(a.group_offsets + mid) <= b) lo = mid;
    else hi = mid;
  }
  if (b < load_in_order(a.group_offsets + lo) || b >= load_in_order(a.group_offsets + lo + 1) ||
      share != load_in_order(a.prefix_len + lo))
    atomicOr(a.err, LORA_ERRF_BAD_ID);
}

// Group v is as it should be, and its prefix's pages are the cache's.
__device__ __forceinline__ void check_prefix_pages(const KvAttendArgs& a, int v, int first, int step) {
  const Span s = load_span<kShared>(a, v, true);
  for (int j = first; j < s.kv >> a.pages.page_shift; j += step)
    if (static_cast<unsigned>(load_in_order(a.table + static_cast<size_t>(s.table_row) * a.max_blocks + j)) >=
        static_cast<unsigned>(a.pages.num_pages))
      atomicOr(a.err, LORA_ERRF_BAD_ID);
}

// Pieces of the kernel for many rows (kv_prompt.cu): m [256], l [256], O [256][D]; a CTA has two, and
// the i-th of a group that is first cut in front of CTA first_cut is this one.
constexpr int kKvPromptRows = 256;
__host__ __device__ constexpr int kv_prompt_piece_floats(int D) { return kKvPromptRows * (D + 2); }
__host__ __device__ constexpr int kv_prompt_piece(int first_cut, int i) {
  return i == 0 ? (first_cut - 1) * 2 + 1 : (first_cut + i - 1) * 2;
}
// In the place of a row's (m, l), told apart by l (a sum is not negative): its group's result is `count`
// pieces, where it is row `row`; with `only`, there is no other part of the row.
struct KvPieces {
  int first_cut, count, row;
  __device__ __forceinline__ KvPieces(int first_cut_, int count_, int row_)
      : first_cut(first_cut_), count(count_), row(row_) {}
  __device__ __forceinline__ explicit KvPieces(float2 ml) {
    const uint32_t v = __float_as_uint(ml.x);
    first_cut = v >> 21, count = v >> 10 & 0x7FF, row = v & 0x3FF;
  }
  static __device__ __forceinline__ bool are(float2 ml) { return ml.y == -1.f || ml.y == -2.f; }
  static __device__ __forceinline__ bool only(float2 ml) { return ml.y == -2.f; }
  __device__ __forceinline__ float2 packed(bool only) const {
    return make_float2(__uint_as_float(static_cast<uint32_t>(first_cut) << 21 | count << 10 | row), only ? -2.f : -1.f);
  }
};
// Or O is all of the row's result, and the output is it times f.
__device__ __forceinline__ float2 kv_row_times(float f) { return make_float2(f, -3.f); }
__device__ __forceinline__ bool kv_is_row_times(float2 ml) { return ml.y == -3.f; }
static_assert(kKvMaxCtas < 1 << 11 && kKvPromptRows <= 1 << 10, "what KvPieces holds");

// A result's factor: what O times is the output.
__device__ __forceinline__ float kv_factor(const KvAttendArgs& a, float l) {
  return l == 0.f ? 0.f : kKvUnit * a.v_scale / l;
}
// Where a span's unnormalised results go: row r's head h at index r q_heads + h.
struct PartRows {
  float* o;    // [.][D]
  float2* ml;  // m, l
  __device__ __forceinline__ PartRows(const KvAttendArgs& a, SpanKind kind)
      : o(a.part_o[kind == kSpanPrefix]), ml(a.part_ml[kind == kSpanPrefix]), all(kind == kSpanWhole) {}
  bool all;  // the span is all of its rows
  __device__ __forceinline__ void put(const KvAttendArgs& a, size_t row, float m, float l) const {
    ml[row] = all ? kv_row_times(kv_factor(a, l)) : make_float2(m, l);
  }
};

}  // namespace lora
