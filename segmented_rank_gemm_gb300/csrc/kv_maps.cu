// kv_maps.cu -- block tables and slot maps of a batch from its requests' lengths, and the
// return of finished requests' pages (include/lora_kv.h: lora_kv_maps, lora_kv_release).
//
// Everything follows from two prefix sums over the requests,
//     off_b   = sum_{a<b} new_a                                  (rows of the token arrays)
//     first_b = sum_{a<b} ceil(end_a / P) - ceil(len_a / P)      (pages taken before b)
// Page j of the batch's new pages is free[n_free - 1 - j], and row t belongs to the request
// with off_b <= t < off_{b+1}, found by bisection.  A token on a new page takes its id from
// the stack itself, not from the table entry another thread writes, so no step waits for
// another and the call is one kernel.
//
// Bound: latency.  A decode step of 512 requests moves 16 KB; what takes time is the chain
// launch -> lengths -> prefix sums -> bisection -> table -> store.  So every CTA repeats the
// prefix sums (the lengths come from L2) and keeps them in shared memory; batches of at most
// kRowsPerCta rows run in one CTA.  Larger ones split rows and pages over CTAs; the
// last CTA to finish writes kv_len and the counts, which may overwrite inputs the others read.
// Measured: 512 single tokens 4.1 us, 520 requests with 3247 rows 5.5, 2999 with 42455 7.7; with
// four rows a thread the last two take 6.9 and 10.9, with half the threads idle (512 a CTA) the
// first takes 5.4.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "lora_common.cuh"
#include "lora_kernels.h"
#include "lora_kv.h"

namespace lora {
namespace {

constexpr int kThreads = 1024;
constexpr int kRowsPerCta = 1024;  // one a thread: a row is a chain of loads
constexpr int kMaxCtas = 128;
constexpr int kMaxRequests = 16384;
constexpr int kMaxRows = 1 << 20;

constexpr int kBadLength = 1, kNoPages = 2, kBadPage = 4;  // error flags of counts[3]
constexpr int kPagesInUse = 4;                             // and, with the first two, of a release

struct MapsArgs {
  const int32_t *len, *add, *adapter;
  int B, T, page_shift;
  int32_t* table;
  int max_blocks;
  const int32_t* free_pages;
  int stack_size;
  const int32_t* n_free;
  int32_t *kv_len, *q_offsets, *position, *kv_slot, *token_slot, *counts;
};

__device__ __forceinline__ long long warp_inclusive_sum(long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Exclusive sums over the CTA's kThreads threads of two non-negative values, and the totals.
// warp_sums: 2 x 32 entries of shared memory.
__device__ __forceinline__ void cta_exclusive_sums(long long& a, long long& b, long long& total_a,
                                                   long long& total_b, long long (*warp_sums)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long ia = warp_inclusive_sum(a, lane), ib = warp_inclusive_sum(b, lane);
  if (lane == 31) {
    warp_sums[0][warp] = ia;
    warp_sums[1][warp] = ib;
  }
  __syncthreads();
  if (warp == 0) {
    const long long sa = warp_inclusive_sum(warp_sums[0][lane], lane);
    const long long sb = warp_inclusive_sum(warp_sums[1][lane], lane);
    warp_sums[0][lane] = sa;
    warp_sums[1][lane] = sb;
  }
  __syncthreads();
  total_a = warp_sums[0][kThreads / 32 - 1];
  total_b = warp_sums[1][kThreads / 32 - 1];
  a = ia - a + (warp ? warp_sums[0][warp - 1] : 0);
  b = ib - b + (warp ? warp_sums[1][warp - 1] : 0);
}

// The last index i in [0, n) with prefix[i] <= v (prefix ascending, prefix[0] = 0 <= v): the
// owner of v, past owners of nothing.
__device__ __forceinline__ int owner(const int32_t* prefix, int n, int v) {
  int lo = 0, hi = n;  // prefix[lo] <= v < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Whether the page's slots are int32 values.  (Whether a cache has the page is for the calls
// on the cache to check: one table serves the caches of all blocks.)
__device__ __forceinline__ bool page_ok(int page, int page_shift) {
  return page >= 0 && page < INT_MAX >> page_shift;
}

__global__ void __launch_bounds__(kThreads) kv_maps_kernel(MapsArgs a) {
  griddep_wait();
  extern __shared__ int32_t smem[];
  int32_t* off = smem;              // [B + 1]
  int32_t* first = smem + a.B + 1;  // [B + 1]
  __shared__ long long warp_sums[2][32];
  __shared__ int last_cta;
  const int tid = threadIdx.x;
  const int P = 1 << a.page_shift;
  const long long cap = static_cast<long long>(a.max_blocks) << a.page_shift;

  // the requests' sums, a run of consecutive requests a thread
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  long long rows = 0, pages = 0;
  int bad = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {  // (no branch in it: its loads are asked for together)
    const int len = a.len[b], add = a.add[b];
    const long long end = static_cast<long long>(len) + add;
    const bool good = len >= 0 && add >= 0 && end <= cap;
    bad |= !good;
    rows += good ? add : 0;
    pages += good ? ((end + P - 1) >> a.page_shift) -
                        ((len + static_cast<long long>(P) - 1) >> a.page_shift)
                  : 0;
  }
  const int n_free = *a.n_free;
  long long row0 = rows, page0 = pages, all_rows, all_pages;
  cta_exclusive_sums(row0, page0, all_rows, all_pages, warp_sums);
  int flags = __syncthreads_or(bad) ? kBadLength : 0;
  if (all_rows > a.T) flags |= kBadLength;
  if (n_free < 0 || n_free > a.stack_size || all_pages > n_free) flags |= kNoPages;
  const bool fits = flags == 0;
  const int n_rows = fits ? static_cast<int>(all_rows) : 0;
  const int n_pages = fits ? static_cast<int>(all_pages) : 0;
  if (fits) {
    int r = static_cast<int>(row0), p = static_cast<int>(page0);
    for (int b = b0; b < b1; ++b) {
      const int len = a.len[b], end = len + a.add[b];
      off[b] = r;
      first[b] = p;
      r += end - len;
      p += ((end + P - 1) >> a.page_shift) - ((len + P - 1) >> a.page_shift);
    }
    if (tid == 0) {
      off[a.B] = n_rows;
      first[a.B] = n_pages;
    }
  }
  __syncthreads();

  const int step = gridDim.x * kThreads, t0 = blockIdx.x * kThreads + tid;
  bool bad_page = false;
  // the pages taken
  for (int j = t0; j < n_pages; j += step) {
    const int b = owner(first, a.B, j);
    const int have = (a.len[b] + P - 1) >> a.page_shift;
    const int page = a.free_pages[n_free - 1 - j];
    bad_page |= !page_ok(page, a.page_shift);
    a.table[static_cast<size_t>(b) * a.max_blocks + have + (j - first[b])] = page;
  }
  // the rows
  for (int t = t0; t < a.T; t += step) {
    int pos = 0, slot = -1, adapter = -1;
    if (t < n_rows) {
      const int b = owner(off, a.B, t);
      const int len = a.len[b];
      if (a.adapter) adapter = a.adapter[b];
      pos = len + (t - off[b]);
      const int have = (len + P - 1) >> a.page_shift, blk = pos >> a.page_shift;
      const int page = blk < have ? a.table[static_cast<size_t>(b) * a.max_blocks + blk]
                                  : a.free_pages[n_free - 1 - (first[b] + blk - have)];
      if (page_ok(page, a.page_shift))
        slot = (page << a.page_shift) + (pos & (P - 1));
      else
        bad_page = true;
    }
    a.position[t] = pos;
    a.kv_slot[t] = slot;
    a.token_slot[t] = adapter;
  }
  for (int b = t0; b <= a.B; b += step) a.q_offsets[b] = fits ? off[b] : 0;

  // The flags travel with the CTAs' tickets: flag bits above the ticket count.
  if (__syncthreads_or(bad_page)) flags |= kBadPage;
  if (gridDim.x > 1) {
    if (tid == 0) {
      __threadfence();
      if (flags & kBadPage) atomicOr(a.counts + 4, kBadPage << 16);
      const int seen = atomicAdd(a.counts + 4, 1);
      last_cta = (seen & 0xffff) == static_cast<int>(gridDim.x) - 1;
      __threadfence();
      if (last_cta) flags |= seen >> 16;
    }
    __syncthreads();
    if (!last_cta) return;
  }
  if (fits) {
    for (int b = tid; b < a.B; b += kThreads) a.kv_len[b] = a.len[b] + (off[b + 1] - off[b]);
  } else if (a.kv_len != a.len) {
    for (int b = tid; b < a.B; b += kThreads) a.kv_len[b] = a.len[b];
  }
  if (tid == 0) {
    a.counts[0] = n_rows;
    a.counts[1] = n_free - n_pages;
    a.counts[2] = n_pages;
    a.counts[3] = flags;
    a.counts[4] = 0;
  }
}

// shared: positions at the start of a request that are not its own (whole pages), or null.  A request that
// stays and shares pages of one that is done has them at the same places of its row (a fork copies them
// there), the first of that one's own pages among them, which is nobody else's: one comparison a pair of
// such requests.  (11 done of 512 requests, the rest sharers: 4.4 us, 3.2 without the comparisons; 60 of 3000:
// 16 us, 4.3.)
__global__ void __launch_bounds__(kThreads)
    kv_release_kernel(const int32_t* __restrict__ done, int32_t* __restrict__ len, int32_t* __restrict__ shared,
                      int B, int page_shift, const int32_t* __restrict__ table, int max_blocks,
                      int32_t* __restrict__ free_pages, int stack_size, int32_t* n_free,
                      int32_t* status) {
  extern __shared__ int32_t first[];  // [B + 1], with `shared` [2 (B + 1)]
  __shared__ long long warp_sums[2][32];
  const int tid = threadIdx.x;
  const int P = 1 << page_shift;
  const long long cap = static_cast<long long>(max_blocks) << page_shift;
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  long long pages = 0, none = 0;
  int bad = 0;
  const auto kept = [&](int b) { return shared ? shared[b] >> page_shift : 0; };  // pages that stay
  for (int b = b0; b < b1; ++b) {
    if (!done[b]) continue;
    const int n = len[b], s = shared ? shared[b] : 0;
    if (n < 0 || n > cap || s < 0 || s > n || (s & (P - 1))) bad = 1;
    else pages += ((n + static_cast<long long>(P) - 1) >> page_shift) - kept(b);
  }
  const int held = *n_free;
  long long page0 = pages, all, unused;
  cta_exclusive_sums(page0, none, all, unused, warp_sums);
  int flags = __syncthreads_or(bad) ? kBadLength : 0;
  if (held < 0 || held + all > stack_size) flags |= kNoPages;
  if (shared && flags == 0) {
    // of those that are done, the place of the first own page and the page
    __shared__ int n_done;
    if (tid == 0) n_done = 0;
    __syncthreads();
    for (int b = b0; b < b1; ++b) {
      if (!done[b] || len[b] <= shared[b]) continue;
      const int i = atomicAdd(&n_done, 1), at = kept(b);
      first[2 * i] = at;
      first[2 * i + 1] = table[static_cast<size_t>(b) * max_blocks + at];
    }
    __syncthreads();
    int used = 0;
    for (int c = tid; n_done > 0 && c < B; c += kThreads) {
      if (done[c]) continue;
      const int pages_shared = kept(c);
      int place = 0;  // of its row, and the page there (most requests that are done own all of their pages)
      int32_t page = pages_shared > 0 ? table[static_cast<size_t>(c) * max_blocks] : 0;
      for (int i = 0; i < (pages_shared > 0 ? n_done : 0); ++i) {
        const int at = first[2 * i];
        if (at >= pages_shared) continue;
        if (at != place) page = table[static_cast<size_t>(c) * max_blocks + (place = at)];
        used |= page == first[2 * i + 1];
      }
    }
    if (__syncthreads_or(used)) flags |= kPagesInUse;
  }
  if (flags == 0) {
    int p = static_cast<int>(page0);
    for (int b = b0; b < b1; ++b) {
      first[b] = p;
      if (!done[b]) continue;
      p += ((len[b] + P - 1) >> page_shift) - kept(b);
      len[b] = 0;
    }
    if (tid == 0) first[B] = static_cast<int>(all);
    __syncthreads();
    for (int j = tid; j < static_cast<int>(all); j += kThreads) {
      const int b = owner(first, B, j);
      free_pages[held + j] = table[static_cast<size_t>(b) * max_blocks + kept(b) + (j - first[b])];
    }
    if (shared) {
      __syncthreads();  // shared has been read
      for (int b = b0; b < b1; ++b)
        if (done[b]) shared[b] = 0;
    }
  }
  if (tid == 0) {
    if (flags == 0) *n_free = held + static_cast<int>(all);
    *status = flags;
  }
}

// One CTA, as a fork changes little: its requests are checked, then a warp copies a row at a time.
__global__ void __launch_bounds__(kThreads)
    kv_fork_kernel(const int32_t* __restrict__ parent, const int32_t* __restrict__ want, int32_t* len,
                   int32_t* shared, int B, int page_shift, int32_t* table, int max_blocks, int32_t* status) {
  const int tid = threadIdx.x, lane = tid & 31;
  const long long cap = static_cast<long long>(max_blocks) << page_shift;
  int bad = 0;
  for (int b = tid; b < B; b += kThreads) {
    const int p = parent[b];
    if (p < 0) {
      bad |= p != -1;
      continue;
    }
    bad |= p >= B || len[b] != 0 || (want && want[b] < 0);
    if (p < B) bad |= parent[p] != -1 || len[p] < 0 || len[p] > cap;
  }
  const int flags = __syncthreads_or(bad) ? kBadLength : 0;
  if (flags == 0) {
    for (int b = tid >> 5; b < B; b += kThreads / 32) {
      const int p = parent[b];
      if (p < 0) continue;
      const int whole = len[p] >> page_shift;  // (a parent's length does not change here)
      const int pages = want ? min(want[b] >> page_shift, whole) : whole;
      for (int j = lane; j < pages; j += 32)
        table[static_cast<size_t>(b) * max_blocks + j] = table[static_cast<size_t>(p) * max_blocks + j];
      if (lane == 0) len[b] = shared[b] = pages << page_shift;
    }
  }
  if (tid == 0) *status = flags;
}

int page_shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

bool table_ok(int B, int page_size, int max_blocks, int stack_size) {
  return B >= 1 && B <= kMaxRequests && page_shift_of(page_size) >= 0 && max_blocks >= 1 &&
         static_cast<long long>(B) * max_blocks <= INT_MAX &&
         static_cast<long long>(max_blocks) * page_size <= INT_MAX && stack_size >= 1;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

int lora_kv_maps(const int32_t* len_dev, const int32_t* new_dev, const int32_t* adapter_dev, int B,
                 int T, int page_size, int32_t* block_table, int max_blocks,
                 const int32_t* free_pages, int stack_size, const int32_t* n_free_dev,
                 int32_t* kv_len, int32_t* q_offsets, int32_t* position, int32_t* kv_slot,
                 int32_t* token_slot, int32_t* counts, void* stream) {
  if (!table_ok(B, page_size, max_blocks, stack_size) || T < 0 || T > kMaxRows) return LORA_EINVAL;
  if (!len_dev || !new_dev || !block_table || !free_pages || !n_free_dev || !kv_len ||
      !q_offsets || !counts || (T > 0 && (!position || !kv_slot || !token_slot)))
    return LORA_EINVAL;
  MapsArgs a{len_dev, new_dev, adapter_dev, B, T, page_shift_of(page_size), block_table, max_blocks,
             free_pages, stack_size, n_free_dev, kv_len, q_offsets, position, kv_slot, token_slot,
             counts};
  const int smem = 2 * (B + 1) * static_cast<int>(sizeof(int32_t));
  static int limit[kAttrDevices] = {};
  if (smem > 40 * 1024 && ensure_smem_limit(kv_maps_kernel, smem, limit) != cudaSuccess)
    return LORA_ECUDA;
  const int ctas = std::min(kMaxCtas, std::max(1, (std::max(T, B) + kRowsPerCta - 1) / kRowsPerCta));
  return launch_dependent(kv_maps_kernel, dim3(ctas), kThreads, smem, static_cast<cudaStream_t>(stream),
                          a) == cudaSuccess
             ? LORA_OK
             : LORA_ECUDA;
}

namespace {

int release(const int32_t* done_dev, int32_t* len_dev, int32_t* shared_dev, int B, int page_size,
            const int32_t* block_table, int max_blocks, int32_t* free_pages, int stack_size,
            int32_t* n_free_dev, int32_t* status_dev, void* stream) {
  if (!table_ok(B, page_size, max_blocks, stack_size)) return LORA_EINVAL;
  if (!done_dev || !len_dev || !block_table || !free_pages || !n_free_dev || !status_dev)
    return LORA_EINVAL;
  const int smem = (shared_dev ? 2 : 1) * (B + 1) * static_cast<int>(sizeof(int32_t));
  static int limit[kAttrDevices] = {};
  if (smem > 40 * 1024 && ensure_smem_limit(kv_release_kernel, smem, limit) != cudaSuccess)
    return LORA_ECUDA;
  kv_release_kernel<<<1, kThreads, smem, static_cast<cudaStream_t>(stream)>>>(
      done_dev, len_dev, shared_dev, B, page_shift_of(page_size), block_table, max_blocks, free_pages, stack_size,
      n_free_dev, status_dev);
  return cudaGetLastError() == cudaSuccess ? LORA_OK : LORA_ECUDA;
}

}  // namespace

int lora_kv_release(const int32_t* done_dev, int32_t* len_dev, int B, int page_size,
                    const int32_t* block_table, int max_blocks, int32_t* free_pages,
                    int stack_size, int32_t* n_free_dev, int32_t* status_dev, void* stream) {
  return release(done_dev, len_dev, nullptr, B, page_size, block_table, max_blocks, free_pages, stack_size,
                 n_free_dev, status_dev, stream);
}

int lora_kv_release_shared(const int32_t* done_dev, int32_t* len_dev, int32_t* shared_dev, int B,
                           int page_size, const int32_t* block_table, int max_blocks,
                           int32_t* free_pages, int stack_size, int32_t* n_free_dev,
                           int32_t* status_dev, void* stream) {
  if (!shared_dev) return LORA_EINVAL;
  return release(done_dev, len_dev, shared_dev, B, page_size, block_table, max_blocks, free_pages, stack_size,
                 n_free_dev, status_dev, stream);
}

int lora_kv_fork(const int32_t* parent_dev, const int32_t* want_dev, int32_t* len_dev,
                 int32_t* shared_dev, int B, int page_size, int32_t* block_table, int max_blocks,
                 int32_t* status_dev, void* stream) {
  if (!table_ok(B, page_size, max_blocks, 1)) return LORA_EINVAL;
  if (!parent_dev || !len_dev || !shared_dev || !block_table || !status_dev) return LORA_EINVAL;
  kv_fork_kernel<<<1, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      parent_dev, want_dev, len_dev, shared_dev, B, page_shift_of(page_size), block_table, max_blocks, status_dev);
  return cudaGetLastError() == cudaSuccess ? LORA_OK : LORA_ECUDA;
}

}  // extern "C"
