/*
 * lora_kv.h -- C ABI of a paged key/value cache held in 4 bits, the attention that reads it,
 * and the block tables and slot maps of a batch, on GB300 (sm_103a).
 *
 * These are the steps between the q/k/v and output projections of a decoder block whose
 * projections are lora_layer.h's layers.  One batch mixes prompts and single tokens:
 *
 *   lora_kv_maps      per batch: from each request's cached and new token counts, the pages
 *                     it takes, and per new token its position, its cache slot and its
 *                     request's adapter slot (what set_batch_segments takes)
 *   lora_kv_append    per block: the new tokens' keys and values into the cache
 *   lora_kv_attend    per block: their queries over everything their requests have cached
 *   lora_kv_release   finished requests' pages back to the free stack
 *
 * The conventions of lora_layer.h hold: "stream" is a cudaStream_t passed as void*; calls
 * enqueue work and return without synchronising except where they say so; LORA_OK or a
 * negative lora_status (lora_layer.h) is returned; host-detectable errors enqueue nothing;
 * device-detectable errors never trap but raise a flag.  No call but lora_kv_cache_create
 * allocates; every other one can be captured in a CUDA graph.  The current device has to be the
 * one a cache was created on (LORA_EINVAL else), and the arrays' own.
 *
 * Pages.  A page holds page_size consecutive positions of one request, for every head.
 * block_table [B, max_blocks] int32 names request b's pages in order; entries past
 * ceil(length / page_size) are not read.  Slot page * page_size + i is position i of a page.
 *
 * The 4-bit format.  16 consecutive dimensions of one token and head share a scale
 *     s = e4m3( max|x| / (7 g) ),   nearest even, at most 448
 * with g the cache's k_scale or v_scale; their codes are n = round(x / (s g)) in -7 .. 7
 * (ties to even; 0 where s is 0), and n s g is the value held.  Divisions are fp32, correctly
 * rounded.  NaN elements count as 0, infinities saturate.  A symmetric uniform code is used
 * because it decodes in one logic and one fused multiply-add instruction a pair, exactly
 * (n s has at most 7 significant bits), and because its error on a group of 16 is below that of
 * a 4-bit float of the same size.  At 4.5 bits an element the cache takes 0.28 of bf16's bytes.
 */
#ifndef LORA_KV_H
#define LORA_KV_H

#include <stdint.h>

#include "lora_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct lora_kv_cache lora_kv_cache_t; /* opaque */

/*
 * The maps of one batch of B requests, and the pages their new tokens need.
 *   len_dev      [B] tokens each request has cached; new_dev [B] tokens it adds (0: idle).
 *   adapter_dev  [B] each request's adapter slot (-1: base only), or NULL (all -1).
 *   T            rows of the token arrays; the batch's new tokens may be fewer (padding).
 *   block_table  [B, max_blocks], entries below ceil(len / page_size) valid; the entries of
 *                pages taken are written.
 *   free_pages   [stack_size] a stack of free page ids, n_free_dev [1] its height.  Pages are
 *                taken from the top, in request order.
 * Outputs, with end[b] = len[b] + new[b]:
 *   kv_len [B] = end; may be len_dev.
 *   q_offsets [B + 1]: request b's tokens are rows q_offsets[b] .. q_offsets[b+1] - 1.
 *   position [T], kv_slot [T], token_slot [T]: each row's position in its request, its
 *     cache slot, its adapter slot; 0, -1, -1 for rows past the batch's tokens.
 *   counts [5]: tokens, height of the stack afterwards, pages taken, error flags, and a
 *     word the call itself uses: zero before the first call and after every one.
 *     n_free_dev may be counts + 1.
 * A batch that does not fit takes nothing (a request beyond max_blocks pages, too few
 * free pages, more than T tokens, a negative count): kv_len = len, q_offsets all zero, every
 * kv_slot -1, and counts[3] nonzero (1: counts or lengths, 2: pages).
 * counts[3] also has 4 where a page id used is negative or its slots pass 2^31; its tokens
 * alone get kv_slot -1.  (Ids a cache does not have are flagged by the calls on the cache.)
 * Limits: 1 <= B <= 16384, 0 <= T <= 1 << 20, page_size one of 16, 32, 64, 128, 256,
 * max_blocks >= 1, stack_size >= 1; B * max_blocks and max_blocks * page_size below 2^31.
 * Errors: LORA_EINVAL, LORA_ECUDA.
 */
int lora_kv_maps(const int32_t* len_dev, const int32_t* new_dev, const int32_t* adapter_dev, int B,
                 int T, int page_size, int32_t* block_table, int max_blocks,
                 const int32_t* free_pages, int stack_size, const int32_t* n_free_dev,
                 int32_t* kv_len, int32_t* q_offsets, int32_t* position, int32_t* kv_slot,
                 int32_t* token_slot, int32_t* counts, void* stream);

/*
 * The pages of every request with done_dev[b] != 0 go back on the stack, in request
 * order, and its len_dev[b] becomes 0.
 *   len_dev [B], block_table, free_pages, n_free_dev (updated), stack_size: as lora_kv_maps.
 *   status_dev [1]: 0, or 1 (a length is negative or past max_blocks pages) or 2 (the stack
 *   would exceed stack_size); then nothing is released.
 * Errors: LORA_EINVAL, LORA_ECUDA.
 */
int lora_kv_release(const int32_t* done_dev, int32_t* len_dev, int B, int page_size,
                    const int32_t* block_table, int max_blocks, int32_t* free_pages,
                    int stack_size, int32_t* n_free_dev, int32_t* status_dev, void* stream);

/*
 * Create a cache of num_pages pages for kv_heads heads of head_dim dimensions.
 *   head_dim 64 or 128; page_size 16, 32, 64, 128 or 256; 1 <= kv_heads <= 256;
 *   1 <= num_pages; num_pages * page_size < 2^31; 1 <= max_requests <= 16384: the most
 *   requests of an attention call; k_scale, v_scale: positive, and finite times 7 (up to 4.8e37).
 * The pages are zero (value 0) until written; the call synchronises `stream`.  The cache
 * owns its pages and the attention's workspace.
 * Errors: LORA_EINVAL, LORA_ENOMEM, LORA_ECUDA (then *out is NULL).
 */
int lora_kv_cache_create(lora_kv_cache_t** out, int num_pages, int page_size, int kv_heads,
                         int head_dim, int max_requests, float k_scale, float v_scale,
                         void* stream);

/*
 * Write T tokens.  k_dev and v_dev: rows of kv_heads * head_dim bf16, ldk and ldv elements
 * apart (multiples of 8; the pointers 16-byte aligned).  kv_slot_dev [T]: each row's slot;
 * a row with slot -1 is skipped, one with another slot outside the cache is skipped and
 * flagged.  Slots of one call are distinct.  Errors: LORA_EINVAL, LORA_ECUDA.
 */
int lora_kv_append(lora_kv_cache_t* cache, const void* k_dev, int ldk, const void* v_dev, int ldv,
                   const int32_t* kv_slot_dev, int T, void* stream);

/*
 * The values held in T slots, as bf16 (rounded from the fp32 product n s g): k_out and v_out
 * [T, kv_heads * head_dim] dense, 16-byte aligned.  Zeros for slot -1, and for slots outside the
 * cache, which are flagged.  Errors: LORA_EINVAL, LORA_ECUDA.
 */
int lora_kv_read(lora_kv_cache_t* cache, const int32_t* kv_slot_dev, int T, void* k_out,
                 void* v_out, void* stream);

/*
 * o = softmax(scale q K^T) V for T query rows over the cached keys and values of their
 * requests (the new tokens' own must have been appended before).
 *   q_dev, out_dev  rows of q_heads * head_dim bf16, ldq and ldo elements apart (multiples
 *                   of 8; pointers 16-byte aligned); they must not overlap.  q_heads is a
 *                   multiple of kv_heads: query head i reads cache head i / (q_heads / kv_heads).
 *   q_offsets [B+1], kv_len [B], block_table [B, max_blocks]: as from lora_kv_maps.
 *   max_q           an upper bound of a request's new tokens (q_offsets[b+1] - q_offsets[b]);
 *                   a request above it is flagged and its rows are unspecified.
 * With q rows and n cached tokens, row i of a request sees positions 0 .. n - q + i.  A row
 * that sees nothing is zero, and so are rows outside every request.  Scores, the softmax's
 * maximum and sum and the output's accumulation are fp32; the products run on the tensor
 * cores from q as it is (bf16, or scaled by a power of two into fp16, exactly from 2^-19 of a
 * row's largest element on), the cache's exact values, and probabilities as fp16.  Scores have to
 * stay below 2^24 in size: beyond, fp32 holds none of their fractions, and rows may be NaN.
 * Offsets that are not ascending within [0, T], lengths outside [0, max_blocks * page_size]
 * and page ids outside the cache are flagged (lora_kv_get_status) and read nothing outside
 * the cache; the results of such requests are unspecified.
 * One call at a time per cache: calls share its workspace, so calls on several streams must
 * be ordered by the caller.
 * Limits: 1 <= B <= max_requests, 0 <= T <= 1 << 20, q_heads / kv_heads <= 64; scale finite, and
 * |scale| k_scale at most 7e36 (from about 7.3e36 on it is refused).
 * Errors: LORA_EINVAL, LORA_ECUDA.
 */
int lora_kv_attend(lora_kv_cache_t* cache, const void* q_dev, int ldq, int q_heads,
                   const int32_t* q_offsets, const int32_t* kv_len, const int32_t* block_table,
                   int max_blocks, int B, int T, int max_q, float scale, void* out_dev, int ldo,
                   void* stream);

/*
 * Synchronise `stream`, read and clear the cache's device error flags: LORA_OK, LORA_EID (a
 * slot, page id, length or offset out of range), LORA_ETIMEOUT (a wait inside a kernel gave
 * up; the results of calls since then are invalid) or LORA_ECUDA.  After LORA_ETIMEOUT the
 * attention's workspace is as new: the calls that follow on `stream` are sound.
 */
int lora_kv_get_status(lora_kv_cache_t* cache, void* stream);

/*
 * Self-test of a wait that gives up: enqueues a kernel whose wait nothing completes (it gives up
 * after 2 s) and which leaves the cache as an attention call leaves it whose wait ran out.
 * lora_kv_get_status then returns LORA_ETIMEOUT, the expected result, and the cache is usable again.
 * Errors: LORA_EINVAL, LORA_ECUDA.
 */
int lora_kv_wait_selftest(lora_kv_cache_t* cache, void* stream);

/* Bytes of the cache's pages (not of its workspace).  0 for NULL. */
int64_t lora_kv_cache_bytes(const lora_kv_cache_t* cache);

/* Text of the last error raised on this cache ("" if none).  Owned by the cache. */
const char* lora_kv_last_error(const lora_kv_cache_t* cache);

/* Synchronise the cache's device, then free everything it owns.  NULL is a no-op. */
void lora_kv_cache_destroy(lora_kv_cache_t* cache);

#ifdef __cplusplus
}
#endif

#endif /* LORA_KV_H */
