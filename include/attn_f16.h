/*
 * attn_f16 — scaled dot-product attention forward, head dimension 256, for
 * GB300 (sm_103a), and the calls of a serving step over a paged key/value
 * cache (second half of this file).  C ABI, plain pointers and sizes.
 *
 * What it computes, per batch b, head h and query row i:
 *
 *     O[b,h,i,:] = sum_j softmax_j(scale * Q[b,h,i,:] . K[b,h,j,:]) * V[b,h,j,:]
 *
 * with binary16 Q, K, V, O, FP32 scores, softmax statistics and
 * accumulation, softmax weights rounded to binary16 for the product with V
 * (the sum is of the FP32 weights; one below 2^-25 of the row's largest may be 0
 * in the product), and O rounded to binary16 (round to nearest even).  This is
 * the flash-attention ("SDP") kernel of the "Xe2 Nbarrier Pipelining" page,
 * section "Proven Pattern: SDP Kernel Split Barrier B" (head dimension 256):
 * per block of 64 keys, S = Q K^T, a softmax with a running row maximum,
 * P written to shared memory, then — across the split barrier — the sum
 * update and the next copies while the P V product waits for P.  The page
 * states no mask, so none is applied (every query attends to every key).
 *
 * Uses a gemm_f16 plan (include/gemm_f16.h) for its device, status word
 * and the options GEMM_F16_OPT_TIMEOUT_NS and GEMM_F16_OPT_FAULT_UNIT (here:
 * for the single-CTA kernel the linear index x + gx*(y + gy*z) of the CTA
 * whose first key tile gets no copy, for the CTA-pair kernel the work unit
 * (item * ranges + range) whose first key tile gets no copy from the
 * leader; for the timeout test).  Errors found on the device are reported
 * later by gemm_f16_status.
 */
#ifndef ATTN_F16_H
#define ATTN_F16_H

#include <stdint.h>

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Head dimension the kernel supports. */
#define ATTN_F16_HEAD_DIM 256

/*
 * Enqueue the attention forward pass on `stream` (asynchronous).
 *   batch, heads      >= 1 and <= 65535 each.
 *   seq_q, seq_kv     >= 1 (query rows, key/value rows per head).
 *   head_dim          must be ATTN_F16_HEAD_DIM (256).
 *   Q, K, V, O        device pointers to binary16, 16-byte aligned; element
 *                     (b, h, i, d) of X is at X[b*xs[0] + h*xs[1] + i*xs[2] + d]
 *                     (d contiguous).  The strides xs[0..2] are in elements,
 *                     positive multiples of 8, with xs[2] >= 256; a stride
 *                     of a dimension of extent 1 is not used.  So both
 *                     [batch, head, seq, 256] and [batch, seq, head, 256]
 *                     storage work.  O is written (every row of every head)
 *                     and must not overlap Q, K or V.
 *   scale             finite; usually 1/sqrt(256) = 0.0625.
 * Returns GEMM_F16_OK, GEMM_F16_ERR_INVALID_ARG (sizes, strides, scale,
 * null pointers), GEMM_F16_ERR_MISALIGNED (pointer or stride alignment) or
 * GEMM_F16_ERR_CUDA (encode or launch failure) or GEMM_F16_ERR_OOM;
 * nothing is enqueued on an error.  Without a key split the call allocates
 * nothing; with one (GEMM_F16_OPT_ATTN_SPLIT, automatic when the
 * (batch, head, 256-row) items are too few to fill the GPU) the CTA-pair
 * kernel writes each key range's normalised FP32 partial of O (256 KB per
 * 256 rows and range) and its row offsets and sums into the plan's
 * workspace, which grows on the stream as needed (as for split GEMM runs),
 * and a second kernel merges the ranges into O.
 */
int attn_f16_fwd(gemm_f16_plan_t plan, int batch, int heads, int seq_q, int seq_kv,
                 int head_dim, const void *Q, const int64_t q_strides[3],
                 const void *K, const int64_t k_strides[3], const void *V,
                 const int64_t v_strides[3], void *O, const int64_t o_strides[3],
                 float scale, gemm_f16_stream_t stream);

/*
 * The same forward pass with HOST operands: hQ [batch, heads, seq_q, 256],
 * hK and hV [batch, heads, seq_kv, 256], hO [batch, heads, seq_q, 256], all
 * contiguous binary16 in host memory (pinned memory gives asynchronous
 * copies).  Q, K, V are copied into one of two plan-owned sets of device
 * buffers on a plan-internal stream, the pass runs on `stream` once they
 * have arrived, and O is copied back on `stream`; consecutive calls
 * alternate the two sets, so one call's input copies overlap the previous
 * call's pass and output copy.  hQ, hK, hV must therefore be ready when the
 * call is made; synchronise `stream` before reading hO or reusing the
 * inputs.  A set grows (after a device synchronisation) when a call needs
 * more room than it has.  Calls on different streams must be ordered by
 * the caller, as for every use of a plan (one pass at a time); the plan
 * orders its own input copies after the output copy of the call that last
 * used the same set, whatever stream that call ran on.  Returns the codes
 * of attn_f16_fwd (the sizes and scale are checked as there; null host
 * pointers give GEMM_F16_ERR_INVALID_ARG).
 */
int attn_f16_fwd_host(gemm_f16_plan_t plan, int batch, int heads, int seq_q, int seq_kv,
                      int head_dim, const void *hQ, const void *hK, const void *hV, void *hO,
                      float scale, gemm_f16_stream_t stream);

/*
 * The number of key ranges attn_f16_fwd would cut each item's keys into for
 * these sizes with this plan's current options (1: no split, one kernel
 * launch; n > 1: the CTA-pair kernel plus the merging kernel).  Enqueues
 * nothing.  Returns GEMM_F16_OK or GEMM_F16_ERR_INVALID_ARG (null pointers,
 * sizes < 1).
 */
int attn_f16_key_ranges(gemm_f16_plan_t plan, int batch, int heads, int seq_q, int seq_kv,
                        int *ranges);

/* Host-only argument check used by attn_f16_fwd (no device needed). */
int attn_f16_validate(int batch, int heads, int seq_q, int seq_kv, int head_dim,
                      const void *Q, const int64_t q_strides[3], const void *K,
                      const int64_t k_strides[3], const void *V,
                      const int64_t v_strides[3], const void *O,
                      const int64_t o_strides[3], float scale);

/*
 * ---------------------------------------------------------------------------
 * Serving from a paged cache
 * ---------------------------------------------------------------------------
 * Keys and values live in caches of `num_pages` pages of `page_size` rows
 * (a row: one token's kv_heads heads of 256 binary16 numbers).  Element
 * (page, row, head, d) of a cache is at X[page*xs[0] + row*xs[1] +
 * head*xs[2] + d], strides in elements: [page][row][head][256] and
 * [page][head][row][256] storage both work.  A request's token at position
 * p is in row p % page_size of the page block_table[b*table_stride +
 * p / page_size]; its slot is page * page_size + row.  All maps are 32-bit
 * integers in device memory, so that a step's lengths need not be known on
 * the host.  A step has, per request, `cached` tokens in the cache already
 * and `added` new ones; the new tokens of all requests follow one another in
 * the step's token buffers, request b's from starts[b] to starts[b+1] - 1.
 *
 * Lengths, pages and slots read on the device are checked there: one out of
 * range is never followed, GEMM_F16_ERR_BAD_INDEX is reported through
 * gemm_f16_status, and what the call writes for that request or token is
 * described with each call.  Other requests are not affected.
 *
 * Every call below is asynchronous on `stream` and can be captured into a
 * CUDA graph, as the plan's first call too (the plan must outlive the graph's
 * replays).  The first attn_f16_paged_fwd of a plan allocates its workspace:
 * partial sums of tiles of queries that are cut between workers, about 40 MB
 * on a GB300 whatever the step.  The maps and
 * the rotation are one kernel launch each, the attention two (its kernel and
 * the merge of cut tiles) or, where some requests may have many new tokens and
 * others few, four.  GEMM_F16_OPT_SM_LIMIT bounds the attention's kernels,
 * GEMM_F16_OPT_KERNEL_TIMING times them (not the merges),
 * GEMM_F16_OPT_FAULT_UNIT names the CTA or CTA pair whose first key copy is
 * left out; results do not depend on the number of SMs beyond rounding.
 */

/*
 * The maps of one step.  For each request b, in order, the pages that its
 * new tokens need beyond those that hold its cached ones,
 *     ceil((cached+added) / page_size) - ceil(cached / page_size),
 * are taken from free_pages[*free_head ..] and written into its row of
 * block_table (entries of pages it already has are read, never written);
 * then
 *     starts[0 .. batch]        running sums of `added`, starts[0] = 0
 *     kv_lens[b]                cached + added
 *     positions[t], slots[t]    of new token t, for t < starts[batch];
 *                               0 and -1 for starts[batch] <= t < max_tokens
 *     *free_head_out            *free_head + the pages taken
 *   batch        1 .. 65535; max_tokens >= 0 (the room in positions and
 *                slots, which may be NULL when 0); page_size 1 .. 2^20.
 *   block_table  batch rows of max_pages entries (1 .. 2^24), table_stride
 *                >= max_pages apart.
 *   free_pages   num_free >= 0 page numbers (may be NULL when 0).  free_head
 *                and free_head_out are single integers on the device; taking
 *                the call again with the same free_head gives the same maps.
 *   No buffer that the call writes (starts, kv_lens, positions, slots,
 *   free_head_out, the rows of block_table) may overlap another one of the
 *   call: the lengths are read while the maps are written, so a step cannot
 *   advance them in place (kv_lens is not `cached`, free_head_out not
 *   free_head).  Overlaps are refused.
 * Out of range on the device, each reported: a negative length counts as 0;
 * cached and added tokens past max_pages * page_size are cut off (the
 * request then has fewer new tokens); a page that the free list does not
 * hold any more is -1 in block_table, and its tokens' slots are -1; new
 * tokens past max_tokens are cut off, those of the last requests first.
 * Returns GEMM_F16_OK, GEMM_F16_ERR_INVALID_ARG, GEMM_F16_ERR_MISALIGNED
 * (a pointer that is no multiple of 4 bytes) or GEMM_F16_ERR_CUDA.
 */
int attn_f16_paged_maps(gemm_f16_plan_t plan, int batch, const int32_t *cached,
                        const int32_t *added, int32_t *block_table, int64_t table_stride,
                        int max_pages, const int32_t *free_pages, int num_free,
                        const int32_t *free_head, int page_size, int max_tokens,
                        int32_t *starts, int32_t *kv_lens, int32_t *positions,
                        int32_t *slots, int32_t *free_head_out, gemm_f16_stream_t stream);

/* Pairings of attn_f16_rope: pair i is (x[i], x[i + rot_dim/2]) or
 * (x[2i], x[2i+1]). */
enum {
    ATTN_F16_ROPE_HALF = 0,
    ATTN_F16_ROPE_INTERLEAVED = 1
};

/*
 * Rotary positions: the first rot_dim numbers of every head are rotated in
 * pairs; the others are copied.  Pair i of a token at position p turns by
 * the angle p * w_i (w_i: the pair's frequency):
 *     y0 = factor * (x0 cos - x1 sin),   y1 = factor * (x1 cos + x0 sin)
 * (`inverse`: by -p * w_i, which is the gradient's rotation: the gradient
 * with respect to x is the inverse rotation, with the same factor, of the
 * one with respect to y).  Computed in FP32, rounded once to binary16.
 *   turns      rot_dim/2 frequencies on the device, each as 2^64 times the
 *              part of a full turn per position (attn_f16_rope_turns): the
 *              product with the position modulo 2^64 is the angle, exact to
 *              2^-20 of a turn at any 32-bit position (to the 53 bits of the
 *              frequency: 2^-32 at a position of a million).
 *   positions  `tokens` device integers.
 *   Q, Qo      q_heads heads of 256 numbers per token; element (t, h, d) at
 *              X[t*xs[0] + h*xs[1] + d].  Qo may be Q (same strides) or must
 *              not overlap it.
 *   K, V       kv_heads heads per token, laid out like Q.  K is rotated into
 *              and V copied into row slots[t] of the caches Kc and Vc (whose
 *              pages and strides are described above; neither may overlap
 *              K, V or Q).  A token with slot -1 writes nothing; one with
 *              any other slot outside [0, num_pages * page_size) neither,
 *              and is reported.  Two tokens must not have the same slot.
 *              With kv_heads = 0 only Q is rotated and these arguments are
 *              not used; with q_heads = 0 only K and V are written.
 *   tokens >= 0; q_heads, kv_heads in 0 .. 65535, not both 0; head_dim 256;
 *   rot_dim a multiple of 16 in 16 .. 256; layout as above; factor finite;
 *   page_size, num_pages >= 1.  Strides are positive multiples of 8 and at
 *   least 256 (of a dimension of extent 1: not used); 16-byte aligned
 *   pointers, 4-byte for the integers, 8-byte for turns.
 * Returns GEMM_F16_OK, GEMM_F16_ERR_INVALID_ARG, GEMM_F16_ERR_MISALIGNED or
 * GEMM_F16_ERR_CUDA.
 */
int attn_f16_rope(gemm_f16_plan_t plan, int tokens, int q_heads, int kv_heads, int head_dim,
                  int rot_dim, int layout, int inverse, float factor, const uint64_t *turns,
                  const int32_t *positions, const void *Q, const int64_t q_strides[2], void *Qo,
                  const int64_t qo_strides[2], const void *K, const int64_t k_strides[2],
                  const void *V, const int64_t v_strides[2], const int32_t *slots, void *Kc,
                  const int64_t kc_strides[3], void *Vc, const int64_t vc_strides[3],
                  int num_pages, int page_size, gemm_f16_stream_t stream);

/*
 * Host-only: n frequencies in radians per position -> turns[n] (host
 * memory).  Each must be finite, 0 <= w < 2 pi.  Returns GEMM_F16_OK or
 * GEMM_F16_ERR_INVALID_ARG.
 */
int attn_f16_rope_turns(const double *radians, int n, uint64_t *turns);

/*
 * Attention of a step's new tokens over their requests' paged keys and
 * values (which hold the new tokens' own: call attn_f16_rope first).  The
 * i-th of the n = starts[b+1] - starts[b] new tokens of request b stands at
 * position p = kv_lens[b] - n + i and sees the keys j <= p of its request;
 * with window > 0 only those with j > p - window or j < sinks.  Query head h
 * reads key/value head h / (q_heads / kv_heads):
 *     O[t,h,:] = sum_j softmax_j(scale * Q[t,h,:] . K[j,:]) * V[j,:]
 * FP32 scores, softmax statistics and accumulation, O rounded to binary16.  The
 * softmax weights are rounded to binary16 for the product with V (not for their
 * sum): each is off by at most 2^-11 of itself, or 2^-32 of the row's largest.
 * A row that sees no key (kv_lens[b] < n), or only keys whose scores are -inf,
 * is 0, and so are the rows from starts[batch] to total_q - 1; rows before
 * starts[0] are not written.  Rows of a page that no position of the request
 * has reached, pages past it, and pages that no query of it sees may hold
 * anything (NaN included) and their table entries are not used.  On a page
 * that some query of the request sees, an infinity or NaN in a V row at a
 * position that the request has reached may reach all of the request's rows,
 * whether they see that key or not (a weight of 0 times infinity).
 *   batch        1 .. 65535.   total_q >= 0: rows of Q and O (0: nothing is
 *                enqueued).   max_q >= 0: the largest n, or more.
 *   q_heads      a multiple of kv_heads, at most 64 times as many;
 *                kv_heads 1 .. 1024; head_dim 256.
 *   Q, O         element (t, h, d) at X[t*xs[0] + h*xs[1] + d].  O must not
 *                overlap Q or the caches.
 *   page_size    a multiple of 8, 8 .. 32768.   num_pages >= 1.
 *   window, sinks >= 0 (window 0: no window, sinks unused).   scale finite.
 * Strides and alignment as for attn_f16_rope.
 * Out of range on the device: starts that decrease or pass total_q, more
 * than max_q new tokens, and lengths past max_pages * page_size are clamped;
 * a page outside [0, num_pages) reads as zeros; each is reported and leaves
 * that request's rows unspecified.
 * Returns the codes of attn_f16_fwd.
 */
int attn_f16_paged_fwd(gemm_f16_plan_t plan, int batch, int total_q, int max_q, int q_heads,
                       int kv_heads, int head_dim, const void *Q, const int64_t q_strides[2],
                       const void *Kc, const int64_t kc_strides[3], const void *Vc,
                       const int64_t vc_strides[3], int num_pages, int page_size,
                       const int32_t *block_table, int64_t table_stride, int max_pages,
                       const int32_t *starts, const int32_t *kv_lens, void *O,
                       const int64_t o_strides[2], float scale, int window, int sinks,
                       gemm_f16_stream_t stream);

/* Host-only argument checks of the three calls (no device needed). */
int attn_f16_paged_maps_validate(int batch, const int32_t *cached, const int32_t *added,
                                 const int32_t *block_table, int64_t table_stride, int max_pages,
                                 const int32_t *free_pages, int num_free,
                                 const int32_t *free_head, int page_size, int max_tokens,
                                 const int32_t *starts, const int32_t *kv_lens,
                                 const int32_t *positions, const int32_t *slots,
                                 const int32_t *free_head_out);
/* Whether buffers of a maps call (arguments that passed the check above)
 * overlap where they must not: GEMM_F16_OK or GEMM_F16_ERR_INVALID_ARG. */
int attn_f16_paged_maps_overlap(int batch, const int32_t *cached, const int32_t *added,
                                const int32_t *block_table, int64_t table_stride, int max_pages,
                                const int32_t *free_pages, int num_free,
                                const int32_t *free_head, int max_tokens, const int32_t *starts,
                                const int32_t *kv_lens, const int32_t *positions,
                                const int32_t *slots, const int32_t *free_head_out);
int attn_f16_rope_validate(int tokens, int q_heads, int kv_heads, int head_dim, int rot_dim,
                           int layout, float factor, const uint64_t *turns,
                           const int32_t *positions, const void *Q, const int64_t q_strides[2],
                           const void *Qo, const int64_t qo_strides[2], const void *K,
                           const int64_t k_strides[2], const void *V, const int64_t v_strides[2],
                           const int32_t *slots, const void *Kc, const int64_t kc_strides[3],
                           const void *Vc, const int64_t vc_strides[3], int num_pages,
                           int page_size);
int attn_f16_paged_validate(int batch, int total_q, int max_q, int q_heads, int kv_heads,
                            int head_dim, const void *Q, const int64_t q_strides[2],
                            const void *Kc, const int64_t kc_strides[3], const void *Vc,
                            const int64_t vc_strides[3], int num_pages, int page_size,
                            const int32_t *block_table, int64_t table_stride, int max_pages,
                            const int32_t *starts, const int32_t *kv_lens, const void *O,
                            const int64_t o_strides[2], float scale, int window, int sinks);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_F16_H */
