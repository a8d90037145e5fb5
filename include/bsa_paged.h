/*
 * bsa_paged.h -- C ABI of libbsa, second part: rotary positions with several
 * axes, a paged key/value cache, and attention of new tokens over it.
 *
 * These calls stand around the ones of bsa.h.  bsap_rope_axes turns Q and K
 * before bsa_select / bsa_forward (and bsap_rope_axes with `backward` turns
 * the gradients bsa_backward returns); bsap_cache_append keeps the keys and
 * values of the understanding stream, or of any token stream, in pages;
 * bsap_forward is the form of bsa_forward_causal for tokens that come later:
 * one new token per request, a few, or a chunk, over the pages, with a prefix
 * that every request of the batch shares.
 *
 * The conventions of bsa.h hold: device memory is the caller's, nothing is
 * allocated, no call synchronises, all work is enqueued on the caller's
 * stream, arguments are checked on the host before anything is launched, the
 * message of a refusal comes from bsa_get_last_error(), and every call can be
 * captured in a CUDA graph.  Head dim 64 or 128, bf16.  Sizes of zero are
 * refused, as in bsa.h.  The symbols carry the prefix bsap_.
 *
 * Lengths and tables that change from step to step (kv_lens, new_lens, the
 * page tables, positions, frequencies) are DEVICE arrays that the kernels read
 * when they run, so that a captured step follows them; they may not change while
 * a call runs.  The host cannot check their values.  The kernels do: they never
 * read or write outside the given buffers, and a table entry that names no
 * page, or a length that the table has no pages for, sets an error word that the
 * next bsa_device_status() returns as BSA_ERR_INVALID_INDICES (results of the
 * requests concerned are then unspecified, as are all after BSA_ERR_TIMEOUT).
 */
#ifndef BSA_PAGED_H_
#define BSA_PAGED_H_

#include "bsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------- rotation ---
 * For Q and K that bsa_select reads next and whose positions are a table of fp32
 * sines and cosines per row, halves paired, bsa_select_rope rotates in the
 * selector's pooling pass (one reading of Q and K less); positions with axes,
 * neighbours paired, part of the channels, positions per request, far positions,
 * the gradient, and keys on their way into pages are here.
 *
 * Pair p of `pairs` (a multiple of 8, at most D / 2) is the channels
 * (p, p + pairs), or with interleaved != 0 (2p, 2p + 1).  Its angle at a token
 * is position[axes[p]] * inv_freq[p], and
 *     y_lo = x_lo cos - x_hi sin,    y_hi = x_hi cos + x_lo sin.
 * Channels from 2 * pairs on, and pairs whose axis is outside [0, n_axes),
 * are passed through bit for bit.  Angles are formed in 64-bit fixed point
 * (turns modulo one), so that they are as exact at position 2^30 as at position
 * 1; products are fp32, rounded to bf16 once.
 * inv_freq: device double [pairs], finite, |inv_freq| < 2^10 (radians per
 *   position).  axes: device int32 [pairs].  n_axes: 1 to 4. */
typedef struct bsap_rope {
  const double* inv_freq;
  const int32_t* axes;
  int32_t pairs, n_axes, interleaved;
} bsap_rope;

/* int32 positions [B, S, n_axes] in device memory; strides in elements, a
 * stride of 0 shares positions along that axis. */
typedef struct bsap_positions {
  const int32_t* ptr;
  int64_t stride_b, stride_s, stride_a;
} bsap_positions;

/* Rotates q, and k too unless it is NULL, in one launch.
 * q [B, S, Hq, D], k [B2, S2, Hk, D]: inputs as bsa_tensor; here a stride may
 *   be 0 (a broadcast input), and strides of axes of length 1 are not looked at.
 * q_out, k_out: bf16 contiguous, 16-byte aligned, of the input's shape; may be
 *   the input's own storage when the input is contiguous, and may otherwise
 *   not overlap any input.
 * backward != 0: the transposed rotation, which takes the gradients of q_out
 *   and k_out to those of q and k. */
BSA_API bsa_status bsap_rope_axes(const bsa_tensor* q, const bsa_tensor* k, const bsap_positions* pos_q,
                                  const bsap_positions* pos_k, const bsap_rope* rope, int32_t backward,
                                  void* q_out, void* k_out, bsa_stream_t stream);

/* ---------------------------------------------------------- paged cache ---
 * k_cache, v_cache: bsa_tensor with B = number of pages, S = page size (16,
 *   32, 64, 128 or 256 slots), H = Hkv, D; same shape, any strides that keep
 *   rows 16-byte aligned and slots apart.
 * page_table: device int32, request b's pages at page_table[b * table_stride
 *   + 0 .. max_pages).  Key j of request b lies in page table[b][j / S], slot
 *   j % S.  Entries behind a request's length are not read.
 * kv_lens: device int32 [B], keys of request b INCLUDING the call's new tokens.
 * new_lens: device int32 [B], the request's real new tokens, or NULL = all T;
 *   clamped to [0, T].
 *
 * Append: token t < new_lens[b] of k and v [B, T, Hkv, D] is written to key
 *   position kv_lens[b] - new_lens[b] + t of request b; a token whose position
 *   is negative or behind the table, or whose page does not exist, is dropped
 *   and reported.  Nothing else of the cache changes.  With `rope`, k is
 *   rotated on the way at pos [B, T, n_axes], and so are the queries q [B, T,
 *   Hq, D] into q_out (contiguous, all T rows, also behind new_lens; in place
 *   when q is contiguous); q may be NULL, and rope NULL copies k (q must then
 *   be NULL).  Two tokens with the same page and slot are the caller's
 *   mistake: which of them stays, K and V each, is unspecified.  k, v, q and
 *   q_out may not lie between a cache's first and last byte, q_out not overlap
 *   k or v, and k_cache and v_cache not share slots (refused where they are the
 *   same pointer). */
BSA_API bsa_status bsap_cache_append(const bsa_tensor* k, const bsa_tensor* v, const bsa_tensor* k_cache,
                                     const bsa_tensor* v_cache, const int32_t* page_table, int64_t table_stride,
                                     int32_t max_pages, const int32_t* kv_lens, const int32_t* new_lens,
                                     const bsap_rope* rope, const bsap_positions* pos, const bsa_tensor* q,
                                     void* q_out, bsa_stream_t stream);

/* ------------------------------------------------------------ attention ---
 * Workspace bytes of bsap_forward for B requests of T new tokens on a device
 * with num_sms SMs (0: the current device): partial sums of the key ranges
 * that the thread blocks split the keys into.  0 for sizes that bsap_forward refuses. */
BSA_API size_t bsap_forward_workspace_size(int B, int T, int Hq, int Hkv, int d, int has_prefix, int num_sms);

/* Row i < n = new_lens[b] of request b (q [B, T, Hq, D]) attends, with query
 * head h reading KV head h / (Hq / Hkv),
 *   - the prefix_len first keys of the pages prefix_table[0 .. ceil(prefix_len
 *     / S)), the same for every request (see below on how often they are read),
 *     and
 *   - its request's own keys j < kv_lens[b]; with causal != 0 only
 *     j <= kv_lens[b] - n + i.
 * out_i = sum_j softmax(z)_j v_j (bf16), z_j = softmax_scale q_i . k_j;
 * lse_i = ln sum_j exp(z_j).  Rows i >= n and rows without a key: out 0, lse
 * -inf.  A row with a score of NaN or +infinity (of a Q that is not finite, or a
 * product past the range of fp32), or with scores of -infinity alone, has NaN as
 * its output; other rows do not feel it.  Slots behind a request's keys are never
 * read into a result, whatever they hold; real keys and their values have to be
 * finite.
 * out: bf16 [B, T, Hq, D] contiguous; lse: fp32 [B, Hq, T] contiguous or NULL.
 * out, lse and workspace share no memory with one another nor with anything that
 * the call reads (refused from the first to behind the last byte of each).
 * softmax_scale <= 0 selects D^-1/2.  prefix_len 0: prefix_table may be NULL.
 * max_pages 0: no own keys (page_table and kv_lens may be NULL).
 * Results do not depend on scheduling (no atomics), but the split of the keys
 * depends on the lengths of the whole batch and on the number of SMs.
 * Scores, weights' sums, maxima and partial results are fp32; the weights are
 * rounded to bf16 (off by at most 2^-8 of each) where they meet V on the tensor
 * cores, as in bsa_forward.
 * The prefix is read once for every 256 rows (b, i, g) of the batch under a KV
 * head, padded rows counted: once for up to 256 / (Hq / Hkv) single tokens.
 * Where T tokens fill tiles of 128 rows by themselves, it is read with each
 * request's own keys instead.  Both go by T, whatever new_lens says: the padded
 * rows of a batch in which one request has many new tokens and the others one
 * cost what real ones do, and two calls, one for each kind, take a fraction of
 * the time (a chunk of 500 tokens beside 63 single tokens on a prefix of 8,192
 * keys, 32/8 heads of 128: 551 us in one call, 76 + 47 in two).
 * Sizes above 2^28 key tiles, B Hkv ceil(T Hq / Hkv / 256) ceil(keys / 128) with
 * the keys that the tables could hold, are refused, and from 2.7 10^7 on prefix
 * tiles and others weigh the same in the division of work (up to a third slower,
 * or half where the prefix is a tile or two): pass a view of the table's first
 * columns where it is much wider than the requests are long.
 * B <= 4096, Hq <= 256.  workspace: device, 256-byte aligned; every byte that
 * counts was written by the same call, so calls that follow one another on a
 * stream, captured or not, may share one; calls that overlap may not. */
BSA_API bsa_status bsap_forward(const bsa_tensor* q, const bsa_tensor* k_cache, const bsa_tensor* v_cache,
                                const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                const int32_t* kv_lens, const int32_t* new_lens, const int32_t* prefix_table,
                                int32_t prefix_len, int32_t causal, float softmax_scale, void* out, float* lse,
                                void* workspace, size_t ws_bytes, bsa_stream_t stream);

/* bsa_debug_wait_probe for the paged attention: the bounded wait of one thread
 * gives up after limit_ns (1 ms to 10 s) and the next bsa_device_status() returns
 * BSA_ERR_TIMEOUT.  No fault, trap or hang is involved. */
BSA_API bsa_status bsap_debug_wait_probe(uint64_t limit_ns, bsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BSA_PAGED_H_ */
