/*
 * bsa_quant.h -- C ABI of libbsa, third part: the paged key/value cache of
 * bsa_paged.h held in 4 bits.
 *
 * bsaq_cache_append quantises new keys and values as it writes them into pages,
 * bsaq_cache_read turns pages back into bf16 rows (for bsa_select, bsa_forward
 * and their kin, which take rows), and bsaq_forward is bsap_forward over such
 * pages: it reads 17/64 of the bytes.
 *
 * The conventions of bsa.h and bsa_paged.h hold: device memory is the caller's,
 * nothing is allocated, no call synchronises, all work is enqueued on the
 * caller's stream, arguments are checked on the host before anything is launched,
 * the message of a refusal comes from bsa_get_last_error(), and every call can be
 * captured in a CUDA graph.  Head dim 64 or 128, bf16.  Sizes of zero are refused.
 * Lengths and tables are DEVICE arrays that the kernels read when they run; what
 * bsa_paged.h says of bad values holds here, too.  The symbols carry the prefix
 * bsaq_.
 *
 * The format.  Of each token and head, 32 neighbouring channels (a group) share a
 * scale.  It is held in a byte b: s = (1 + (b mod 8) / 8) 2^(floor(b / 8) - 15)
 * for b = 0 .. 254; b = 255 marks a group in which some value was not finite, and
 * all of it reads as NaN.  Each value x is held as a code c = -7 .. 7:
 *     a = max |x| of the group;
 *     s = a / 7 rounded to four significant bits (ties to even), at least 2^-15
 *         and at most 1.75 2^16 (values of more than 7 times that saturate); a = 0 has b = 0;
 *     c = sign(x) min(floor(|x| / s + 1/2), 7).
 * The value held is c s: at most seven significant bits, so that it is exact in
 * bf16.  It is off by at most s / 2, which is at most the larger of a / 13 and
 * 2^-16 (but for values that saturate).  All of this is exact arithmetic: the same
 * input always gives the same bytes.
 *
 * A page of S slots (16, 32, 64, 128 or 256) holds for each head S / 16 blocks
 * of 16 slots, 17 D / 2 bytes each:
 *     K: codes [D / 32 groups][16 slots][16 bytes], then scales [D / 32][16 slots];
 *     V: codes [D channels][8 bytes = 16 slots],    then scales [D / 32][16 slots].
 * Codes are held as c + 8 in four bits; of eight that follow one another (channels
 * of K, slots of V) in a little-endian 32-bit word, number e is in bits 4 n .. 4 n
 * + 3 with n = e / 2 + 4 (e mod 2).
 */
#ifndef BSA_QUANT_H_
#define BSA_QUANT_H_

#include "bsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache: bytes [pages, heads, blocks, 17 D / 2], blocks = S / 16 of a page; the
 * blocks of a page and head follow one another, page and head strides (in bytes)
 * are multiples of 16 that keep them apart (strides of axes of length 1 are not
 * looked at).  ptr: 16-byte aligned.  K and V have the same shape. */
typedef struct bsaq_cache {
  void* ptr;
  int64_t pages, heads, blocks, D;
  int64_t stride_page, stride_head;
} bsaq_cache;

/* page_table, table_stride, max_pages, kv_lens, new_lens: as in bsap_cache_append
 * (bsa_paged.h).
 *
 * Append: token t < new_lens[b] of k and v [B, T, Hkv, D] is quantised into key
 *   position kv_lens[b] - new_lens[b] + t of request b; a token whose position is
 *   negative or behind the table, or whose page does not exist, is dropped and
 *   reported.  What other slots hold is kept.  K is written as it is given: keys
 *   with rotary positions are rotated before (bsap_rope_axes).  The bytes of V of
 *   neighbouring slots are shared, so a block of 16 slots that one request's new
 *   tokens touch may not be touched by another's in the same call (requests that
 *   grow have a last page of their own).  k and v may not lie between a cache's
 *   first and last byte, and k_cache and v_cache not share bytes (refused where
 *   they are the same pointer). */
BSA_API bsa_status bsaq_cache_append(const bsa_tensor* k, const bsa_tensor* v, const bsaq_cache* k_cache,
                                     const bsaq_cache* v_cache, const int32_t* page_table, int64_t table_stride,
                                     int32_t max_pages, const int32_t* kv_lens, const int32_t* new_lens,
                                     bsa_stream_t stream);

/* Read: row t of request b of k_out and v_out (bf16 [B, S, Hkv, D], any strides of
 *   multiples of 8 elements that keep rows apart) is what the pages hold of key
 *   first[b] + t, for keys below kv_lens[b]; rows behind, and rows from S on, are
 *   not written.  first: device int32 [B], or NULL = 0; taken as 0 where negative.
 *   A negative length is reported, as a missing page of a row that is asked for is.
 *   The outputs share no memory with the caches, the table, the lengths, first or one
 *   another (refused from the first to behind the last byte of each). */
BSA_API bsa_status bsaq_cache_read(const bsaq_cache* k_cache, const bsaq_cache* v_cache, const int32_t* page_table,
                                   int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                                   const int32_t* first, const bsa_tensor* k_out, const bsa_tensor* v_out,
                                   bsa_stream_t stream);

/* Workspace bytes of bsaq_forward for B requests of T new tokens on a device with
 * num_sms SMs (0: the current device).  0 for sizes that bsaq_forward refuses. */
BSA_API size_t bsaq_forward_workspace_size(int B, int T, int Hq, int Hkv, int d, int has_prefix, int num_sms);

/* bsap_forward (bsa_paged.h) over 4-bit pages: the same rows, keys, limits,
 * prefix, results and refusals, with k_j and v_j the values that the pages hold.
 * Codes times scales are exact in bf16; scores, weights' sums, maxima and partial
 * results are fp32, and the weights are rounded to bf16 (off by at most 2^-8 of
 * each) where they meet V on the tensor cores.  Real keys and their values have
 * to be finite; slots behind a request's keys are never read into a result,
 * whatever they hold. */
BSA_API bsa_status bsaq_forward(const bsa_tensor* q, const bsaq_cache* k_cache, const bsaq_cache* v_cache,
                                const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                const int32_t* kv_lens, const int32_t* new_lens, const int32_t* prefix_table,
                                int32_t prefix_len, int32_t causal, float softmax_scale, void* out, float* lse,
                                void* workspace, size_t ws_bytes, bsa_stream_t stream);

/* bsap_debug_wait_probe for the attention over 4-bit pages (1 ms to 10 s). */
BSA_API bsa_status bsaq_debug_wait_probe(uint64_t limit_ns, bsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BSA_QUANT_H_ */
