/*
 * bsa_cache.h -- C ABI of attention over packed sequences and paged caches (libbsa.so; the
 * block-sparse attention is in bsa.h, the operators around it in bsa_block.h).
 *
 *   bsa_cache_write      -- keys and values of new tokens into the pages of a cache, as they are
 *                           or quantised to 8 bits
 *   bsa_cache_read       -- and read back, packed
 *   bsa_cache_attention  -- attention of one new token per sequence over the cache
 *   bsa_prompt_attention -- attention over packed sequences of different lengths, causal or not,
 *                           with grouped heads
 *
 * Conventions
 *   - As in bsa.h: the caller owns every buffer; no call allocates, frees or synchronises; work is
 *     enqueued on `stream` of the current device, where every buffer lives; argument checks run on
 *     the host before any launch, and a failed check enqueues nothing.
 *   - d in {64, 128}; tensors are bf16 (dt = BSA_BF16). Packed tensors [T][heads][d] are given by a
 *     pointer and element strides of token and head; channels are contiguous. Pointers are 16-byte
 *     aligned, strides positive multiples of 16 bytes (the stride of a dimension of length one is
 *     not looked at): views of a fused projection do, and [heads][T][d]. Tokens and heads of an
 *     output must not overlap.
 *   - Sequence b of B owns tokens [cu[b], cu[b + 1]) of a packed tensor, cu int32 [B + 1], cu[0] >= 0.
 *     Tokens in front of cu[0] and from cu[B] on belong to no sequence: nothing depends on them, and as results
 *     they are left as they were.
 *   - Query heads share keys in groups: H a multiple of Hk, head h uses key head h / (H / Hk).
 *   - What only the device can see goes to the workspace's first word, which bsa_check_device_error
 *     returns and clears: BSA_ERR_INVALID_ARG for a page outside the cache, a length below zero or
 *     beyond its page table, and a cu that decreases or leaves its tensor. Such a token or sequence
 *     is left out (see each call); nothing outside the buffers is read or written. Where a cu
 *     decreases, which tokens of the other sequences bsa_cache_write and bsa_cache_read move is
 *     unspecified, as are results of sequences that overlap. BSA_ERR_TIMEOUT: a bounded wait gave up.
 *   - Workspaces are 256-byte aligned; the first BSA_CACHE_ROWS_WORKSPACE bytes of a new one are
 *     zero-filled once before its first call. Calls that share one must not overlap on the GPU. One
 *     workspace of sufficient size serves all four calls in turn, captured into graphs or not. Its size
 *     does not depend on lengths or on the cache.
 *   - A result depends on the call's inputs and the device alone: sums run in an order fixed by the
 *     lengths, without atomics on values.
 *   - NaN and infinities among what a query sees go where the formulas take them, but for an infinite
 *     value whose weight lies below fp32's range: NaN, as zero times infinity, or the infinity.
 */
#ifndef BSA_CACHE_H_
#define BSA_CACHE_H_

#include "bsa.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BSA_CACHE_BF16 = 0, /* rows as they are */
    BSA_CACHE_E4M3 = 1  /* 8-bit floats with one power of two per row */
} bsa_cache_kind;

/* A cache of keys and values: pages of page_size tokens, a row of d channels per token and head.
 *
 * E4M3: a row x is held as data[c] * 2^(exp - 127): with a the largest |x[c]| of its finite
 * channels, exp - 127 is the least whole number e with a <= 448 * 2^e, within [-100, 119] (-100 for
 * a row of zeros), and data[c] is x[c] * 2^-e rounded to nearest even, saturating at 448. A channel
 * that is not finite is held as NaN. Every value held is a bf16 number. */
typedef struct {
    void *k, *v;           /* device [n_pages][heads][page_size][d] of the kind, contiguous, 16-byte aligned */
    uint8_t *k_exp, *v_exp; /* device [n_pages][heads][page_size], 16-byte aligned; not read for BF16 */
    int kind;              /* bsa_cache_kind */
    int n_pages;           /* >= 1 */
    int page_size;         /* 16, 32, 64, 128 or 256 */
    int heads, d;
} bsa_kv_cache;

/* The pages of B sequences: token t of sequence b is row t % page_size of page
 * pages[b * stride + t / page_size]. Entries behind a sequence's last page are not read. */
typedef struct {
    const int32_t *pages; /* device [B][width] */
    int64_t stride;       /* elements between sequences, >= width */
    int B, width;         /* >= 1 */
} bsa_page_table;

/* [T][heads][d], by element strides */
typedef struct {
    void *ptr;
    int64_t token, head;
} bsa_packed;

/*
 * bsa_cache_write -- the T packed tokens k, v [T][heads][d] become the last tokens of their
 * sequences: sequence b, which holds kv_lens[b] tokens with them, gets tokens cu[b] .. cu[b + 1] - 1
 * at places kv_lens[b] - (cu[b + 1] - cu[b]) on.
 *   kv_lens     device int32 [B]
 *   cu          device int32 [B + 1], or NULL: one token per sequence (T == B)
 * No other row of the cache changes. Places that two tokens of one call share (sequences that
 * share a page and both write to it) have unspecified contents. T may be 0.
 * A token whose sequence is malformed, or whose page is outside the cache, is not written. Malformed
 * sequences are reported with new tokens or without.
 * One launch. Errors: BSA_ERR_SHAPE, BSA_ERR_DTYPE, BSA_ERR_INVALID_ARG (null or misaligned
 * pointers, strides, kind, page size, k or v overlapping the cache), BSA_ERR_WORKSPACE, BSA_ERR_CUDA.
 */
bsa_status bsa_cache_write(const bsa_kv_cache *cache, const bsa_packed *k, const bsa_packed *v, int dt, int T,
                           const bsa_page_table *table, const int32_t *kv_lens, const int32_t *cu, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * bsa_cache_read -- the first cu[b + 1] - cu[b] tokens of each sequence b into tokens cu[b] ..
 * cu[b + 1] - 1 of k, v [T][heads][d]: the values that the cache holds, exactly.
 * A token whose sequence is malformed is not written; one whose page is outside the cache becomes
 * zeros. One launch. Errors: as bsa_cache_write.
 */
bsa_status bsa_cache_read(const bsa_kv_cache *cache, const bsa_page_table *table, const int32_t *cu,
                          const bsa_packed *k, const bsa_packed *v, int dt, int T, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * bsa_cache_attention -- for sequence b, head h, over its kv_lens[b] tokens j in the cache (the
 * new one among them):
 *   s_j = scale * q . k_j,   O = sum softmax(s)_j v_j,   LSE = ln sum exp(s_j)
 *   q           [B][H][d]: the token stride is the one between sequences; H a multiple of cache->heads
 *   scale       > 0, finite; 0 means 1 / sqrt(d)
 *   O           [B][H][d] (written)
 *   LSE         device fp32 [B][H], contiguous (written), or NULL
 * A sequence of length 0, or with no scores but -inf (over finite values), has O = 0 and LSE = -inf;
 * so has a malformed one. Tokens of a page outside the cache count as zeros. With an 8-bit cache the
 * products are those of the values held; scores, sums and accumulators are fp32, weights are rounded
 * to 11 bits (bf16 cache: 8 bits, and O is divided by the sum of the rounded weights). A weight of an
 * 8-bit cache is rounded together with its row's power of two, so its product is off by up to 2^-24 of
 * the largest one; the sum, of unrounded weights, has every one of them at fp32's precision, whatever
 * the values beside it. Beside an 8-bit cache q is fp16, relative to the row's largest channel: a
 * channel below 2^-17 of that is off by up to 2^-25 of it, and a score by that times scale sum |k|.
 * One launch. Errors: as bsa_cache_write.
 */
bsa_status bsa_cache_attention(const bsa_kv_cache *cache, const bsa_packed *q, int dt, int H,
                               const bsa_page_table *table, const int32_t *kv_lens, float scale, const bsa_packed *O,
                               float *LSE, void *workspace, size_t workspace_bytes, void *stream);

/*
 * bsa_prompt_attention -- attention over packed sequences: query i of sequence b (of n_q = cu_q[b + 1]
 * - cu_q[b]) sees key j (of n_k = cu_k[b + 1] - cu_k[b]) when causal == 0 or j <= i + n_k - n_q: the
 * queries are the last n_q tokens of the n_k, as in a later chunk of a prompt.
 *   q, O        [T_q][H][d];  k, v  [T_k][Hk][d];  H a multiple of Hk, H / Hk <= 128
 *   cu_q, cu_k  device int32 [B + 1]
 *   scale       as bsa_cache_attention
 *   LSE         device fp32 [H][T_q], contiguous (written), or NULL
 * A query that sees no key (no keys, or causal with n_q > n_k), or none but with scores of -inf and
 * finite values, has O = 0 and LSE = -inf. Rows of O and LSE that belong to no sequence, and those of
 * a malformed sequence, are left as they were. What a query does not see does not reach it, NaN and
 * infinities included. O must not overlap an input. T_q may be 0: nothing is enqueued, and nothing
 * reported.
 * Scores, sums and accumulators are fp32; weights are rounded to bf16, and O is divided by their sum
 * before the rounding. One to three launches (one for few sequences with T_k <= 1024).
 * Errors: as bsa_cache_write.
 */
bsa_status bsa_prompt_attention(const bsa_packed *q, const bsa_packed *k, const bsa_packed *v, int dt, int T_q,
                                int T_k, int B, int H, int Hk, int d, const int32_t *cu_q, const int32_t *cu_k,
                                int causal, float scale, const bsa_packed *O, float *LSE, void *workspace,
                                size_t workspace_bytes, void *stream);

/* Workspace bytes of bsa_cache_write and bsa_cache_read, whatever their shape; all of it is what has to be zero in a new
 * workspace of any of the calls. */
#define BSA_CACHE_ROWS_WORKSPACE 8192

/* Host-only: workspace bytes of all four calls, for at most T query tokens of at most B sequences in a call. Errors:
 * BSA_ERR_SHAPE, BSA_ERR_INVALID_ARG. */
bsa_status bsa_cache_workspace_size(int T, int B, int H, int Hk, int d, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* BSA_CACHE_H_ */
