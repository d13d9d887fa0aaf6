/*
 * attn_cache_gb300.h -- C ABI of the 8-bit paged key / value cache: appending tokens, attention
 * over the cached tokens, and eviction by accumulated attention weight.  Part of the library of
 * attn_gb300.h; status codes, dtypes, softmax types and the rules on streams and errors are
 * that header's.
 *
 * The cache.  Pages of page_size tokens; each page holds, per kv head, page_size rows of D codes
 * and one scale for the keys and one for the values:
 *   k, v            [num_pages, Hkv, page_size, D]   8-bit codes (enum attn_cache_kind)
 *   k_scale, v_scale [num_pages, Hkv]                float, finite and >= 0
 * The value a code stands for is code * scale.  A sequence is a row of the page table and a
 * length: its token t lives in page table[b, t / page_size], slot t % page_size.  Sequences may
 * share pages that none of them appends to (a common prefix).
 *
 * Scales written by this library are powers of two,
 *   need(amax) = the least 2^e >= 2^-60 with amax <= qmax * 2^e    (qmax: 448 e4m3, 127 int8),
 * so that dividing by them is exact, and moving e4m3 codes to a larger scale is exact but for
 * codes that become subnormal.  Attention and eviction take any scale, up to 2^100 for values; a
 * value scale below 2^-60 counts as 0.
 *
 * Errors found on the device (a page id outside [0, num_pages) at a position below the length, a
 * length below 0 or past the table) are recorded in the cache's status word, read and cleared
 * with attn_check_device_status(status, stream).  Nothing is read or written through a bad page
 * id: its tokens are invisible to attention, appends to it are dropped, an eviction takes them
 * as zeros.  A length past the table counts as the table's end, a negative one as 0.
 *
 * Every call is asynchronous on `stream`, keeps no state, and may be captured into a CUDA graph
 * (lengths and tables are read on the device).  Calls that only read the cache may run at once
 * on several streams, each with its own workspace.
 */
#ifndef ATTN_CACHE_GB300_H
#define ATTN_CACHE_GB300_H

#include "attn_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif

enum attn_cache_kind {
    ATTN_CACHE_E4M3 = 1,  /* 8-bit floats, 4 exponent and 3 mantissa bits, no infinities */
    ATTN_CACHE_INT8 = 2   /* integers; this library writes -127 .. 127                   */
};

typedef struct {
    int kind;                  /* enum attn_cache_kind                                    */
    int num_pages;             /* >= 1                                                    */
    int page_size;             /* tokens per page: 16, 32, 64 or 128                      */
    int Hkv, D;                /* Hkv in 1 .. 65535; D % 16 == 0, 16 <= D <= 512          */
    void *k, *v;               /* dense, 16-byte aligned                                  */
    float *k_scale, *v_scale;  /* dense                                                   */
    uint32_t *status;          /* 256 bytes, zero-filled once: the device status word and
                                  its details (as the first 256 bytes of attn_fwd's ws)  */
} attn_cache;

/* The sequences of a call. */
typedef struct {
    int B;                     /* 0: nothing to do                                        */
    int max_pages;             /* columns of the table that hold pages; at most 2^24 tokens */
    const int32_t *table;      /* [B, max_pages], rows table_stride elements apart        */
    int64_t table_stride;
    const int32_t *lengths;    /* [B] tokens                                              */
} attn_cache_seqs;

/*
 * Append: token s < counts[b] of sequence b is quantised into position lengths[b] + s.  A page's
 * scale becomes need(amax of the new rows in it) or, if the page holds earlier tokens of the
 * sequence (positions below lengths[b]), the larger of that and its present scale; when that
 * grows, the earlier tokens' codes are requantised, code' = rn(code * old / new).  New codes are
 * rn(x * (1 / scale)) (ties to even; exact products for this library's scales).  amax runs over finite values; infinities saturate, a NaN becomes
 * e4m3's NaN, in int8 0; either is recorded in the status word.
 * Two sequences of one call must not append to the same page.  Positions past the table are
 * dropped and recorded.  lengths is not changed: lengths_out[b] = lengths[b] + counts[b], for
 * tokens that had a place (lengths_out may not alias lengths).
 */
typedef struct {
    int dtype;                 /* of k and v: enum attn_dtype                             */
    int S;                     /* rows per sequence (>= 0)                                */
    const void *k, *v;         /* [B, S, Hkv, D], element strides; d contiguous; 16-byte
                                  aligned bases and strides                               */
    int64_t k_stride_b, k_stride_s, k_stride_h;
    int64_t v_stride_b, v_stride_s, v_stride_h;
    const int32_t *counts;     /* [B] in 0 .. S (clamped), or NULL: S for every sequence  */
    int32_t *lengths_out;      /* [B] or NULL                                             */
    /* Optional accumulated weights [B, Hkv, >= max_pages * page_size] float with element
     * strides (rows may not overlap): those of the new tokens are set to 0.               */
    float *weights;
    int64_t weights_stride_b, weights_stride_h;
} attn_cache_append_args;

int attn_cache_append(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_append_args *a,
                      attn_stream_t stream);

/*
 * Attention of Sq query tokens per sequence over its cached tokens, with attn_fwd's definition
 * (scale, tanh soft-cap, sink or off-by-one column, GQA) and Sk = lengths[b] per sequence: query
 * i of sequence b stands at position p = lengths[b] - Sq + i, and key j < lengths[b] is visible
 * iff (!causal || j <= p) && (window <= 0 || p - j < window).  (A decoding step appends its tokens
 * first.)  Sequences shorter than Sq have leading queries that see nothing when causal.
 *   O   [B, Sq, Hq, D] dense, dtype of q;  LSE [B, Hq, Sq] float, natural log, sink included.
 * Rows that see nothing: O = 0, LSE = -inf or the extra column's logit.
 *
 * weights_out, if given, takes for every cached key j < lengths[b]
 *   weights_out[b, hkv, j] = weights[b, hkv, j] + sum over the queries i and the heads h of kv
 *                            head hkv of exp(t_ij - LSE_i)                       (0 if unseen)
 * in float, summed in a fixed order (no atomics).  weights == weights_out adds in place, else the
 * two may not overlap; both are [B, Hkv, >= max_pages * page_size] with the same element strides,
 * whose rows may not overlap.  Nor may O, LSE and the workspace overlap anything that the call reads.
 *
 * Head dims up to 256 run on the tensor cores with the codes widened to fp16 (exact) and
 * the queries scaled per row by a power of two into fp16: bf16 queries exactly (elements within
 * 2^-31 of the row's largest) with probabilities rounded to fp16, float queries and their
 * probabilities in two fp16 terms (22 bits).  Many bf16 rows per kv head at head dims up to
 * 128 take tcgen05 products.  What is rounded is a probability times its value's scale: half a step
 * is 2^-11 of it down to 2^-28 (tcgen05: 2^-25) of the row's largest such product, and below 2^-39
 * (2^-36) of that largest one.  Larger head dims run on fp32 FFMA kernels; there the products are
 * 0 below 2^-149 of the largest.  Logit and log2(scale) are added in float: a scale of 2^e costs
 * |e| 2^-24 of each probability.  Long key ranges are split
 * over CTAs and joined in a fixed order; how, depends on the shapes and the lengths alone.
 */
typedef struct {
    int dtype;                 /* of q and O: enum attn_dtype                             */
    int Sq, Hq;                /* Sq >= 0; Hq % Hkv == 0                                  */
    const void *q;             /* [B, Sq, Hq, D], element strides; d contiguous; 16-byte
                                  aligned base and strides                                */
    int64_t q_stride_b, q_stride_s, q_stride_h;
    int causal, window;
    float softcap, scale;
    const float *sink;         /* [Hq] or NULL                                            */
    int softmax_type;          /* enum attn_softmax_type                                  */
    const float *weights;      /* both or neither                                         */
    float *weights_out;
    int64_t weights_stride_b, weights_stride_h;
} attn_cache_fwd_args;

/* Bytes of workspace (256-byte multiple, >= 256), 0 for invalid arguments.  Grows with the
 * grid; with weights also by 4 * B * Hq * Sq * max_pages * page_size bytes (the scores), so give a
 * table no wider than the longest sequence needs. */
size_t attn_cache_fwd_workspace_size(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_fwd_args *a);

/* ws: 256-byte aligned, any content. */
int attn_cache_fwd(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_fwd_args *a, void *O,
                   float *LSE, void *ws, size_t ws_bytes, attn_stream_t stream);

/* "tc" (tcgen05), "mma" (warp-level tensor-core products), "simt" (FFMA) or "" (rejected).  Static string. */
const char *attn_cache_path_name(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_fwd_args *a);

/*
 * Eviction: per sequence and kv head, n = min(lengths[b], keep) tokens survive -- all of them if
 * lengths[b] <= keep, else the `first` first, the `recent` last, and of the others the keep -
 * first - recent of largest accumulated weight (ties: the lower position; a NaN counts as
 * largest).  They are gathered, in order, to positions 0 .. n - 1 of the pages of table_out, each
 * page and head with the scale need(amax of the values gathered into it) and codes rn(value /
 * scale); value = code * scale in float.  Heads keep different tokens.
 *
 * Out of place: a page of table_out may not hold a token that any sequence of the call still
 * reads (sequences may share pages, so an eviction in place could take another's keys).
 *   kept        [B, Hkv, keep] int32: the surviving positions, ascending, -1 past the n-th
 *   lengths_out [B] int32: n
 *   weights_out [B, Hkv, >= keep] float: their weights, 0 from the n-th to the keep-th, what lies behind
 *               as it was.  Rows as wide as table_out (its pages times page_size) are the weights that
 *               the sequences' next append and attention take.  May not overlap weights, nor lie
 *               between its rows.
 * Positions (causality, windows) count the tokens that are left from here on.
 */
typedef struct {
    int keep, first, recent;   /* keep >= 1; first, recent >= 0; first + recent <= keep   */
    const float *weights;      /* [B, Hkv, >= max_pages * page_size], element strides     */
    int64_t weights_stride_b, weights_stride_h;
    const int32_t *table_out;  /* [B, >= ceil(keep / page_size)]                          */
    int64_t table_out_stride;
    int32_t *kept, *lengths_out;
    float *weights_out;
    int64_t weights_out_stride_b, weights_out_stride_h;  /* elements; both 0: dense [B, Hkv, keep].
                                                            Rows of keep elements may not overlap */
} attn_cache_evict_args;

int attn_cache_evict(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_evict_args *a,
                     attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_CACHE_GB300_H */
