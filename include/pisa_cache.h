/*
 * pisa_cache.h — a paged key/value cache next to the dense calls of pisa.h: tokens are appended to
 * it, read back into dense tensors, and attended over.
 *
 * What it is for: a video that is generated frame after frame (or a prompt that grows token after
 * token) keeps the keys and values of what it has already seen.  pisa_cache_append stores the new
 * tokens' keys and values, pisa_cache_attention lets the new tokens attend over everything stored,
 * and pisa_cache_read gives stored tokens back as the dense [B, H, L, d] tensors that
 * pisa_precompute and pisa_attention take.
 *
 * The pool is a dense array of pages, [num_pages, kv_heads, page, head_dim] for keys and the same
 * for values; a sequence owns any pages in any order, listed in its row of the page table: token p of
 * sequence b lives in page page_table[b][p / page], slot p % page.  Sequences may share pages that
 * are only read.  The method's description has no counterpart to these calls.
 *
 * Conventions are those of pisa.h: device pointers on the current CUDA device, 16-byte aligned,
 * caller-owned memory, work enqueued on `stream` and asynchronous, arguments checked before
 * anything is enqueued.  What only the device knows (lengths, page numbers) is checked there: a bad
 * value sets the status word of ws (pisa_read_device_error) and is never followed.
 */
#ifndef PISA_CACHE_H_
#define PISA_CACHE_H_

#include "pisa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of the stored keys and values.  Token tensors (q, k, v, o) are bf16 with PISA_CACHE_BF16 and
 * PISA_CACHE_E4M3, fp32 with PISA_CACHE_FP32.
 *
 * PISA_CACHE_E4M3 stores each token's head as head_dim e4m3 codes and one biased exponent byte:
 *     value = code * 2^(exp - 127),  exp - 127 = the smallest e with max|x| <= 448 * 2^e, kept in
 *     [-50, 50]; code = e4m3(x * 2^-e), to nearest even, saturated.
 * A power of two keeps every stored value a bf16 number (reading back is exact) and lets the
 * attention kernels carry it in the exponents of the softmax weights; the limit of 50 is what their
 * fp32 sums can take.  Rows above 448 * 2^50 saturate, an infinity is stored as the largest code,
 * NaN stays NaN.
 *
 * Attention and read expect an exponent byte in [PISA_CACHE_EXP_MIN, PISA_CACHE_EXP_MAX] in every slot of the
 * lengths that they are given, and pisa_cache_append writes no other.  A caller whose lengths may cover slots that were
 * never appended fills the exponents with PISA_CACHE_EXP_MIN, a row of zeros' (zeroed codes with a byte of 0 are not zeros). */
#define PISA_CACHE_EXP_MIN 77
#define PISA_CACHE_EXP_MAX 177
typedef enum { PISA_CACHE_BF16 = 0, PISA_CACHE_FP32 = 1, PISA_CACHE_E4M3 = 2 } pisa_cache_dtype;

typedef struct {
  int32_t num_pages;      /* >= 1; num_pages * kv_heads * page < 2^31 */
  int32_t kv_heads;       /* >= 1 */
  int32_t page;           /* tokens a page: 16, 32, 64 or 128 */
  int32_t head_dim;       /* 64 or 128 */
  int32_t dtype;          /* pisa_cache_dtype */
  void* k;                /* [num_pages, kv_heads, page, head_dim] */
  void* v;
  uint8_t* k_exp;         /* PISA_CACHE_E4M3 only: [num_pages, kv_heads, page] */
  uint8_t* v_exp;
} pisa_cache;

/* The sequences of a call.  `max_new` and `max_len` are the host's upper bounds on what the device
 * arrays hold (they size the launch and are checked against); n_b is the number of sequence b's new
 * tokens, which are always its last ones: positions lens[b] - n_b ... lens[b] - 1.
 *   packed  (starts non-null):  sequence b's new tokens are rows starts[b] ... starts[b+1] - 1 of
 *           the token tensors, n_b = starts[b+1] - starts[b];
 *   padded  (starts null):  its i-th new token is row i of its own part of the token tensors
 *           (pisa_rows.seq_stride), n_b = counts[b], or max_new for every sequence if counts is null.
 * At most one of starts and counts may be non-null. */
typedef struct {
  int32_t batch;               /* >= 0 */
  int32_t max_pages;           /* row length of page_table */
  int32_t max_len;             /* >= every lens[b]; <= max_pages * page */
  int32_t max_new;             /* >= every n_b */
  const int32_t* page_table;   /* [batch, max_pages]; of a row only the first ceil(lens[b] / page) are read, and
                                * none whose tokens all lie before what a windowed attention sees */
  const int32_t* lens;         /* [batch] tokens of each sequence, the new ones included */
  const int32_t* starts;       /* nullable [batch + 1] */
  const int32_t* counts;       /* nullable [batch] */
} pisa_sequences;

/* A token tensor: element (b, row, head, c) is data[b * seq_stride + row * row_stride +
 * head * head_stride + c], strides in elements (seq_stride is not used for packed sequences).  Rows
 * are `head_dim` contiguous elements; every used stride is a multiple of 16 bytes.  `rows` is the
 * number of rows there are: of the whole tensor (packed; data may be null if there is none) or of each
 * sequence (padded, >= max_new).
 * [B, H, L, d] is {data, L, H*L*d, d, L*d}; packed [T, H, d] is {data, T, 0, H*d, d}. */
typedef struct {
  void* data;
  int32_t rows;
  int64_t seq_stride;
  int64_t row_stride;
  int64_t head_stride;
} pisa_rows;

#define PISA_DEVERR_BAD_PAGE 3     /* a page number out of [0, num_pages) */
#define PISA_DEVERR_BAD_LENGTH 4   /* a length, count or start out of its range */

/* Bytes of device scratch that the three calls need, for any sequences: the status word (256 bytes),
 * then partial results of sequences that several thread blocks share.  0 if the cache's sizes or
 * type are not supported.  ws must be zeroed once before its first use; after a reported device
 * timeout zero it again.  Calls that share one ws must not run at the same time. */
PISA_API size_t pisa_cache_workspace_bytes(const pisa_cache* cache);

/* Writes the new tokens' keys and values into their pages.  Two sequences must not append to the
 * same slot (the result would be one or the other).  A sequence whose length or count is out of
 * range, or with more new tokens than lens[b], is skipped; so is a token whose page is out of range.
 * Nothing else of the pool changes. */
PISA_API pisa_status pisa_cache_append(const pisa_cache* cache, const pisa_sequences* seqs, const pisa_rows* k,
                                       const pisa_rows* v, void* ws, size_t ws_bytes, pisa_stream_t stream);

/* Copies each sequence's last n_b tokens out of their pages (n_b = lens[b]: the whole sequence), as
 * values.  Rows that no token belongs to, and skipped ones (as for pisa_cache_append), are left as
 * they were. */
PISA_API pisa_status pisa_cache_read(const pisa_cache* cache, const pisa_sequences* seqs, const pisa_rows* k,
                                     const pisa_rows* v, void* ws, size_t ws_bytes, pisa_stream_t stream);

/* Attention of the new tokens over the cached tokens of their sequence (append them first).  Token i
 * of sequence b has position p = lens[b] - n_b + i and sees the cached positions j with
 *     0 <= j < lens[b],   j <= p if causal != 0,   j > p - window if window > 0:
 *     o = sum_j w_j v_j / sum_j w_j,   w_j = exp(softmax_scale * q . k_j).
 * Sums, maxima and logits are fp32.  Where products run on the tensor cores the weights enter the one with V in the
 * type that it asks of them: fp32 pools in three bf16 parts (24 bits), e4m3 pools as fp16 (11 bits), bf16 pools in two
 * bf16 parts (16 bits) for at most 16 rows (new tokens times heads / kv_heads) and as bf16 (8 bits) for more.
 * Query head h reads key/value head h / (heads / kv_heads).  Without causal, n_b may exceed lens[b]
 * (queries that are not in the cache).  A token that sees nothing gets o = 0 and lse = -inf; a
 * position that a token does not see has no part in its result, whatever is stored there.
 * lse: nullable fp32, log(sum_j w_j) of row r, head h at lse[r * heads + h] (packed) or
 * lse[(b * heads + h) * q->rows + r] (padded); with it, results over several caches can be joined.
 * A sequence whose length is out of range counts as empty; one whose count or start is out of range
 * is skipped; the keys of a page out of range are not seen.  o must not overlap q. */
PISA_API pisa_status pisa_cache_attention(const pisa_cache* cache, const pisa_sequences* seqs, int32_t heads,
                                          int32_t causal, int32_t window, float softmax_scale, const pisa_rows* q,
                                          const pisa_rows* o, float* lse, void* ws, size_t ws_bytes,
                                          pisa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PISA_CACHE_H_ */
