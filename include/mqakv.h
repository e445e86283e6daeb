/*
 * mqakv: a paged key/value cache in 8 bits beside the index selection of
 * mqatopk.h, for one GB300 GPU (sm_103a): appending to it, attention over it
 * (dense, or over the keys mqa_topk_prefill selected), and its pages' copying,
 * forking, freeing and compacting.
 *
 * The cache.  A page holds page_size consecutive positions of one sequence for
 * every key/value head.  Keys and values are FP8 e4m3fn codes; each (page,
 * head) has one power-of-two scale for its keys and one for its values, held
 * as a UE8M0 byte e (2^(e - 127), 1 <= e <= 254):
 *     K[t, d] = E(k[page, head, t % page_size, d]) * 2^(k_exps[page, head] - 127)
 * Sequence s holds positions [0, seq_lens[s]) in the pages page_table[s, 0],
 * page_table[s, 1], ...; refcounts[p] counts the sequences whose tables name
 * page p (0: free).  A page that is not full belongs to one sequence only
 * (mqa_kv_fork keeps it so), which is what lets mqa_kv_append write into it.
 *
 * Conventions are those of mqatopk.h: device pointers of the current device,
 * caller-owned memory, work enqueued on `stream`, MQA_* return codes, argument
 * errors found on the host before any work, no allocation, no synchronisation
 * except in mqa_kv_get_status.  Every other call may be captured into a CUDA
 * graph; replays read the buffers' current contents.  Lengths, tables and lists are
 * read on the device: an index there that leaves its range is never followed,
 * and is recorded in the status word.
 *
 * Rows.  row_starts [max_seqs + 1] int32 (non-decreasing) says which rows of a
 * call belong to which sequence: rows [row_starts[s], row_starts[s + 1]) are
 * the LAST positions of sequence s: row i of n is position seq_lens[s] - n + i
 * (seq_lens already counts them; mqa_kv_reserve does that).  Rows before
 * row_starts[0] and at or behind row_starts[max_seqs] belong to no sequence:
 * nothing is read for them, and their outputs are left as they were.
 */
#ifndef MQAKV_H_
#define MQAKV_H_

#include "mqatopk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MQA_KV_MAX_EXTRA 4
#define MQA_KV_MAX_SEQS 65536

/* Element types of rows (queries, new keys and values, outputs). */
#define MQA_KV_BF16 0
#define MQA_KV_FP16 1
#define MQA_KV_FP32 2 /* mqa_kv_append only */

/* Device-side status bits, collected in the cache's scratch until
 * mqa_kv_get_status reads and clears them. */
#define MQA_KV_DEV_OUT_OF_PAGES 1 /* too few free pages: the call changed nothing */
#define MQA_KV_DEV_BAD_INDEX 2    /* a page or sequence index outside its range was skipped */
#define MQA_KV_DEV_BAD_LIST 4     /* a list the call refuses (see each call): it changed nothing */
#define MQA_KV_DEV_BAD_LENGTH 8   /* a length that is negative or longer than the page table */
#define MQA_KV_DEV_WAIT_TIMEOUT 16 /* a bounded wait expired: the call's outputs are undefined, later calls are not affected */

typedef struct mqa_kv_pool {
  void *data;        /* [num_pages, page_bytes] */
  size_t page_bytes;
} mqa_kv_pool;

typedef struct mqa_kv_cache {
  uint8_t *k, *v;           /* [num_pages, kv_heads, page_size, head_dim] e4m3fn codes, 16-byte aligned */
  uint8_t *k_exps, *v_exps; /* [num_pages, kv_heads] UE8M0 */
  int32_t *page_table;      /* [max_seqs, max_pages] */
  int32_t *seq_lens;        /* [max_seqs] */
  int32_t *refcounts;       /* [num_pages] (page operations only) */
  void *scratch;            /* mqa_kv_scratch_bytes, 256-byte aligned, zeroed once by the caller: the
                               status word and the page operations' lists */
  size_t scratch_bytes;
  int num_pages;            /* num_pages * kv_heads * page_size < 2^31 */
  int page_size;            /* 16, 32, 64 or 128 */
  int kv_heads;             /* 1 .. 256 */
  int head_dim;             /* 64 or 128 */
  int max_seqs;             /* 1 .. MQA_KV_MAX_SEQS */
  int max_pages;            /* columns of page_table; max_pages * page_size <= 2^30 */
  int n_extra;              /* further pools of the program's, whose pages move along */
  mqa_kv_pool extra[MQA_KV_MAX_EXTRA];
} mqa_kv_cache;

/* Bytes of `scratch` for a cache of this many pages and sequences. */
int mqa_kv_scratch_bytes(int num_pages, int max_seqs, size_t *bytes);

/* Write new keys and values: row i of sequence s goes to its position (see
 * Rows).  For each page and head it touches, the scale becomes the least power
 * of two that holds the new values' largest magnitude within 448, but not less
 * than the page's scale if the page held earlier positions of the sequence
 * (and not less than 2^-120); when it grows, the earlier codes are rounded
 * again under it.  Values are rounded to nearest even; infinities are stored
 * as 448 times the scale of the finite values, NaN as the NaN code.
 *  k, v      [rows, kv_heads, head_dim] of `type` (MQA_KV_*), the row strides in
 *            elements; heads contiguous; 16-byte aligned rows
 * Rows whose position is negative or past the table are not written.  Two
 * sequences must not share a page that the call writes. */
int mqa_kv_append(const mqa_kv_cache *cache, const void *k, const void *v, long long k_row_stride,
                  long long v_row_stride, int type, const int32_t *row_starts, int rows, void *stream);

/* Bytes of workspace for mqa_kv_attention over `rows` rows of `q_heads` heads. */
int mqa_kv_attention_workspace_bytes(int device, const mqa_kv_cache *cache, int rows, int q_heads, size_t *bytes);

/* Attention of query rows over the cache: for row r (position p of sequence s)
 * and query head h, which reads key/value head h / (q_heads / kv_heads),
 *     out[r, h] = sum_t softmax_t(scale * q[r, h] . K[t]) V[t]
 * over the positions t that the row sees: t <= p when causal, else every
 * t < seq_lens[s]; with `selected`, the listed ones among them.
 *  q         [rows, q_heads, head_dim] bf16 or fp16, 16-byte aligned rows
 *            q_row_stride elements apart; q_heads a multiple of kv_heads
 *  selected  NULL, or [rows, n_selected] int32 positions within the sequence in
 *            any order (what mqa_topk_prefill writes, whose indices are relative
 *            to the row's start); entries below 0 or not seen by the row are
 *            ignored; a position listed twice counts twice
 *  out       [rows, q_heads, head_dim] of q's type, contiguous, 16-byte aligned
 *  lse       NULL, or [rows, q_heads] fp32: the logarithm of the softmax's sum
 *  scale     in (0, 65536]
 *  max_rows  the most rows any sequence has, if the caller knows it, else 0: it
 *            only chooses the kernels (any value gives correct results).  Calls
 *            for single tokens should give it: without it one sequence may have
 *            all rows, and the kernels for prompts run as well (6 to 55 us)
 * A row that sees nothing gives zeros and lse = -inf.  A NaN code in a key or
 * value that a row sees gives NaN in every component of the heads it serves,
 * and is without effect on rows that do not see it; an infinite or NaN query
 * value does so for its row and head.  Dot products, softmax statistics and
 * sums are held in fp32; the softmax weights enter the product with V in fp16
 * (11 bits, down to 2^-24 of the largest weight times scale).  Query rows are
 * scaled by a power of two and enter the product with K in fp16, or as sums of
 * e4m3 terms (by the call's and the sequences' sizes): in either form what is
 * lost is below 2^-17 of the row's largest magnitude.  Query magnitudes below
 * 2^110 and scores within fp32's range are served, as long as scale times the
 * row's largest magnitude (1 for a row of zeros) times a page's key scale stays
 * below 2^127, whatever the codes there.
 * `out` must not overlap `q`.  `workspace` may be shared by calls that do not
 * overlap; one for `rows` rows serves every call of fewer rows, whatever
 * max_rows and `selected`.  Calls that do not write to the cache may overlap,
 * each with a workspace of its own. */
int mqa_kv_attention(const mqa_kv_cache *cache, const void *q, long long q_row_stride, int type, int q_heads,
                     const int32_t *row_starts, int rows, int max_rows, const int32_t *selected, int n_selected,
                     int causal, float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                     void *stream);

/* Test-only knobs for mqa_kv_attention_debug.  Zero-initialise for defaults. */
typedef struct mqa_kv_debug_options {
  int stall;           /* nonzero: dense attention waits for something that never
                          comes: 1 the copies of keys (and values), 2 the lookups
                          (where sequences of few columns are served: 1).  The
                          time limit ends the waits, the kernels leave and
                          MQA_KV_DEV_WAIT_TIMEOUT is recorded */
  int wait_timeout_ms; /* limit of every wait in the kernels, up to 10000; 0 = default (2000) */
} mqa_kv_debug_options;

/* mqa_kv_attention with test-only knobs (opt may be NULL). */
int mqa_kv_attention_debug(const mqa_kv_cache *cache, const void *q, long long q_row_stride, int type, int q_heads,
                           const int32_t *row_starts, int rows, int max_rows, const int32_t *selected, int n_selected,
                           int causal, float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream, const mqa_kv_debug_options *opt);

/* Extend sequences: sequence s grows by counts[s] >= 0 positions, with new
 * pages (the lowest free ones, in sequence order, then position order) behind
 * its last; their refcounts become 1.  All or nothing: too few free pages, a
 * negative count or a length past the table change nothing. */
int mqa_kv_reserve(const mqa_kv_cache *cache, const int32_t *counts, void *stream);

/* Fork: each children[i], an empty sequence, becomes a copy of parents[i]:
 * the full pages are shared, a last page that is not full is copied to a new
 * one (lowest free pages, in list order).  All or nothing: a child that is not
 * empty or is listed twice, or an index outside the sequences, is refused
 * (MQA_KV_DEV_BAD_LIST).  A child of an empty parent stays empty.  Table
 * entries behind a sequence's pages are left as they were. */
int mqa_kv_fork(const mqa_kv_cache *cache, const int32_t *parents, const int32_t *children, int n, void *stream);

/* Free sequences: each page's refcount drops by one, the sequence's table
 * entries become -1 and its length 0.  A sequence listed twice is freed once;
 * one outside the range is skipped. */
int mqa_kv_free(const mqa_kv_cache *cache, const int32_t *seqs, int n, void *stream);

/* Compact: with `live` pages in use, the i-th free page below `live` receives
 * the i-th used page at or above it, contents, refcount and every sequence's
 * table entries with it.  Afterwards pages [0, live) are used. */
int mqa_kv_compact(const mqa_kv_cache *cache, void *stream);

/* Copy pages' contents (codes, scales, extra pools): page src[i] to dst[i].
 * Tables and refcounts are not touched.  A page that is a target twice, or
 * both a source and a target, or an index outside the pages is refused
 * (MQA_KV_DEV_BAD_LIST) and nothing is copied. */
int mqa_kv_copy_pages(const mqa_kv_cache *cache, const int32_t *src, const int32_t *dst, int n, void *stream);

/* The status bits collected since the last call; clears them.  Synchronises
 * `stream`; one that is being captured is refused (MQA_ERR_INVALID_ARGUMENT),
 * and its capture goes on. */
int mqa_kv_get_status(const mqa_kv_cache *cache, int32_t *status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MQAKV_H_ */
