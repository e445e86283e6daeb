/*
 * mqaqk: query and key heads on their way to the paged cache of mqakv.h, for one
 * GB300 GPU (sm_103a): each head's RMS norm and position rotation in one pass.
 *
 * Conventions are those of mqatopk.h: device pointers of the current device,
 * caller-owned memory, work enqueued on `stream`, MQA_* return codes, argument
 * errors found on the host before any work, no allocation, no synchronisation.
 * The call may be captured into a CUDA graph.
 */
#ifndef MQAQK_H_
#define MQAQK_H_

#include "mqatopk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of rows and weights. */
#define MQA_QK_BF16 0
#define MQA_QK_FP16 1
#define MQA_QK_FP32 2

/* Heads of `rows` rows: [rows, heads, head_dim], heads contiguous, rows
 * row_stride elements apart (a slice of a wider projection), 16-byte aligned. */
typedef struct mqa_qk_heads {
  const void *in;
  void *out;               /* may be `in` (with its stride): the heads are replaced */
  const void *weight;      /* NULL (ones), or [head_dim] of weight_type, 16-byte aligned */
  long long in_stride, out_stride;
  int heads;               /* 0: nothing to do, the pointers are not looked at */
} mqa_qk_heads;

/* For every head x of q and k at row r:
 *     y = x / sqrt(mean(x^2) + eps) * weight        (y = x * weight where !norm)
 *     (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
 * for the pairs i < rotary / 2: (a, b) = (i, i + rotary / 2), or (2i, 2i + 1) where
 * interleaved; components from `rotary` on are not turned.  t is 2 pi times the
 * fraction of positions[r] * turns[i] / 2^64: turns[i] is the pair's frequency in
 * turns per position as a 64-bit fraction, so the product wraps as the angle does
 * and far positions are turned as exactly as near ones (the angle is rounded to fp32,
 * by at most 2^-26 of a turn).
 * All the rest is held in fp32 and rounded once to the rows' type.
 *  type         of rows in and out, MQA_QK_*;  weight_type of both weights
 *  head_dim     64, 128 or 256
 *  rotary       a multiple of 16, 0 <= rotary <= head_dim
 *  turns        [rotary / 2] int64 (NULL where rotary is 0)
 *  positions    [rows] int32 (NULL where rotary is 0)
 *  eps          >= 0, finite
 * A head that holds an infinity or NaN becomes NaN as the formula has it; nobody
 * else's does. */
int mqa_qk_norm_rope(const mqa_qk_heads *q, const mqa_qk_heads *k, int rows, int type, int weight_type, int head_dim,
                     int rotary, int interleaved, int norm, float eps, const int64_t *turns, const int32_t *positions,
                     void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MQAQK_H_ */
