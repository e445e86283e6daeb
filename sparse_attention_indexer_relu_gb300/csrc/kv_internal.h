// Definitions shared by the paged key/value cache's translation units (public
// C ABI: include/mqakv.h).
#pragma once
#include "../../include/mqakv.h"

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mqa {

// The calling thread's current device, checked to be a GB300 (mqatopk_api.cu).
int require_device(int *sms);
// SM count of a device (any model).
int device_sms(int device, int *sms);
// Tensor map over `rows` rows of `dim` (64 or 128) codes, boxes of `box` rows,
// swizzled by the row length.
int encode_code_rows(CUtensorMap *map, const void *base, uint64_t rows, int dim, uint32_t box);

// Cache fields as the kernels take them.
struct KvView {
  uint8_t *k, *v, *k_exps, *v_exps;
  int32_t *table, *lens, *refs, *status;
  int pages, page, page_log2, heads, dim, seqs, max_pages;
};

// Scratch: a 256-byte header of int32 words, then lists.
enum KvWord : int {
  kKvStatus = 0,  // MQA_KV_DEV_* bits, sticky
  kKvOk = 1,      // the planned page operation goes ahead
  kKvCount = 2,   // pages to move
  kKvLive = 3,    // compact: pages in use
};
constexpr size_t kKvHeaderBytes = 256;
constexpr int kCompactPages = 4096;  // pages per block of the compaction's scans
struct KvScratch {
  size_t src, dst, rank, seq_a, seq_b, sums, total;  // byte offsets
};
inline KvScratch kv_scratch(int pages, int seqs) {
  KvScratch s;
  const size_t p = ((size_t)pages * 4 + 255) / 256 * 256, q = ((size_t)seqs * 4 + 255) / 256 * 256;
  s.src = kKvHeaderBytes;
  s.dst = s.src + p;
  s.rank = s.dst + p;
  s.seq_a = s.rank + p;
  s.seq_b = s.seq_a + q;
  s.sums = s.seq_b + q;
  s.total = s.sums + ((size_t)(pages + kCompactPages - 1) / kCompactPages * 4 + 255) / 256 * 256;
  return s;
}

// Attention call.
struct AttnParams {
  KvView c;
  const void *q;
  void *out;
  float *lse;
  const int32_t *starts;    // [seqs + 1]
  const int32_t *selected;  // [rows, n_selected] or null
  long long q_stride;
  int rows, q_heads, group, n_selected, causal, bf16;
  float scale_log2;  // softmax scale * log2(e)
  int max_cols;      // sequences of more (row, head of the group) columns go to the tiled kernel
  int4 *desc;        // per CTA: the split item it began, for the joining kernel
  float *slots;      // per CTA: two slots of partial results
  const float *q_scale;  // tiled kernel: per column, what its products are multiplied with
  // tests only (mqa_kv_debug_options): their compilations are to run, with this
  // limit of a wait, and waits that nothing ends
  int test;
  unsigned long long wait_ns;
  int stall;
};

// Column block sizes (8 * NB) of the split kernel, its CTAs per SM and threads.
constexpr int kAttnThreads = 128;
int attn_ctas_per_sm(int nb, int dim);
size_t attn_slot_floats(int nb, int dim);
// Columns per item of the tiled kernel (p.max_cols: it takes the sequences of
// more columns).
constexpr int kTiledCols = 256;
constexpr int kQueryTerms = 3;  // e4m3 terms of an fp16 query value; a bf16 one has 2
// map: the keys' codes as rows of head_dim bytes, boxes of one page; q_map: the
// query terms (q8, workspace of kQueryTerms * rows * q_heads * head_dim bytes)
// in boxes of 128 rows; factor: rows * q_heads floats, p.q_scale.
cudaError_t launch_kv_prefill(const AttnParams &p, const CUtensorMap &map, const CUtensorMap &q_map, uint8_t *q8,
                              float *factor, int ctas, cudaStream_t stream);
// Its joining pass (p.desc and p.slots are the tiled kernel's).
cudaError_t launch_kv_join_tiled(const AttnParams &p, int ctas, cudaStream_t stream);
// follows: another kernel of the same call is before it on the stream.
// k_map, v_map: codes as rows of head_dim bytes, boxes of 16 rows (not used for
// selected keys).
cudaError_t launch_kv_attention(const AttnParams &p, const CUtensorMap &k_map, const CUtensorMap &v_map, int nb,
                                int ctas, bool follows, cudaStream_t stream);

cudaError_t launch_kv_append(const KvView &c, const void *k, const void *v, long long ks, long long vs, int type,
                             const int32_t *starts, int rows, int sms, cudaStream_t stream);

struct KvPools {
  uint8_t *data[4 + MQA_KV_MAX_EXTRA];
  unsigned long long bytes[4 + MQA_KV_MAX_EXTRA];
  int n;
};
struct KvLists {
  int32_t *head, *src, *dst, *rank, *seq_a, *seq_b, *sums;
};
cudaError_t launch_kv_reserve(const KvView &c, const KvLists &l, const int32_t *counts, cudaStream_t stream);
cudaError_t launch_kv_fork(const KvView &c, const KvLists &l, const KvPools &pools, const int32_t *parents,
                           const int32_t *children, int n, int sms, cudaStream_t stream);
cudaError_t launch_kv_free(const KvView &c, const int32_t *seqs, int n, cudaStream_t stream);
cudaError_t launch_kv_compact(const KvView &c, const KvLists &l, const KvPools &pools, int sms, cudaStream_t stream);
cudaError_t launch_kv_copy(const KvView &c, const KvLists &l, const KvPools &pools, const int32_t *src,
                           const int32_t *dst, int n, int sms, cudaStream_t stream);

}  // namespace mqa
