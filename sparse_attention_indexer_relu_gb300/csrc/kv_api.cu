// C ABI of the paged key/value cache (include/mqakv.h): argument checks,
// workspace sizing and launches.  Host code only.
#include "kv_internal.h"

#include <algorithm>
#include <climits>
#include <cstring>

namespace {

using namespace mqa;

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

int log2_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1; }

// What a call needs of the cache beside its codes, exponents and scratch.
enum Needs { kTables = 1, kRefs = 2 };

int check_cache(const mqa_kv_cache *c, int needs) {
  if (!c) return MQA_ERR_INVALID_ARGUMENT;
  if (c->num_pages < 1 || log2_of(c->page_size) < 0 || c->kv_heads < 1 || c->kv_heads > 256 ||
      (c->head_dim != 64 && c->head_dim != 128) || c->max_seqs < 1 || c->max_seqs > MQA_KV_MAX_SEQS ||
      c->max_pages < 1 || c->n_extra < 0 || c->n_extra > MQA_KV_MAX_EXTRA)
    return MQA_ERR_INVALID_ARGUMENT;
  if ((long long)c->num_pages * c->kv_heads * c->page_size > INT_MAX ||
      (long long)c->max_pages * c->page_size > 1 << 30)  // positions, with room for a tile behind the last
    return MQA_ERR_INVALID_ARGUMENT;
  if (!c->k || !c->v || !c->k_exps || !c->v_exps || !c->scratch) return MQA_ERR_INVALID_ARGUMENT;
  if ((needs & kTables) && (!c->page_table || !c->seq_lens)) return MQA_ERR_INVALID_ARGUMENT;
  if ((needs & kRefs) && !c->refcounts) return MQA_ERR_INVALID_ARGUMENT;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->scratch, 256) || !aligned(c->page_table, 4) ||
      !aligned(c->seq_lens, 4) || !aligned(c->refcounts, 4))
    return MQA_ERR_MISALIGNED;
  for (int i = 0; i < c->n_extra; ++i)
    if (!c->extra[i].data || c->extra[i].page_bytes == 0) return MQA_ERR_INVALID_ARGUMENT;
  if (c->scratch_bytes < kv_scratch(c->num_pages, c->max_seqs).total) return MQA_ERR_WORKSPACE_TOO_SMALL;
  return MQA_OK;
}

KvView view_of(const mqa_kv_cache *c) {
  KvView v;
  v.k = c->k;
  v.v = c->v;
  v.k_exps = c->k_exps;
  v.v_exps = c->v_exps;
  v.table = c->page_table;
  v.lens = c->seq_lens;
  v.refs = c->refcounts;
  v.status = reinterpret_cast<int32_t *>(c->scratch) + kKvStatus;
  v.pages = c->num_pages;
  v.page = c->page_size;
  v.page_log2 = log2_of(c->page_size);
  v.heads = c->kv_heads;
  v.dim = c->head_dim;
  v.seqs = c->max_seqs;
  v.max_pages = c->max_pages;
  return v;
}

KvLists lists_of(const mqa_kv_cache *c) {
  const KvScratch s = kv_scratch(c->num_pages, c->max_seqs);
  uint8_t *b = reinterpret_cast<uint8_t *>(c->scratch);
  auto at = [&](size_t off) { return reinterpret_cast<int32_t *>(b + off); };
  return KvLists{at(0), at(s.src), at(s.dst), at(s.rank), at(s.seq_a), at(s.seq_b), at(s.sums)};
}

KvPools pools_of(const mqa_kv_cache *c) {
  KvPools p;
  std::memset(&p, 0, sizeof p);
  auto add = [&](void *data, size_t bytes) {
    p.data[p.n] = reinterpret_cast<uint8_t *>(data);
    p.bytes[p.n++] = bytes;
  };
  const size_t codes = (size_t)c->kv_heads * c->page_size * c->head_dim;
  add(c->k, codes);
  add(c->v, codes);
  add(c->k_exps, (size_t)c->kv_heads);
  add(c->v_exps, (size_t)c->kv_heads);
  for (int i = 0; i < c->n_extra; ++i) add(c->extra[i].data, c->extra[i].page_bytes);
  return p;
}

int code(cudaError_t e) {
  if (e == cudaSuccess) return MQA_OK;
  cudaGetLastError();
  return MQA_ERR_CUDA;
}

// Times 2^110, the largest power of two that a small query takes, it stays within fp32.
constexpr float kMaxScale = 65536.f;
// Which kernels a call runs and where their parts of the workspace lie.  The
// split kernel (kv_attn.cu) takes blocks of 8 to 32 columns; calls in which a
// sequence may have more, for which it would read the cache twice, run the tiled
// kernel (kv_prefill.cu).  In graphs, split and tiled, 8 heads of 128: 32
// sequences of up to 8K positions, 40 columns 236 and 190 us, 64: 248 and 186; 8
// of them 73 and 73, 76 and 72; heads of 64: 183 and 155, 194 and 153; 59 and 58,
// 62 and 59.  (The host knows neither lengths nor sequences with rows: one
// sequence of 32K positions would be better off in the split kernel up to 64
// columns, 57 to 59 us against 61 to 63, heads of 64 45 to 47 against 50.)
// Tiled calls leave sequences of up to kSplitCols to the split kernel (16
// columns: 40 and 46 us): beside a prompt of 2,048 rows, 63 single tokens at 32K
// positions take 0.80 ms so, and 1.90 ms with every sequence in the tiled kernel.
// The host does not know whether there are such sequences; a call without any
// pays for a launch that finds no work (3 us; joining is one launch for both
// kernels).  Nor does it know that there
// is nothing else where max_rows is missing: 32 single tokens over up to 16K
// positions take 107 us with max_rows = 1 and 130 without (4 query heads per
// key/value head of 128; 32 query heads: 70 and 108, as their 32 columns go to
// the tiled kernel then).
constexpr int kTiledFrom = 32;
constexpr int kSplitCols = 16;
// Windows and trees run the split kernel, in blocks of 16 columns, for more: where
// the call's rows x query heads x positions that a row may see stay below
// kSplitWork, as the tiled kernel's start (terms, parts, joining) takes longer than
// that work (heads of 128, 4 query heads for each of 8 key/value heads: windows of
// 1,024, 9 rows 15.5 us against 26.6 tiled, 64: 24.7 and 31.8, 16 x 16: 44.5 and 47.4,
// work 8.5 M; windows of 4,096, 64 rows: 39.7 and 47.2, work 8.5 M, 128: 62.6 and 46.1,
// 17 M; heads of 64 alike).  How far a tree's rows see the host does not know: the page
// table's width stands for it, and trees of up to kSplitTree columns in all go to the
// split kernel under any table (13 rows of 4 query heads per key/value head, 52 columns,
// after 3,001 positions: 21.7 us against 27.3 tiled; after 32K they lose, 57.6 against
// 53.0).  A wide table sends larger drafts to the tiled kernel whatever their lengths: 104
// columns of two sequences of 9,000 take 41.2 us there and 39.2 split, 208 of four of
// 3,001 31.2 and 33.1.
constexpr long long kSplitWork = 10000000;
constexpr int kSplitTree = 64;
struct AttnPlan {
  bool split, tiled, many;
  int nb, ctas, tiled_ctas;
  size_t slots_off, tiled_off, cuts_off, tiled_slots_off, factor_off, terms_off, bytes;
};
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
AttnPlan plan_attention(int sms, const mqa_kv_cache *c, int rows, int max_rows, int q_heads, bool selected,
                        const mqa_kv_view *view = nullptr) {
  const int group = q_heads / c->kv_heads;
  if (max_rows <= 0 || max_rows > rows) max_rows = rows;
  const long long cols = selected ? group : (long long)group * max_rows;
  AttnPlan p;
  bool little = false;
  if (view && (view->window || view->tree)) {
    long long sees = (long long)c->max_pages * c->page_size;
    if (view->window) sees = std::min(sees, (long long)view->window + view->sinks + max_rows);
    little = (long long)rows * q_heads * sees <= kSplitWork || (view->tree && (long long)rows * group <= kSplitTree);
  }
  p.tiled = !selected && cols > kTiledFrom && !little;
  p.split = !p.tiled || c->max_seqs > 1;
  // how the tiled kernel's parts are joined: items, were all rows one sequence's, are
  // so few that each has four parts or more
  p.many = (long long)c->kv_heads * (((long long)rows * group + kTiledCols - 1) / kTiledCols) * 4 <= sms;
  p.nb = cols <= 8 ? 1 : cols <= 16 || p.tiled || little ? 2 : cols <= 24 ? 3 : 4;
  p.ctas = sms * attn_ctas_per_sm(p.nb, c->head_dim);
  // Room for whichever block width needs most: a workspace holds for every
  // max_rows and for selected keys as well.
  int most_ctas = 0;
  size_t most_floats = 0;
  for (int nb = 1; nb <= 4; ++nb) {
    const int ctas = sms * attn_ctas_per_sm(nb, c->head_dim);
    most_ctas = std::max(most_ctas, ctas);
    most_floats = std::max(most_floats, (size_t)ctas * 2 * attn_slot_floats(nb, c->head_dim));
  }
  p.slots_off = up256((size_t)most_ctas * sizeof(int4));
  p.tiled_off = up256(p.slots_off + most_floats * sizeof(float));
  p.tiled_ctas = sms;
  p.cuts_off = p.tiled_off + up256((size_t)sms * sizeof(int4));
  p.tiled_slots_off = p.cuts_off + up256((size_t)(sms + 1) * kCutBytes);
  p.factor_off = p.tiled_slots_off + up256((size_t)sms * 2 * kTiledCols * (c->head_dim + 4) * sizeof(float));
  p.terms_off = p.factor_off + up256((size_t)rows * q_heads * sizeof(float));
  p.bytes = p.tiled ? p.terms_off + (size_t)kQueryTerms * rows * q_heads * c->head_dim : p.tiled_off;
  return p;
}

// Kernels by what their rows see.
cudaError_t launch_tiled(KvKind kind, const AttnParams &p, const CUtensorMap &map, const CUtensorMap &q_map, uint8_t *q8,
                         float *factor, int ctas, cudaStream_t stream) {
  return kind == kWindow ? launch_kv_prefill<kWindow>(p, map, q_map, q8, factor, ctas, stream)
         : kind == kTree ? launch_kv_prefill<kTree>(p, map, q_map, q8, factor, ctas, stream)
                         : launch_kv_prefill<kDense>(p, map, q_map, q8, factor, ctas, stream);
}
cudaError_t launch_split(KvKind kind, const AttnParams &p, const CUtensorMap &k_map, const CUtensorMap &v_map, int nb,
                         int ctas, bool follows, cudaStream_t stream) {
  return kind == kWindow ? launch_kv_attention<kWindow>(p, k_map, v_map, nb, ctas, follows, stream)
         : kind == kTree ? launch_kv_attention<kTree>(p, k_map, v_map, nb, ctas, follows, stream)
                         : launch_kv_attention<kDense>(p, k_map, v_map, nb, ctas, follows, stream);
}

int check_attention(const mqa_kv_cache *c, int rows, int q_heads) {
  const int rc = check_cache(c, kTables);
  if (rc != MQA_OK) return rc;
  if (rows < 0 || q_heads < 1 || q_heads % c->kv_heads != 0 || q_heads > 65536 ||
      (long long)rows * q_heads > INT_MAX / kQueryTerms)
    return MQA_ERR_INVALID_ARGUMENT;
  return MQA_OK;
}

// The call behind every attention entry; view may be null.
int attention(const mqa_kv_cache *cache, const void *q, long long q_row_stride, int type, int q_heads,
              const int32_t *row_starts, int rows, int max_rows, const int32_t *selected, int n_selected, int causal,
              const mqa_kv_view *view, float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
              void *stream, const mqa_kv_debug_options *opt) {
  int rc = check_attention(cache, rows, q_heads);
  if (rc != MQA_OK) return rc;
  if (opt && (opt->stall < 0 || opt->stall > 2 || opt->wait_timeout_ms < 0 || opt->wait_timeout_ms > 10000))
    return MQA_ERR_INVALID_ARGUMENT;
  if ((type != MQA_KV_BF16 && type != MQA_KV_FP16) || n_selected < 0 || (!selected && n_selected > 0) ||
      !(scale > 0.f && scale <= kMaxScale))
    return MQA_ERR_INVALID_ARGUMENT;
  // a window of 0 sees everything up to the row's position; a mask goes without a window
  if (view && (view->window < 0 || view->sinks < 0 || (view->sinks > 0 && view->window == 0) ||
               (view->tree ? view->tree_words < 1 || view->window != 0 : view->tree_words != 0)))
    return MQA_ERR_INVALID_ARGUMENT;
  const KvKind kind = view && view->tree ? kTree : view && view->window ? kWindow : kDense;
  if (rows == 0) return MQA_OK;
  if (!q || !out || !row_starts || !workspace ||
      (rows > 1 && q_row_stride < (long long)q_heads * cache->head_dim))
    return MQA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(out, 16) || q_row_stride % 8 || !aligned(row_starts, 4) || !aligned(selected, 4) ||
      !aligned(lse, 4) || !aligned(workspace, 256) || (kind == kTree && !aligned(view->tree, 4)))
    return MQA_ERR_MISALIGNED;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  const AttnPlan P = plan_attention(sms, cache, rows, max_rows, q_heads, selected != nullptr, view);
  if (workspace_bytes < P.bytes) return MQA_ERR_WORKSPACE_TOO_SMALL;
  AttnParams p;
  std::memset(&p, 0, sizeof p);
  p.c = view_of(cache);
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.starts = row_starts;
  p.selected = selected;
  p.q_stride = q_row_stride;
  p.rows = rows;
  p.q_heads = q_heads;
  p.group = q_heads / cache->kv_heads;
  p.n_selected = n_selected;
  p.causal = causal != 0 && kind != kTree;  // a mask alone says what is seen behind the first row
  // (positions stay below 2^30)
  if (kind == kWindow) p.window = std::min(view->window, 1 << 30), p.sinks = std::min(view->sinks, 1 << 30);
  if (kind == kTree) p.tree = view->tree, p.tree_words = view->tree_words;
  p.bf16 = type == MQA_KV_BF16;
  p.scale_log2 = scale * 1.44269504088896341f;
  p.wait_ns = (opt && opt->wait_timeout_ms ? opt->wait_timeout_ms : 2000) * 1000000ULL;
  p.stall = opt ? opt->stall : 0;
  p.test = p.stall || (opt && opt->wait_timeout_ms);
  uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
  if (P.tiled) {
    p.max_cols = P.split ? kSplitCols : 0;
    p.desc = reinterpret_cast<int4 *>(ws + P.tiled_off);
    p.slots = reinterpret_cast<float *>(ws + P.tiled_slots_off);
    p.cuts = ws + P.cuts_off;
    CUtensorMap map, q_map;
    uint8_t *terms = ws + P.terms_off;
    float *factor = reinterpret_cast<float *>(ws + P.factor_off);
    p.q_scale = factor;
    rc = encode_code_rows(&map, cache->k, (uint64_t)cache->num_pages * cache->kv_heads * cache->page_size,
                          cache->head_dim, (uint32_t)cache->page_size);
    if (rc != MQA_OK) return rc;
    rc = encode_code_rows(&q_map, terms, (uint64_t)(type == MQA_KV_BF16 ? 2 : 3) * rows * q_heads, cache->head_dim, 128);
    if (rc != MQA_OK) return rc;
    rc = code(launch_tiled(kind, p, map, q_map, terms, factor, P.tiled_ctas, as_stream(stream)));
    if (rc == MQA_OK && !P.split) rc = code(launch_kv_join_tiled(p, P.tiled_ctas, P.many, as_stream(stream)));
    if (rc != MQA_OK || !P.split) return rc;
  }
  const AttnParams tiled = p;
  p.max_cols = P.tiled ? kSplitCols : INT_MAX;
  p.desc = reinterpret_cast<int4 *>(ws);
  p.slots = reinterpret_cast<float *>(ws + P.slots_off);
  const uint64_t code_rows = (uint64_t)cache->num_pages * cache->kv_heads * cache->page_size;
  CUtensorMap k_map, v_map;
  std::memset(&k_map, 0, sizeof k_map);
  std::memset(&v_map, 0, sizeof v_map);
  if (!selected) {
    rc = encode_code_rows(&k_map, cache->k, code_rows, cache->head_dim, 16);
    if (rc == MQA_OK) rc = encode_code_rows(&v_map, cache->v, code_rows, cache->head_dim, 16);
    if (rc != MQA_OK) return rc;
  }
  rc = code(launch_split(kind, p, k_map, v_map, P.nb, P.ctas, P.tiled, as_stream(stream)));
  if (rc != MQA_OK) return rc;
  return code(P.tiled ? launch_kv_join_both(tiled, P.tiled_ctas, P.many, p, P.nb, P.ctas, as_stream(stream))
                      : launch_kv_join(p, P.nb, P.ctas, as_stream(stream)));
}

}  // namespace

extern "C" {

int mqa_kv_scratch_bytes(int num_pages, int max_seqs, size_t *bytes) {
  if (!bytes || num_pages < 1 || max_seqs < 1 || max_seqs > MQA_KV_MAX_SEQS) return MQA_ERR_INVALID_ARGUMENT;
  *bytes = kv_scratch(num_pages, max_seqs).total;
  return MQA_OK;
}

int mqa_kv_append(const mqa_kv_cache *cache, const void *k, const void *v, long long k_row_stride,
                  long long v_row_stride, int type, const int32_t *row_starts, int rows, void *stream) {
  int rc = check_cache(cache, kTables);
  if (rc != MQA_OK) return rc;
  if (rows < 0 || type < MQA_KV_BF16 || type > MQA_KV_FP32) return MQA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MQA_OK;
  const long long width = (long long)cache->kv_heads * cache->head_dim;
  if (!k || !v || !row_starts || (rows > 1 && (k_row_stride < width || v_row_stride < width)))
    return MQA_ERR_INVALID_ARGUMENT;
  const int per16 = type == MQA_KV_FP32 ? 4 : 8;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(row_starts, 4) || k_row_stride % per16 || v_row_stride % per16)
    return MQA_ERR_MISALIGNED;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  return code(launch_kv_append(view_of(cache), k, v, k_row_stride, v_row_stride, type, row_starts, rows, sms,
                               as_stream(stream)));
}

int mqa_kv_attention_workspace_bytes(int device, const mqa_kv_cache *cache, int rows, int q_heads, size_t *bytes) {
  int rc = check_attention(cache, rows, q_heads);
  if (rc != MQA_OK) return rc;
  if (!bytes) return MQA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  rc = device_sms(device, &sms);
  if (rc != MQA_OK) return rc;
  // the form for the most columns needs the most, whatever max_rows a call gives
  *bytes = plan_attention(sms, cache, rows, rows, q_heads, false).bytes;
  return MQA_OK;
}

int mqa_kv_attention(const mqa_kv_cache *cache, const void *q, long long q_row_stride, int type, int q_heads,
                     const int32_t *row_starts, int rows, int max_rows, const int32_t *selected, int n_selected,
                     int causal, float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                     void *stream) {
  return mqa_kv_attention_debug(cache, q, q_row_stride, type, q_heads, row_starts, rows, max_rows, selected,
                                n_selected, causal, scale, out, lse, workspace, workspace_bytes, stream, nullptr);
}

int mqa_kv_attention_debug(const mqa_kv_cache *cache, const void *q, long long q_row_stride, int type, int q_heads,
                           const int32_t *row_starts, int rows, int max_rows, const int32_t *selected, int n_selected,
                           int causal, float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream, const mqa_kv_debug_options *opt) {
  return attention(cache, q, q_row_stride, type, q_heads, row_starts, rows, max_rows, selected, n_selected, causal,
                   nullptr, scale, out, lse, workspace, workspace_bytes, stream, opt);
}

int mqa_kv_attention_view(const mqa_kv_cache *cache, const void *q, long long q_row_stride, int type, int q_heads,
                          const int32_t *row_starts, int rows, int max_rows, const mqa_kv_view *view, float scale,
                          void *out, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  return mqa_kv_attention_view_debug(cache, q, q_row_stride, type, q_heads, row_starts, rows, max_rows, view, scale, out,
                                     lse, workspace, workspace_bytes, stream, nullptr);
}

int mqa_kv_attention_view_debug(const mqa_kv_cache *cache, const void *q, long long q_row_stride, int type, int q_heads,
                                const int32_t *row_starts, int rows, int max_rows, const mqa_kv_view *view, float scale,
                                void *out, float *lse, void *workspace, size_t workspace_bytes, void *stream,
                                const mqa_kv_debug_options *opt) {
  if (!view) return MQA_ERR_INVALID_ARGUMENT;
  return attention(cache, q, q_row_stride, type, q_heads, row_starts, rows, max_rows, nullptr, 0, 1, view, scale, out,
                   lse, workspace, workspace_bytes, stream, opt);
}

int mqa_kv_tree_mask(const mqa_kv_cache *cache, const int32_t *parents, const int32_t *row_starts, int rows,
                     int32_t *mask, int words, int32_t *positions, void *stream) {
  int rc = check_cache(cache, kTables);
  if (rc != MQA_OK) return rc;
  if (rows < 0 || words < 1) return MQA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MQA_OK;
  if (!parents || !row_starts || !mask) return MQA_ERR_INVALID_ARGUMENT;
  if (!aligned(parents, 4) || !aligned(row_starts, 4) || !aligned(mask, 4) || !aligned(positions, 4))
    return MQA_ERR_MISALIGNED;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  return code(launch_kv_tree_mask(view_of(cache), parents, row_starts, rows, mask, words, positions, sms,
                                  as_stream(stream)));
}

int mqa_kv_accept(const mqa_kv_cache *cache, const int32_t *row_starts, int rows, const int32_t *counts,
                  const int32_t *accepted, void *stream) {
  int rc = check_cache(cache, kTables | kRefs);
  if (rc != MQA_OK) return rc;
  if (rows < 0) return MQA_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MQA_OK;
  if (!row_starts || !counts) return MQA_ERR_INVALID_ARGUMENT;
  if (!aligned(row_starts, 4) || !aligned(counts, 4) || !aligned(accepted, 4)) return MQA_ERR_MISALIGNED;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  return code(launch_kv_accept(view_of(cache), lists_of(cache), pools_of(cache), row_starts, counts, accepted, rows, sms,
                               as_stream(stream)));
}

int mqa_kv_reserve(const mqa_kv_cache *cache, const int32_t *counts, void *stream) {
  int rc = check_cache(cache, kTables | kRefs);
  if (rc != MQA_OK) return rc;
  if (!counts) return MQA_ERR_INVALID_ARGUMENT;
  if (!aligned(counts, 4)) return MQA_ERR_MISALIGNED;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  return code(launch_kv_reserve(view_of(cache), lists_of(cache), counts, as_stream(stream)));
}

int mqa_kv_fork(const mqa_kv_cache *cache, const int32_t *parents, const int32_t *children, int n, void *stream) {
  int rc = check_cache(cache, kTables | kRefs);
  if (rc != MQA_OK) return rc;
  if (n < 0 || n > cache->max_seqs) return MQA_ERR_INVALID_ARGUMENT;  // children are distinct sequences
  if (n == 0) return MQA_OK;
  if (!parents || !children) return MQA_ERR_INVALID_ARGUMENT;
  if (!aligned(parents, 4) || !aligned(children, 4)) return MQA_ERR_MISALIGNED;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  return code(launch_kv_fork(view_of(cache), lists_of(cache), pools_of(cache), parents, children, n, sms,
                             as_stream(stream)));
}

int mqa_kv_free(const mqa_kv_cache *cache, const int32_t *seqs, int n, void *stream) {
  int rc = check_cache(cache, kTables | kRefs);
  if (rc != MQA_OK) return rc;
  if (n < 0) return MQA_ERR_INVALID_ARGUMENT;
  if (n == 0) return MQA_OK;
  if (!seqs) return MQA_ERR_INVALID_ARGUMENT;
  if (!aligned(seqs, 4)) return MQA_ERR_MISALIGNED;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  return code(launch_kv_free(view_of(cache), seqs, n, as_stream(stream)));
}

int mqa_kv_compact(const mqa_kv_cache *cache, void *stream) {
  int rc = check_cache(cache, kTables | kRefs);
  if (rc != MQA_OK) return rc;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  return code(launch_kv_compact(view_of(cache), lists_of(cache), pools_of(cache), sms, as_stream(stream)));
}

int mqa_kv_copy_pages(const mqa_kv_cache *cache, const int32_t *src, const int32_t *dst, int n, void *stream) {
  int rc = check_cache(cache, 0);
  if (rc != MQA_OK) return rc;
  if (n < 0 || n > cache->num_pages) return MQA_ERR_INVALID_ARGUMENT;  // targets are distinct pages
  if (n == 0) return MQA_OK;
  if (!src || !dst) return MQA_ERR_INVALID_ARGUMENT;
  if (!aligned(src, 4) || !aligned(dst, 4)) return MQA_ERR_MISALIGNED;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  return code(launch_kv_copy(view_of(cache), lists_of(cache), pools_of(cache), src, dst, n, sms, as_stream(stream)));
}

int mqa_kv_get_status(const mqa_kv_cache *cache, int32_t *status, void *stream) {
  int rc = check_cache(cache, 0);
  if (rc != MQA_OK) return rc;
  if (!status) return MQA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  int32_t *word = reinterpret_cast<int32_t *>(cache->scratch) + kKvStatus;
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(as_stream(stream), &capture);
  if (e == cudaSuccess && capture != cudaStreamCaptureStatusNone) return MQA_ERR_INVALID_ARGUMENT;
  if (e == cudaSuccess) e = cudaMemcpyAsync(status, word, sizeof(int32_t), cudaMemcpyDeviceToHost, as_stream(stream));
  if (e == cudaSuccess) e = cudaMemsetAsync(word, 0, sizeof(int32_t), as_stream(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  return code(e);
}

}  // extern "C"
