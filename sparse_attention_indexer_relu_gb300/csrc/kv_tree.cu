// Drafted tokens over the paged 8-bit cache (include/mqakv.h): the masks and
// positions of a tree of drafts (mqa_kv_tree_mask), and taking over the accepted
// ones (mqa_kv_accept).
#include "kv_pages.cuh"
#include "kv_ptx.cuh"

#include <algorithm>
#include <cuda_fp8.h>

namespace mqa {

namespace {

struct Rows {
  int r0, n;
};
__device__ __forceinline__ Rows rows_of(const int32_t *starts, int s, int rows) {
  Rows r;
  r.r0 = min(max(__ldg(starts + s), 0), rows);
  r.n = max(min(__ldg(starts + s + 1), rows) - r.r0, 0);
  return r;
}

// ------------------------------------------------------------------ masks
// sees(i) = {i} + sees(parent(i)).  A thread walks up from its row; parents come
// before their children, so the words of the mask are finished from the highest
// down, each written once.  Bound by the launch and the walk's depth (one draft of 13
// rows 2.6 us in a graph, 256 of up to 64 rows 3.9).
constexpr int kMaskThreads = 128;
constexpr int kMaskHeld = 1024;  // parents of a sequence kept in shared memory

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const KvView c, const int32_t *__restrict__ parents,
                                                                 const int32_t *__restrict__ starts, int rows,
                                                                 int32_t *__restrict__ mask, int words,
                                                                 int32_t *__restrict__ positions, int per) {
  __shared__ int s_parent[kMaskHeld];
  const int lane = threadIdx.x & 31, s0 = blockIdx.x * per;
  bool on = false;
  if (lane < per && s0 + lane < c.seqs) on = rows_of(starts, s0 + lane, rows).n > 0;
  for (uint32_t left = __ballot_sync(~0u, on); left; left &= left - 1) {
    const int s = s0 + __ffs(left) - 1;
    const Rows r = rows_of(starts, s, rows);
    const int first = min(max(__ldg(c.lens + s), 0), c.max_pages << c.page_log2) - r.n;
    // a parent that is no earlier row counts as none
    auto checked = [&](int i) {
      const int up = __ldg(parents + r.r0 + i);
      if (up >= -1 && up < i) return up;
      atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
      return -1;
    };
    for (int i = threadIdx.x; i < min(r.n, kMaskHeld); i += kMaskThreads) s_parent[i] = checked(i);
    __syncthreads();
    for (int i = threadIdx.x; i < r.n; i += kMaskThreads) {
      int32_t *row = mask + (size_t)(r.r0 + i) * words;
      int w = i >> 5, depth = 0;
      for (int k = words - 1; k > w; --k) row[k] = 0;
      uint32_t bits = 1u << (i & 31);
      for (int at = i;;) {
        at = at < kMaskHeld ? s_parent[at] : checked(at);
        if (at < 0) break;
        ++depth;
        for (; w > at >> 5; bits = 0, --w)
          if (w < words) row[w] = (int32_t)bits;
        bits |= 1u << (at & 31);
      }
      for (; w >= 0; bits = 0, --w)
        if (w < words) row[w] = (int32_t)bits;
      if (positions) positions[r.r0 + i] = first + depth;
    }
    __syncthreads();  // the parents have been read
  }
}

// ------------------------------------------------------------------ accepting
// What a call asks of a sequence, checked: rows [r0, r0 + n) are its last
// positions from `first` on, `keep` of them stay (-1: the sequence is left alone).
struct Asked {
  int r0, n, first, keep;
};
__device__ __forceinline__ Asked asked_of(const KvView &c, const int32_t *starts, const int32_t *counts, int s, int rows,
                                          int32_t *status) {
  const Rows r = rows_of(starts, s, rows);
  Asked a{r.r0, r.n, 0, -1};
  if (r.n == 0) return a;
  const int len = c.lens[s], keep = __ldg(counts + s);  // (the kernel writes lengths: an ordinary load)
  if (len < r.n || len > c.max_pages << c.page_log2) {
    if (status) atomicOr(status, MQA_KV_DEV_BAD_LENGTH);
  } else if (keep < 0 || keep > r.n) {
    if (status) atomicOr(status, MQA_KV_DEV_BAD_LIST);
  } else {
    a.first = len - r.n;
    a.keep = keep;
  }
  return a;
}
// A thread's entry of a sequence's list and the one before it, asked for beside the length
// and the count (those behind the kept ones, which mean nothing, are within the list too).
struct Entry {
  int at, prev;
};
__device__ __forceinline__ Entry entry_of(const int32_t *starts, const int32_t *accepted, int s, int rows) {
  const Rows r = rows_of(starts, s, rows);
  const int32_t *at = accepted + r.r0 + threadIdx.x;
  const bool on = accepted && (int)threadIdx.x < r.n;
  return {on ? __ldg(at) : 0, on && threadIdx.x > 0 ? __ldg(at - 1) : -1};
}
// How many of a sequence's kept rows are where they belong (the first ones); -1, and bad, where
// the list does not ascend within the sequence's rows.  By the CTA.
__device__ __forceinline__ int settled(const Asked &a, const int32_t *accepted, Entry e, int threads, bool &bad) {
  if (!accepted) return a.keep;
  int stay = 0;
  bool odd = false;
  for (int i = threadIdx.x; i - (int)threadIdx.x < a.keep; i += threads) {
    if (i >= threads && i < a.keep) e = {__ldg(accepted + a.r0 + i), __ldg(accepted + a.r0 + i - 1)};
    odd |= i < a.keep && (e.at >= a.n || e.at <= e.prev || e.at < 0);
    stay += __syncthreads_count(i < a.keep && e.at == i);
  }
  bad = __syncthreads_or(odd);
  return bad ? -1 : stay;
}

__device__ __forceinline__ float from_e4m3(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
  return __half2float(__half(h));
}
// The larger of m and the magnitudes of a word's codes, as code bits (ordered like
// the values); NaN codes do not count.
__device__ __forceinline__ uint32_t top_code(uint32_t m, uint32_t w) {
  return __vmaxu4(m, w & 0x7F7F7F7Fu & ~((nan_bytes(w) >> 7) * 255u));
}
// Least exponent byte whose scale holds a code's magnitude, under scale byte e,
// within 448 (0: any).
__device__ __forceinline__ int needed_exp(uint32_t code, int e) {
  const uint32_t b = __float_as_uint(from_e4m3(code));
  return code ? e + (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0) : 0;
}
// Codes times f.
__device__ __forceinline__ uint32_t scaled(uint32_t w, float f) {
  const float2 a = half2_to_float2(cvt2(w)), b = half2_to_float2(cvt2_hi(w));
  return to_e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}
__device__ __forceinline__ uint4 scaled(uint4 v, float f) {
  return make_uint4(scaled(v.x, f), scaled(v.y, f), scaled(v.z, f), scaled(v.w, f));
}
// 2^d, of as much of d as matters for a product with a code.
__device__ __forceinline__ float step_by(int d) { return pow2i(min(max(d, -60), 60)); }

// ---- plan
// What a call does is decided before anything changes, for what one sequence gives back
// another may look at: lists are checked, and pages that rows move into, or in which a
// shortened sequence ends without filling it, are the sequence's own afterwards.  Where
// such a page is shared (its count is above 1) the sequence gets a copy, as kv_fork makes
// of a page that is not full; otherwise appending would write over the others' positions.
//
// A CTA per sequence (of a few, those that have rows) leaves in seq_a how many of its
// rows are where they belong (-1: the sequence is left alone) and in seq_b the number
// of pages to copy (-1: none).  The CTA that is done last deals free pages out, lowest first, by
// sequence, then position, which seldom is needed: src, dst and rank then hold the pairs and the
// places in the table, a sequence's from seq_b on, the sign bit marking its last.
constexpr int kAcceptPlan = 128;

// The places in the table of pages that are to be the sequence's own: [lo, hi).
struct Own {
  int lo, hi;
};
__device__ __forceinline__ Own own_of(const KvView &c, const Asked &a, int stay) {
  const int now = a.first + a.keep, end = (now + c.page - 1) >> c.page_log2;
  if (a.keep == a.n) return {end, end};  // nothing changes
  if (stay < a.keep) return {(a.first + stay) >> c.page_log2, end};
  return {now >> c.page_log2, end};  // empty where the last page is full
}
__device__ __forceinline__ bool shared(const KvView &c, int page) {
  return (unsigned)page < (unsigned)c.pages && c.refs[page] > 1;
}

__device__ __noinline__ void deal_pages(const KvView &c, const KvLists &l, const int32_t *starts, const int32_t *counts,
                                        int rows, int need, int *sums) {
  const bool enough = need <= c.pages && lowest_free<kAcceptPlan>(c, need, l.dst, sums) == need;
  if (!enough && threadIdx.x == 0) atomicOr(c.status, MQA_KV_DEV_OUT_OF_PAGES);
  int total = 0;
  for (int base = 0; base < c.seqs; base += kAcceptPlan) {
    const int s = base + threadIdx.x;
    const int n = s < c.seqs && rows_of(starts, s, rows).n > 0 ? max(__ldcg(l.seq_b + s), 0) : 0;
    int excl;
    const int sum = block_scan(n, excl, sums);
    if (n > 0 && enough) {
      const Own own = own_of(c, asked_of(c, starts, counts, s, rows, nullptr), __ldcg(l.seq_a + s));
      const int32_t *table = c.table + (size_t)s * c.max_pages;
      int k = total + excl;
      for (int j = own.lo; j < own.hi; ++j)
        if (shared(c, table[j])) l.src[k] = table[j], l.rank[k++] = j;
      l.rank[k - 1] |= INT32_MIN;
      l.seq_b[s] = k - n;
    } else if (n > 0) {
      l.seq_a[s] = l.seq_b[s] = -1;
    }
    total += sum;
  }
  __syncthreads();  // the counts have been read
  if (!enough) return;
  for (int s = threadIdx.x; s < c.seqs; s += kAcceptPlan) {
    int k = rows_of(starts, s, rows).n > 0 ? __ldcg(l.seq_b + s) : -1;
    for (bool more = k >= 0; more; ++k) {
      more = l.rank[k] >= 0;
      c.table[(size_t)s * c.max_pages + (l.rank[k] & INT32_MAX)] = l.dst[k];
      c.refs[l.dst[k]] = 1;
      drop_page(c, l.src[k]);
    }
  }
}

__global__ void __launch_bounds__(kAcceptPlan) accept_plan_kernel(const KvView c, const KvLists l,
                                                                  const int32_t *__restrict__ starts,
                                                                  const int32_t *__restrict__ counts,
                                                                  const int32_t *__restrict__ accepted, int rows, int per) {
  grid_dependents();
  __shared__ int sums[32], s_need;
  const int tid = threadIdx.x, lane = tid & 31, s0 = blockIdx.x * per;
  bool on = false;
  int need = 0;  // pages to copy
  if (lane < per && s0 + lane < c.seqs) on = rows_of(starts, s0 + lane, rows).n > 0;
  for (uint32_t left = __ballot_sync(~0u, on); left; left &= left - 1) {
    const int s = s0 + __ffs(left) - 1;
    const Entry entry = entry_of(starts, accepted, s, rows);
    const Asked a = asked_of(c, starts, counts, s, rows, tid == 0 ? c.status : nullptr);
    const int32_t *table = c.table + (size_t)s * c.max_pages;
    // the first pages' counts are on their way while the list is checked
    const int at = (a.first >> c.page_log2) + tid;
    const bool is_shared = a.keep >= 0 && at << c.page_log2 < a.first + a.n && shared(c, table[at]);
    bool bad = false;
    const int stay = a.keep < 0 ? -1 : settled(a, accepted, entry, kAcceptPlan, bad);
    int pages = 0;
    if (bad) {
      if (tid == 0) atomicOr(c.status, MQA_KV_DEV_BAD_LIST);
    } else if (a.keep >= 0) {
      const Own own = own_of(c, a, stay);
      pages = __syncthreads_count(is_shared && at >= own.lo && at < own.hi);
      for (int j = max(own.lo, at - tid + kAcceptPlan) + tid; j - tid < own.hi; j += kAcceptPlan)
        pages += __syncthreads_count(j < own.hi && shared(c, table[j]));
    }
    if (tid == 0) {
      l.seq_a[s] = stay;
      l.seq_b[s] = pages ? pages : -1;
    }
    need += pages;
  }
  if (gridDim.x > 1) {  // the one that comes last learns the sum
    if (tid == 0) {
      unsigned long long *const ticket = reinterpret_cast<unsigned long long *>(l.head + kKvTicket);
      if (need) __threadfence();
      const unsigned long long was = atomicAdd(ticket, (unsigned long long)need << 32 | 1);
      s_need = 0;
      if ((uint32_t)was == gridDim.x - 1) {
        *ticket = 0;
        s_need = (int)(was >> 32) + need;
        if (s_need) __threadfence();
      }
    }
    __syncthreads();
    need = s_need;
  } else {
    __syncthreads();
  }
  if (need) deal_pages(c, l, starts, counts, rows, need, sums);
}

// ---- moving
// Contents of a page, by the CTA.
__device__ __noinline__ void copy_page(const KvPools &p, int from, int to) {
  for (int i = 0; i < p.n; ++i) {
    const unsigned long long size = p.bytes[i];
    const uint8_t *s = p.data[i] + (unsigned long long)from * size;
    uint8_t *d = p.data[i] + (unsigned long long)to * size;
    if (((reinterpret_cast<uintptr_t>(s) | reinterpret_cast<uintptr_t>(d) | size) & 15) == 0) {
      for (unsigned long long x = threadIdx.x; x < size / 16; x += blockDim.x)
        reinterpret_cast<uint4 *>(d)[x] = reinterpret_cast<const uint4 *>(s)[x];
    } else {
      for (unsigned long long x = threadIdx.x; x < size; x += blockDim.x) d[x] = s[x];
    }
  }
}

// A CTA has a sequence (of a few, those that have rows): it makes the copies that the
// plan names, looks up where its kept rows come from and go to, a warp moves a head's
// keys or values, and then the length and the pages behind it follow.
//
// A warp goes over the pages that rows move into, in order.  A page's scale depends on
// all that moves into it, so its rows are read for their largest magnitude first; few
// enough stay in registers, others are read again.  In both cases a row is read
// before its source is overwritten: rows come from their own places or later ones, in
// order, so that what is written at any time lies before all sources still to be read,
// and the scales of pages behind this one have not changed yet.
//
// Bound by the chain of loads bounds -> lengths, list -> table -> scales and rows, all
// from HBM, and for kept rows of more than a page by their order (256 sequences of up
// to 64 rows, a third of them kept, 8 heads of 128, 15 MB moved: 20 us in a graph with
// three copies of tables before it, 13 rows of one sequence 9.2; of it 3.0 and 2.3 for the
// plan's kernel, beside which this one looks its places up; 21.3 and 10.4 where it waits
// for the plan first).
constexpr int kAcceptWarps = 16;
constexpr int kMoved = 1024;  // rows looked up at once

template <int D>
__global__ void __launch_bounds__(32 * kAcceptWarps) accept_kernel(const KvView c, const KvLists l, const KvPools pools,
                                                                   const int32_t *__restrict__ starts,
                                                                   const int32_t *__restrict__ counts,
                                                                   const int32_t *__restrict__ accepted, int rows,
                                                                   int per) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, STEPS = 4, HELD = RPS * STEPS;  // lanes per row, rows per step, rows held
  __shared__ int s_src[kMoved], s_dst[kMoved / 16 + 1];  // source rows (page * page size + slot, or -1), pages
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads / 32;
  const int s0 = blockIdx.x * per;
  bool on = false;
  if (lane < per && s0 + lane < c.seqs) on = rows_of(starts, s0 + lane, rows).n > 0;
  bool planned = false;
  // What is only looked up does not wait for the plan.
  for (uint32_t left = __ballot_sync(~0u, on); left; left &= left - 1) {
    const int s = s0 + __ffs(left) - 1;
    const Entry entry = entry_of(starts, accepted, s, rows);
    const Asked a = asked_of(c, starts, counts, s, rows, nullptr);
    bool bad = false;
    const int stay = a.keep < 0 ? -1 : settled(a, accepted, entry, threads, bad);
    if (stay < 0) continue;
    const int32_t *list = accepted + a.r0;
    int32_t *table = c.table + (size_t)s * c.max_pages;
    // Places of the kept rows from `from` on; those looked up at once end with a page's last one.
    auto look_up = [&](int from) {
      const int begin = a.first + from, to = min(a.keep, ((begin + kMoved) & ~(c.page - 1)) - a.first);
      for (int i = tid; i < to - from; i += threads) {
        const int pos = a.first + __ldg(list + from + i), page = __ldcg(table + (pos >> c.page_log2));
        s_src[i] = (unsigned)page < (unsigned)c.pages ? (page << c.page_log2) + (pos & (c.page - 1)) : -1;
      }
      const int pages = ((a.first + to - 1) >> c.page_log2) - (begin >> c.page_log2) + 1;
      for (int i = tid; i < pages; i += threads) s_dst[i] = __ldcg(table + (begin >> c.page_log2) + i);
      __syncthreads();
      return to;
    };
    const bool moves = stay < a.keep;
    int to = 0;
    if (moves) to = look_up(stay);
    if (!planned) grid_wait();
    planned = true;
    if (__ldcg(l.seq_a + s) < 0) continue;  // too few pages
    int pair = __ldcg(l.seq_b + s);
    if (pair >= 0) {
      for (bool more = true; more; ++pair) {
        more = __ldcg(l.rank + pair) >= 0;
        copy_page(pools, __ldcg(l.src + pair), __ldcg(l.dst + pair));
      }
      __syncthreads();
      if (moves) look_up(stay);  // anew, in the copies
    }
    if (moves) {
      for (int from = stay;;) {
        for (int item = warp; item < 2 * c.heads; item += warps) {
          const int head = item >> 1;
          uint8_t *codes = item & 1 ? c.v : c.k, *exps = item & 1 ? c.v_exps : c.k_exps;
          for (int i = from, n = 0; i < to; ++n) {
            const int slot = (a.first + i) & (c.page - 1), m = min(c.page - slot, to - i), page = s_dst[n];
            const int *src = s_src + (i - from);
            i += m;
            bool in = (unsigned)page < (unsigned)c.pages;
            for (int r = lane; r < m; r += 32) in &= src[r] >= 0;
            if (!__all_sync(~0u, in)) {  // a page outside the pool: nothing moves into this one
              if (lane == 0) atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
              continue;
            }
            const size_t ph = (size_t)page * c.heads + head;
            const int was = exps[ph];
            uint4 x[STEPS];
            int e[STEPS];
            auto load = [&](int r0) {
#pragma unroll
              for (int j = 0; j < STEPS; ++j) {
                const int r = r0 + j * RPS + lane / LPR;
                x[j] = make_uint4(0, 0, 0, 0), e[j] = 0;
                if (r < m) {
                  const int at = src[r];
                  const size_t row = ((size_t)(at >> c.page_log2) * c.heads + head);
                  e[j] = at >> c.page_log2 == page ? was : exps[row];
                  x[j] = *reinterpret_cast<const uint4 *>(codes + ((row << c.page_log2) + (at & (c.page - 1))) * D +
                                                          lane % LPR * 16);
                }
              }
            };
            // more rows than registers hold, behind positions that stay: where the page's
            // scale is no less than those of all rows, it holds them
            bool fits = false;
            if (m > HELD && slot && was >= 7) {
              int most = 0;
              for (int r = lane; r < m; r += 32) {
                const int at = src[r] >> c.page_log2;
                if (at != page) most = max(most, (int)exps[(size_t)at * c.heads + head]);
              }
              fits = __all_sync(~0u, most <= was);
            }
            int need = 0;
            for (int r0 = 0; r0 < m && !fits; r0 += HELD) {
              load(r0);
#pragma unroll
              for (int j = 0; j < STEPS; ++j) {
                if (r0 + j * RPS >= m) break;
                uint32_t top = top_code(top_code(top_code(top_code(0, x[j].x), x[j].y), x[j].z), x[j].w);
                top = __vmaxu4(top, top >> 16);
                top = __vmaxu4(top, top >> 8) & 255u;
                need = max(need, needed_exp(top, e[j]));
              }
            }
            need = min(max(__reduce_max_sync(~0u, need), 7), 247);
            const int now = fits ? was : slot ? max(need, was) : need;
            uint8_t *tile = codes + (ph << c.page_log2) * D;
            if (slot && now > was) {  // earlier positions under the larger scale
              const float f = pow2i(max(was - now, -126));
              for (int j = lane; j < slot * D / 16; j += 32) {
                uint4 *w = reinterpret_cast<uint4 *>(tile) + j;
                *w = scaled(*w, f);
              }
            }
            for (int r0 = 0; r0 < m; r0 += HELD) {
              if (m > HELD) load(r0);
              __syncwarp();  // read, before any lane writes
#pragma unroll
              for (int j = 0; j < STEPS; ++j) {
                const int r = r0 + j * RPS + lane / LPR;
                if (r < m) {
                  if (e[j] != now) x[j] = scaled(x[j], step_by(e[j] - now));
                  *reinterpret_cast<uint4 *>(tile + (size_t)(slot + r) * D + lane % LPR * 16) = x[j];
                }
              }
              __syncwarp();
            }
            if (lane == 0) exps[ph] = (uint8_t)now;
          }
        }
        if (to == a.keep) break;
        __syncthreads();  // the places have been read
        from = to;
        to = look_up(from);
      }
    }
    __syncthreads();  // the length, the table and the places have been read, by every thread
    const int now = a.first + a.keep, held = (now + c.page - 1) >> c.page_log2;
    for (int j = held + tid; j < (a.first + a.n + c.page - 1) >> c.page_log2; j += threads) {
      const int page = table[j];
      table[j] = -1;
      if ((unsigned)page < (unsigned)c.pages) drop_page(c, page);
      else atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
    }
    if (tid == 0) c.lens[s] = now;
  }
  if (!planned) grid_wait();
}

}  // namespace

// Sequences that a CTA looks through: one, or up to 32 of a large table, most of which
// have no rows.
static int sequences_per_cta(const KvView &c, int sms) { return std::min(std::max(c.seqs / (sms * 16), 1), 32); }

cudaError_t launch_kv_tree_mask(const KvView &c, const int32_t *parents, const int32_t *starts, int rows, int32_t *mask,
                                int words, int32_t *positions, int sms, cudaStream_t stream) {
  const int per = sequences_per_cta(c, sms);
  tree_mask_kernel<<<(c.seqs + per - 1) / per, kMaskThreads, 0, stream>>>(c, parents, starts, rows, mask, words, positions,
                                                                         per);
  return cudaGetLastError();
}

cudaError_t launch_kv_accept(const KvView &c, const KvLists &l, const KvPools &pools, const int32_t *starts,
                             const int32_t *counts, const int32_t *accepted, int rows, int sms, cudaStream_t stream) {
  const int warps = accepted ? std::min(2 * c.heads, kAcceptWarps) : 4, per = sequences_per_cta(c, sms);
  const int ctas = (c.seqs + per - 1) / per;
  cudaError_t e = launch_after(accept_plan_kernel, dim3(ctas), kAcceptPlan, 0, stream, false, c, l, starts, counts, accepted,
                               rows, per);
  if (e != cudaSuccess) return e;
  auto run = [&](auto *kernel) {
    return launch_after(kernel, dim3(ctas), 32 * warps, 0, stream, true, c, l, pools, starts, counts, accepted, rows, per);
  };
  return c.dim == 64 ? run(accept_kernel<64>) : run(accept_kernel<128>);
}

}  // namespace mqa
