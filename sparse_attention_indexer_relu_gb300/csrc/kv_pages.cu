// Page operations of the paged key/value cache (include/mqakv.h): reserving,
// forking, freeing, compacting and copying.
//
// Tables and counts are a few words per page, so an operation is planned by
// one CTA (or one short pass over the counts) on the device, without the host
// learning anything, and then carried out by a grid that copies the listed
// pages.  Bound by the copied bytes (each page read once and written once);
// every copying thread keeps two 16-byte loads in flight (compacting 16K pages of
// 64 positions of 8 heads of 128, 527 MB moved: 183 us, 5.8 TB/s; copying 1,000
// scattered pages of 128 KB: 49 us, 5.4 TB/s, 64 of them: 6.1 us, latency).
// Reserving a position for each of 64 sequences takes 3.4 us, of 4,096 sequences
// 45 us: one CTA's work.
//
// Order.  Free pages are taken lowest first and lists are worked in order, so
// results do not depend on timing; refcounts change by integer atomics, whose
// sums do not depend on order either.
#include "kv_pages.cuh"

namespace mqa {

namespace {

constexpr int kPlan = 1024;  // threads of a planning CTA
constexpr int kCopy = 256;   // threads of a copying CTA

__device__ __forceinline__ int pages_of(const KvView &c, int len) { return (len + c.page - 1) >> c.page_log2; }
// A length the table can hold; false (and 0) otherwise.
__device__ __forceinline__ bool length_ok(const KvView &c, int len) {
  return len >= 0 && len <= (c.max_pages << c.page_log2);
}

// Copy unit u of the (pair, 8 KB piece) line; CTA-wide.
constexpr int kPiece = 8192;
__device__ void copy_line(const KvPools &p, const int32_t *src, const int32_t *dst, int count) {
  int pieces = 0;
  for (int i = 0; i < p.n; ++i) pieces += (int)((p.bytes[i] + kPiece - 1) / kPiece);
  const long long total = (long long)count * pieces;
  for (long long u = blockIdx.x; u < total; u += gridDim.x) {
    const int pair = (int)(u / pieces);
    int piece = (int)(u - (long long)pair * pieces), i = 0;
    while (true) {
      const int n = (int)((p.bytes[i] + kPiece - 1) / kPiece);
      if (piece < n) break;
      piece -= n;
      ++i;
    }
    const unsigned long long off = (unsigned long long)piece * kPiece, size = p.bytes[i];
    const int n = (int)min((unsigned long long)kPiece, size - off);
    const uint8_t *s = p.data[i] + (unsigned long long)src[pair] * size + off;
    uint8_t *d = p.data[i] + (unsigned long long)dst[pair] * size + off;
    if (((reinterpret_cast<uintptr_t>(s) | reinterpret_cast<uintptr_t>(d) | n) & 15) == 0) {
      const uint4 *s4 = reinterpret_cast<const uint4 *>(s);
      uint4 *d4 = reinterpret_cast<uint4 *>(d);
      const int m = n >> 4;  // at most 512: two per thread
      uint4 a, b;
      const int x = threadIdx.x, y = threadIdx.x + kCopy;
      if (x < m) a = s4[x];
      if (y < m) b = s4[y];
      if (x < m) d4[x] = a;
      if (y < m) d4[y] = b;
    } else {
      for (int x = threadIdx.x; x < n; x += kCopy) d[x] = s[x];
    }
  }
}

// ------------------------------------------------------------------ reserve
__global__ void __launch_bounds__(kPlan) reserve_kernel(const KvView c, const KvLists l,
                                                       const int32_t *__restrict__ counts) {
  __shared__ int sums[32];
  __shared__ long long wide_sums[32];
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  // The same in every thread.  In 64 bits, a step's sum as well: a sequence may ask
  // for 2^26 pages, and 32 such requests sum to 2^31.
  long long total = 0;
  for (int base = 0; base < c.seqs; base += kPlan) {
    const int s = base + threadIdx.x;
    long long need = 0;
    if (s < c.seqs) {
      const int len = c.lens[s], add = counts[s];
      const long long now = (long long)len + add;
      if (add < 0) atomicOr(&bad, MQA_KV_DEV_BAD_LIST);
      else if (!length_ok(c, len) || now > (long long)(c.max_pages << c.page_log2)) atomicOr(&bad, MQA_KV_DEV_BAD_LENGTH);
      else need = pages_of(c, (int)now) - pages_of(c, len);
    }
    long long excl;
    const long long sum = block_scan(need, excl, wide_sums);
    if (s < c.seqs) l.seq_a[s] = (int)min(total + excl, (long long)INT32_MAX);
    total += sum;
  }
  __syncthreads();
  if (bad == 0 && total > c.pages && threadIdx.x == 0) bad = MQA_KV_DEV_OUT_OF_PAGES;
  __syncthreads();
  if (bad == 0 && lowest_free<kPlan>(c, (int)total, l.dst, sums) < total && threadIdx.x == 0) bad = MQA_KV_DEV_OUT_OF_PAGES;
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0) atomicOr(c.status, bad);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int s = warp; s < c.seqs; s += kPlan / 32) {
    const int len = c.lens[s], add = counts[s];
    if (add == 0) continue;
    const int have = pages_of(c, len), need = pages_of(c, len + add) - have, first = l.seq_a[s];
    for (int j = lane; j < need; j += 32) {
      const int page = l.dst[first + j];
      c.table[(size_t)s * c.max_pages + have + j] = page;
      c.refs[page] = 1;
    }
    __syncwarp();
    if (lane == 0) c.lens[s] = len + add;
  }
}

// ------------------------------------------------------------------ fork
// Plan: seq_b marks children (by sequence) and then holds the parents' lengths
// (by list entry); seq_a[i] is the rank of the new page for the parent's partial
// one among all new pages (-1: none).
__global__ void __launch_bounds__(kPlan) fork_plan_kernel(const KvView c, const KvLists l,
                                                         const int32_t *__restrict__ parents,
                                                         const int32_t *__restrict__ children, int n) {
  __shared__ int sums[32];
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  for (int s = threadIdx.x; s < c.seqs; s += kPlan) l.seq_b[s] = 0;
  __syncthreads();
  int total = 0;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + threadIdx.x;
    int need = 0, src = -1, len = 0;
    if (i < n) {
      const int a = parents[i], b = children[i];
      if ((unsigned)a >= (unsigned)c.seqs || (unsigned)b >= (unsigned)c.seqs) {
        atomicOr(&bad, MQA_KV_DEV_BAD_LIST);
      } else {
        len = c.lens[a];
        if (c.lens[b] != 0 || atomicExch(l.seq_b + b, 1) != 0) atomicOr(&bad, MQA_KV_DEV_BAD_LIST);
        if (!length_ok(c, len)) {
          atomicOr(&bad, MQA_KV_DEV_BAD_LENGTH);
        } else if (len & (c.page - 1)) {
          src = c.table[(size_t)a * c.max_pages + (len >> c.page_log2)];
          if ((unsigned)src >= (unsigned)c.pages) atomicOr(&bad, MQA_KV_DEV_BAD_INDEX);
          else need = 1;
        }
      }
    }
    int excl;
    const int sum = block_scan(need, excl, sums);
    if (i < n) {
      l.seq_a[i] = need ? total + excl : -1;  // rank of its new page
      if (need && total + excl < c.pages) l.src[total + excl] = src;
    }
    total += sum;
  }
  __syncthreads();
  if (bad == 0 && lowest_free<kPlan>(c, total, l.dst, sums) < total && threadIdx.x == 0) bad = MQA_KV_DEV_OUT_OF_PAGES;
  __syncthreads();
  if (threadIdx.x == 0) {
    l.head[kKvOk] = bad == 0;
    l.head[kKvCount] = bad == 0 ? total : 0;
    if (bad) atomicOr(c.status, bad);
  }
  if (bad) return;
  for (int i = threadIdx.x; i < n; i += kPlan) l.seq_b[i] = c.lens[parents[i]];
  for (int i = threadIdx.x; i < total; i += kPlan) c.refs[l.dst[i]] = 1;
}

__global__ void __launch_bounds__(kCopy) fork_kernel(const KvView c, const KvLists l, const KvPools pools,
                                                    const int32_t *__restrict__ parents,
                                                    const int32_t *__restrict__ children, int n) {
  if (!l.head[kKvOk]) return;
  copy_line(pools, l.src, l.dst, l.head[kKvCount]);
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int len = l.seq_b[i], full = len >> c.page_log2;
    const int32_t *from = c.table + (size_t)parents[i] * c.max_pages;
    int32_t *to = c.table + (size_t)children[i] * c.max_pages;
    for (int j = threadIdx.x; j < full; j += kCopy) {
      const int page = from[j];
      to[j] = page;
      if ((unsigned)page < (unsigned)c.pages) atomicAdd(c.refs + page, 1);
      else atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
    }
    if (threadIdx.x == 0) {
      if (l.seq_a[i] >= 0) to[full] = l.dst[l.seq_a[i]];
      c.lens[children[i]] = len;
    }
  }
}

// ------------------------------------------------------------------ free
__global__ void __launch_bounds__(kCopy) free_kernel(const KvView c, const int32_t *__restrict__ seqs) {
  __shared__ int s_len;
  const int s = seqs[blockIdx.x];
  if ((unsigned)s >= (unsigned)c.seqs) {
    if (threadIdx.x == 0) atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
    return;
  }
  if (threadIdx.x == 0) s_len = atomicExch(c.lens + s, 0);  // a second listing finds it empty
  __syncthreads();
  int len = s_len;
  if (!length_ok(c, len)) {
    if (threadIdx.x == 0) atomicOr(c.status, MQA_KV_DEV_BAD_LENGTH);
    len = min(max(len, 0), c.max_pages << c.page_log2);
  }
  int32_t *row = c.table + (size_t)s * c.max_pages;
  for (int j = threadIdx.x; j < pages_of(c, len); j += kCopy) {
    const int page = row[j];
    row[j] = -1;
    if ((unsigned)page < (unsigned)c.pages) drop_page(c, page);
    else atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
  }
}

// ------------------------------------------------------------------ compact
// Pass 1: used pages per block of kCompactPages.
__global__ void __launch_bounds__(kPlan) compact_count_kernel(const KvView c, const KvLists l) {
  __shared__ int sums[32];
  const int at = blockIdx.x * kCompactPages + threadIdx.x * 4;
  int n = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) n += at + i < c.pages && c.refs[at + i] > 0;
  int excl;
  const int total = block_scan(n, excl, sums);
  if (threadIdx.x == 0) l.sums[blockIdx.x] = total;
}

// Pass 2: ranks.  The i-th free page below `live` (dst[i]) is paired with the
// i-th used page at or above it (src[i], rank[page] = i).
__global__ void __launch_bounds__(kPlan) compact_rank_kernel(const KvView c, const KvLists l) {
  __shared__ int sums[32];
  int live = 0, before = 0, excl;
  for (int base = 0; base < (int)gridDim.x; base += kPlan) {
    const int b = base + threadIdx.x;
    const int n = b < (int)gridDim.x ? l.sums[b] : 0;
    live += block_scan(n, excl, sums);
    before += block_scan(b < (int)blockIdx.x ? n : 0, excl, sums);
  }
  // used pages below `live`: whole blocks, then the block that holds the border
  const int edge = live / kCompactPages;
  int low = 0;
  for (int base = 0; base < edge; base += kPlan) {
    const int b = base + threadIdx.x;
    low += block_scan(b < edge ? l.sums[b] : 0, excl, sums);
  }
  {
    const int at = edge * kCompactPages + threadIdx.x * 4;
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) n += at + i < live && c.refs[at + i] > 0;
    low += block_scan(n, excl, sums);
  }
  const int at = blockIdx.x * kCompactPages + threadIdx.x * 4;
  int used[4], n = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    used[i] = at + i < c.pages && c.refs[at + i] > 0;
    n += used[i];
  }
  block_scan(n, excl, sums);
  int r = before + excl;  // used pages before this one
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int page = at + i;
    if (page >= c.pages) break;
    if (page < live) {
      if (!used[i]) l.dst[page - r] = page;
    } else if (used[i]) {
      l.src[r - low] = page;
      l.rank[page] = r - low;
    }
    r += used[i];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    l.head[kKvCount] = live - low;
    l.head[kKvLive] = live;
  }
}

// Pass 3: contents, counts and tables.
__global__ void __launch_bounds__(kCopy) compact_move_kernel(const KvView c, const KvLists l, const KvPools pools) {
  const int count = l.head[kKvCount], live = l.head[kKvLive];
  if (count == 0) return;
  const int stride = gridDim.x * kCopy, id = blockIdx.x * kCopy + threadIdx.x;
  for (int i = id; i < count; i += stride) {
    c.refs[l.dst[i]] = c.refs[l.src[i]];
    c.refs[l.src[i]] = 0;
  }
  // one warp per sequence in turn
  const int warps = stride / 32, lane = threadIdx.x & 31;
  for (int s = id / 32; s < c.seqs; s += warps) {
    const int len = c.lens[s];
    const int n = length_ok(c, len) ? pages_of(c, len) : 0;
    if (!length_ok(c, len) && lane == 0) atomicOr(c.status, MQA_KV_DEV_BAD_LENGTH);
    int32_t *row = c.table + (size_t)s * c.max_pages;
    for (int j = lane; j < n; j += 32) {
      const int page = row[j];
      if ((unsigned)page >= (unsigned)c.pages) atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
      else if (page >= live) {
        const int r = l.rank[page];
        // a page in a table that no count names was not ranked
        if ((unsigned)r < (unsigned)count && l.src[r] == page) row[j] = l.dst[r];
        else atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
      }
    }
  }
  copy_line(pools, l.src, l.dst, count);
}

// ------------------------------------------------------------------ copy
__global__ void __launch_bounds__(kPlan) copy_plan_kernel(const KvView c, const KvLists l,
                                                         const int32_t *__restrict__ src,
                                                         const int32_t *__restrict__ dst, int n) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int a = src[i], b = dst[i];
    if ((unsigned)a >= (unsigned)c.pages || (unsigned)b >= (unsigned)c.pages) bad = 1;
    else l.rank[a] = 0, l.rank[b] = 0;
  }
  __syncthreads();
  if (!bad) {
    for (int i = threadIdx.x; i < n; i += kPlan)
      if (atomicExch(l.rank + dst[i], 1) != 0) bad = 1;
  }
  __syncthreads();
  if (!bad) {
    for (int i = threadIdx.x; i < n; i += kPlan)
      if (l.rank[src[i]] != 0) bad = 1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    l.head[kKvOk] = !bad;
    if (bad) atomicOr(c.status, MQA_KV_DEV_BAD_LIST);
  }
}

__global__ void __launch_bounds__(kCopy) copy_kernel(const KvLists l, const KvPools pools,
                                                    const int32_t *__restrict__ src,
                                                    const int32_t *__restrict__ dst, int n) {
  if (l.head[kKvOk]) copy_line(pools, src, dst, n);
}

constexpr int kCopyCtasPerSm = 8;

}  // namespace

cudaError_t launch_kv_reserve(const KvView &c, const KvLists &l, const int32_t *counts, cudaStream_t stream) {
  reserve_kernel<<<1, kPlan, 0, stream>>>(c, l, counts);
  return cudaGetLastError();
}

cudaError_t launch_kv_fork(const KvView &c, const KvLists &l, const KvPools &pools, const int32_t *parents,
                           const int32_t *children, int n, int sms, cudaStream_t stream) {
  fork_plan_kernel<<<1, kPlan, 0, stream>>>(c, l, parents, children, n);
  fork_kernel<<<sms * kCopyCtasPerSm, kCopy, 0, stream>>>(c, l, pools, parents, children, n);
  return cudaGetLastError();
}

cudaError_t launch_kv_free(const KvView &c, const int32_t *seqs, int n, cudaStream_t stream) {
  free_kernel<<<n, kCopy, 0, stream>>>(c, seqs);
  return cudaGetLastError();
}

cudaError_t launch_kv_compact(const KvView &c, const KvLists &l, const KvPools &pools, int sms, cudaStream_t stream) {
  const int blocks = (c.pages + kCompactPages - 1) / kCompactPages;
  compact_count_kernel<<<blocks, kPlan, 0, stream>>>(c, l);
  compact_rank_kernel<<<blocks, kPlan, 0, stream>>>(c, l);
  compact_move_kernel<<<sms * kCopyCtasPerSm, kCopy, 0, stream>>>(c, l, pools);
  return cudaGetLastError();
}

cudaError_t launch_kv_copy(const KvView &c, const KvLists &l, const KvPools &pools, const int32_t *src,
                           const int32_t *dst, int n, int sms, cudaStream_t stream) {
  copy_plan_kernel<<<1, kPlan, 0, stream>>>(c, l, src, dst, n);
  copy_kernel<<<sms * kCopyCtasPerSm, kCopy, 0, stream>>>(l, pools, src, dst, n);
  return cudaGetLastError();
}

}  // namespace mqa
