// Drafted tokens over the paged 8-bit cache (include/mqakv.h): the masks and
// positions of a tree of drafts (mqa_kv_tree_mask), and taking over the accepted
// ones (mqa_kv_accept).
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
// down, each written once.
constexpr int kMaskThreads = 128;
constexpr int kMaskHeld = 1024;  // parents of a sequence kept in shared memory

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const KvView c, const int32_t *__restrict__ parents,
                                                                 const int32_t *__restrict__ starts, int rows,
                                                                 int32_t *__restrict__ mask, int words,
                                                                 int32_t *__restrict__ positions) {
  __shared__ int s_parent[kMaskHeld];
  const int s = blockIdx.x;
  const Rows r = rows_of(starts, s, rows);
  if (r.n == 0) return;
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
  const int len = __ldg(c.lens + s), keep = __ldg(counts + s);
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
// Whether entry i of a sequence's list is where it may be: ascending rows.
__device__ __forceinline__ bool entry_ok(const int32_t *list, int i, int n) {
  const int at = __ldg(list + i);
  return at < n && at > (i ? __ldg(list + i - 1) : -1);
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
// Four codes times f.
__device__ __forceinline__ uint32_t scaled(uint32_t w, float f) {
  return to_e4m3x4(from_e4m3(w & 255u) * f, from_e4m3(w >> 8 & 255u) * f, from_e4m3(w >> 16 & 255u) * f,
                   from_e4m3(w >> 24) * f);
}
// 2^d, of as much of d as matters for a product with a code.
__device__ __forceinline__ float step_by(int d) { return pow2i(min(max(d, -60), 60)); }

// Moves the kept rows behind each other: a CTA has a head's keys or values of a few
// sequences, and goes over the pages that rows move into, in order.  A page's rows
// come from its own places or later ones, so that a page is read (into registers)
// before anything of it is overwritten, and what later pages need lies in pages
// that have not been written yet.
constexpr int kMoveThreads = 128;
template <int D>
__global__ void __launch_bounds__(kMoveThreads) accept_move_kernel(const KvView c, const int32_t *__restrict__ starts,
                                                                   const int32_t *__restrict__ counts,
                                                                   const int32_t *__restrict__ accepted, int rows,
                                                                   int per) {
  constexpr int LPR = D / 16, RPS = kMoveThreads / LPR, STEPS = 128 / RPS;  // lanes per row, rows per step, steps
  __shared__ int s_need[kMoveThreads / 32];
  grid_dependents();
  const int tid = threadIdx.x, head = blockIdx.y;
  uint8_t *codes = blockIdx.z ? c.v : c.k, *exps = blockIdx.z ? c.v_exps : c.k_exps;
  for (int s = blockIdx.x * per; s < min(c.seqs, (int)(blockIdx.x + 1) * per); ++s) {
    const Asked a = asked_of(c, starts, counts, s, rows, nullptr);
    if (a.keep <= 0) continue;
    const int32_t *list = accepted + a.r0, *table = c.table + (size_t)s * c.max_pages;
    bool ok = true;
    int stay = 0;  // rows that are where they belong: the first ones
    for (int i = tid; i < a.keep; i += kMoveThreads) {
      ok &= entry_ok(list, i, a.n);
      stay += __ldg(list + i) == i;
    }
    if (__syncthreads_or(!ok)) continue;
    stay = __reduce_add_sync(~0u, stay);
    if ((tid & 31) == 0) s_need[tid >> 5] = stay;
    __syncthreads();
    stay = 0;
#pragma unroll
    for (int w = 0; w < kMoveThreads / 32; ++w) stay += s_need[w];
    for (int i = stay; i < a.keep;) {
      const int to = a.first + i, slot = to & (c.page - 1), m = min(c.page - slot, a.keep - i);
      const int to_page = __ldg(table + (to >> c.page_log2));
      bool in = (unsigned)to_page < (unsigned)c.pages;
      uint4 x[STEPS];
      int e[STEPS];
      int need = 0;
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        const int row = j * RPS + tid / LPR;
        x[j] = make_uint4(0, 0, 0, 0);
        e[j] = 0;
        if (row < m) {
          const int from = a.first + __ldg(list + i + row), page = __ldg(table + (from >> c.page_log2));
          if ((unsigned)page < (unsigned)c.pages) {
            const size_t ph = (size_t)page * c.heads + head;
            e[j] = exps[ph];
            x[j] = *reinterpret_cast<const uint4 *>(codes + ((ph << c.page_log2) + (from & (c.page - 1))) * D +
                                                    tid % LPR * 16);
            uint32_t top = top_code(top_code(top_code(top_code(0, x[j].x), x[j].y), x[j].z), x[j].w);
            top = __vmaxu4(top, top >> 16);
            top = __vmaxu4(top, top >> 8) & 255u;
            need = max(need, needed_exp(top, e[j]));
          } else {
            in = false;
          }
        }
      }
      need = __reduce_max_sync(~0u, need);
      __syncthreads();  // what s_need held has been read
      if ((tid & 31) == 0) s_need[tid >> 5] = need;
      const size_t ph = (size_t)max(to_page, 0) * c.heads + head;
      const int was = slot && (unsigned)to_page < (unsigned)c.pages ? exps[ph] : 0;
      if (__syncthreads_or(!in)) {  // a page outside the pool: nothing moves into this one
        if (tid == 0) atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
        i += m;
        continue;
      }
#pragma unroll
      for (int w = 0; w < kMoveThreads / 32; ++w) need = max(need, s_need[w]);
      const int now = max(min(max(need, 7), 247), was);
      uint8_t *tile = codes + (ph << c.page_log2) * D;
      if (slot && now > was) {  // earlier positions under the larger scale
        const float f = pow2i(max(was - now, -126));
        for (int j = tid; j < slot * D / 4; j += kMoveThreads) {
          uint32_t *w = reinterpret_cast<uint32_t *>(tile) + j;
          *w = scaled(*w, f);
        }
      }
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        const int row = j * RPS + tid / LPR;
        if (row < m) {
          const float f = step_by(e[j] - now);
          *reinterpret_cast<uint4 *>(tile + (size_t)(slot + row) * D + tid % LPR * 16) =
              make_uint4(scaled(x[j].x, f), scaled(x[j].y, f), scaled(x[j].z, f), scaled(x[j].w, f));
        }
      }
      if (tid == 0) exps[ph] = (uint8_t)now;
      i += m;
    }
  }
  grid_wait();
}

// Lengths and pages: a warp per sequence.
__global__ void __launch_bounds__(256) accept_trim_kernel(const KvView c, const int32_t *__restrict__ starts,
                                                          const int32_t *__restrict__ counts,
                                                          const int32_t *__restrict__ accepted, int rows) {
  grid_wait();
  const int s = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (s >= c.seqs) return;
  const Asked a = asked_of(c, starts, counts, s, rows, lane == 0 ? c.status : nullptr);
  if (a.keep < 0) return;
  bool ok = true;
  if (accepted)
    for (int i = lane; i < a.keep; i += 32) ok &= entry_ok(accepted + a.r0, i, a.n);
  if (!__all_sync(~0u, ok)) {
    if (lane == 0) atomicOr(c.status, MQA_KV_DEV_BAD_LIST);
    return;
  }
  const int now = a.first + a.keep, held = (now + c.page - 1) >> c.page_log2;
  int32_t *table = c.table + (size_t)s * c.max_pages;
  for (int j = held + lane; j < (a.first + a.n + c.page - 1) >> c.page_log2; j += 32) {
    const int page = table[j];
    table[j] = -1;
    if ((unsigned)page >= (unsigned)c.pages) {
      atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
    } else if (atomicSub(c.refs + page, 1) <= 0) {  // not in use: the count stays
      atomicAdd(c.refs + page, 1);
      atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
    }
  }
  if (lane == 0) c.lens[s] = now;
}

}  // namespace

cudaError_t launch_kv_tree_mask(const KvView &c, const int32_t *parents, const int32_t *starts, int rows, int32_t *mask,
                                int words, int32_t *positions, cudaStream_t stream) {
  tree_mask_kernel<<<c.seqs, kMaskThreads, 0, stream>>>(c, parents, starts, rows, mask, words, positions);
  return cudaGetLastError();
}

cudaError_t launch_kv_accept(const KvView &c, const int32_t *starts, const int32_t *counts, const int32_t *accepted,
                             int rows, int sms, cudaStream_t stream) {
  if (accepted) {
    const long long ctas = (long long)c.seqs * c.heads * 2;
    const int per = (int)std::min(std::max(ctas / (sms * 8LL), 1LL), 32LL);
    const dim3 grid((c.seqs + per - 1) / per, c.heads, 2);
    const cudaError_t e =
        c.dim == 64 ? launch_after(accept_move_kernel<64>, grid, kMoveThreads, 0, stream, false, c, starts, counts,
                                   accepted, rows, per)
                    : launch_after(accept_move_kernel<128>, grid, kMoveThreads, 0, stream, false, c, starts, counts,
                                   accepted, rows, per);
    if (e != cudaSuccess) return e;
  }
  return launch_after(accept_trim_kernel, dim3((c.seqs + 7) / 8), 256, 0, stream, accepted != nullptr, c, starts, counts,
                      accepted, rows);
}

}  // namespace mqa
