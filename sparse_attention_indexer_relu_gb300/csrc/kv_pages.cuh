// Device helpers of the paged key/value cache's page operations.
#pragma once
#include "kv_internal.h"

namespace mqa {

// Exclusive scan of one value per thread over the CTA; returns the total.
template <typename T>
__device__ T block_scan(T v, T &excl, T *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    T x = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    if (lane < warps) warp_sums[lane] = x;
  }
  __syncthreads();
  excl = incl - v + (warp ? warp_sums[warp - 1] : 0);
  return warp_sums[warps - 1];
}

// The lowest `need` free pages, ascending, into list; returns how many there
// are (at most need).  One CTA of THREADS; stops as soon as it has them.  A step looks
// at 16 counts per thread, with the next step's on their way, and costs one vote where
// none is free (1,024 threads, a page behind 2M used ones: 125 us).
template <int THREADS>
__device__ int lowest_free(const KvView &c, int need, int32_t *list, int *warp_sums) {
  constexpr int kRun = 16, kStep = THREADS * kRun;
  const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5) * 32 * kRun + lane;
  int found = 0, refs[kRun];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int page = base + first + 32 * i;
      refs[i] = page < c.pages ? c.refs[page] : 1;
    }
  };
  load(0);
  for (int base = 0; base < c.pages && found < need; base += kStep) {
    uint32_t free[kRun];
    int n = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      free[i] = __ballot_sync(~0u, refs[i] == 0);
      n += __popc(free[i]);
    }
    load(base + kStep);
    if (!__syncthreads_or(n)) continue;
    int excl;
    const int total = block_scan(lane == 0 ? n : 0, excl, warp_sums);
    int at = found + __shfl_sync(~0u, excl, 0);  // free pages before the warp's
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int mine = at + __popc(free[i] & ((1u << lane) - 1));
      if ((free[i] >> lane & 1) && mine < need) list[mine] = base + first + 32 * i;
      at += __popc(free[i]);
    }
    found += total;
  }
  __syncthreads();
  return min(found, need);
}

// A page's count drops by one; one that is not in use keeps its count.
__device__ __forceinline__ void drop_page(const KvView &c, int page) {
  if (atomicSub(c.refs + page, 1) > 0) return;
  atomicAdd(c.refs + page, 1);
  atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
}

}  // namespace mqa
