// Appending to the paged 8-bit cache (include/mqakv.h, mqa_kv_append).
//
// For a page, a head and keys or values, with new magnitudes up to a:
//     e = max(e_old if the page held earlier positions, min e: a <= 448 2^(e - 127))
//     code = RNE_e4m3(x 2^(127 - e));  earlier codes: RNE_e4m3(E(code) 2^(e_old - e))
// Scales are powers of two, so every product is exact and the only rounding is
// the one to e4m3 (half a step: 2^-4 of the value).
//
// At least rows * heads * dim * (input bytes + 1) bytes move, twice (K and V); what
// bounds it is the chain bounds -> length -> page -> rows of each CTA, four CTAs
// to an SM (9.3K bf16 rows of 8 heads of 128 to 4 sequences: 17 us, 3.3 TB/s, in a
// graph; one row for each of 128 sequences: 4.6 us in a graph.  Calls by
// themselves, with new inputs each time, take 24 and 17 to 19 us).  A CTA looks at consecutive rows,
// finds those that begin a page's new positions (its leaders) and writes each
// leader's tile: its rows are loaded into registers at once, their largest
// magnitude found, and the codes written from there.  A tile of more rows than
// that (by a warp, or by a small CTA) is read twice.
#include "kv_ptx.cuh"

#include <cuda_fp8.h>
#include <type_traits>

namespace mqa {

namespace {

constexpr int kMaxRows = 128;    // rows a CTA looks at
constexpr int kStarts = 1024;    // row bounds kept in shared memory

__device__ __forceinline__ float from_e4m3(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
  return __half2float(__half(h));
}

// Least exponent byte whose scale holds amax within 448 (amax finite, >= 0).
__device__ __forceinline__ int needed_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127;  // amax = f 2^e, f in [1, 2); 448 = 1.75 2^8
  const int n = e - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0) + 127;
  return min(max(n, 7), 247);
}

// 8 elements of a row: 16 bytes (bf16, fp16) or 32.
template <int TYPE>
struct Eight {
  uint4 w[TYPE == MQA_KV_FP32 ? 2 : 1];
  __device__ __forceinline__ void load(const void *base, size_t at) {
    if (TYPE == MQA_KV_FP32) {
      const uint4 *s = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(base) + at);
      w[0] = __ldg(s);
      w[TYPE == MQA_KV_FP32 ? 1 : 0] = __ldg(s + 1);
    } else {
      w[0] = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + at));
    }
  }
  __device__ __forceinline__ void clear() {
    w[0] = make_uint4(0, 0, 0, 0);
    if (TYPE == MQA_KV_FP32) w[TYPE == MQA_KV_FP32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
  }
  // The larger of m and the elements' magnitudes, as bit patterns (ordered like
  // the values; two at a time for 16-bit types).
  __device__ __forceinline__ uint32_t top(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < (TYPE == MQA_KV_FP32 ? 2 : 1); ++i) {
      const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        m = TYPE == MQA_KV_FP32 ? max(m, v[k] & 0x7FFFFFFFu) : __vmaxu2(m, v[k] & 0x7FFF7FFFu);
    }
    return m;
  }
  // Its value; infinity or NaN where one of the elements is.
  static __device__ __forceinline__ float value(uint32_t m) {
    if (TYPE == MQA_KV_FP32) return __uint_as_float(m);
    m = max(m & 0xFFFFu, m >> 16);
    return TYPE == MQA_KV_BF16 ? __uint_as_float(m << 16) : half2_to_float2(m).x;
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (TYPE == MQA_KV_FP32) {
        const uint4 &v = w[TYPE == MQA_KV_FP32 ? i >> 1 : 0];
        f[2 * i] = __uint_as_float(i & 1 ? v.z : v.x), f[2 * i + 1] = __uint_as_float(i & 1 ? v.w : v.y);
      } else {
        const uint32_t v = i == 0 ? w[0].x : i == 1 ? w[0].y : i == 2 ? w[0].z : w[0].w;
        const float2 x = TYPE == MQA_KV_BF16 ? bf16x2_to_float2(v) : half2_to_float2(v);
        f[2 * i] = x.x, f[2 * i + 1] = x.y;
      }
    }
  }
};

// A page's new positions of one head: `count` rows from `row` on, behind the
// `held` positions of the page, by kThreads threads (a CTA, or a warp); up to
// STEPS times the rows they cover at once stay in registers.
template <int D, int TYPE, int kThreads, int STEPS>
__device__ __forceinline__ void write_tile(const KvView &c, const void *__restrict__ in, long long stride,
                                           uint8_t *codes, uint8_t *exps, int head, int row, int page, int held, int n,
                                           float *s_max) {
  constexpr int LPR = D / 8, RPS = kThreads / LPR;  // lanes per row, rows per step
  const int tid = threadIdx.x % kThreads, part = tid % LPR, step = tid / LPR;
  const size_t base = (size_t)row * stride + (size_t)head * D + part * 8;
  const size_t ph = (size_t)page * c.heads + head;
  const int was = held ? exps[ph] : 0;
  Eight<TYPE> x[STEPS];
  float amax = 0.f;
  const bool kept = n <= STEPS * RPS;
  for (int j0 = 0; j0 * RPS < n; j0 += STEPS) {
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      x[j].clear();
      if ((j0 + j) * RPS + step < n) x[j].load(in, base + (size_t)((j0 + j) * RPS + step) * stride);
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) m = x[j].top(m);
    float a = Eight<TYPE>::value(m);
    if (!(a <= 3.402823466e38f)) {  // infinities and NaN do not set the scale
      a = 0.f;
#pragma unroll 1
      for (int j = 0; j < STEPS; ++j) {
        if ((j0 + j) * RPS + step >= n) continue;
        Eight<TYPE> y;
        y.load(in, base + (size_t)((j0 + j) * RPS + step) * stride);
        float f[8];
        y.values(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) a = fabsf(f[k]) <= 3.402823466e38f ? fmaxf(a, fabsf(f[k])) : a;
      }
    }
    amax = fmaxf(amax, a);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if (kThreads > 32) {
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    __syncthreads();  // the old exponent has been read by all, too
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
  } else {
    __syncwarp();
  }
  const int e = max(needed_exp(amax), was);
  uint8_t *tile = codes + (ph << c.page_log2) * D;
  if (held && e > was) {  // earlier positions under the larger scale
    const float f = pow2i(max(was - e, -126));
    for (int j = tid; j < held * D / 4; j += kThreads) {
      uint32_t *w = reinterpret_cast<uint32_t *>(tile) + j;
      const uint32_t v = *w;
      *w = to_e4m3x4(from_e4m3(v & 255u) * f, from_e4m3(v >> 8 & 255u) * f, from_e4m3(v >> 16 & 255u) * f,
                     from_e4m3(v >> 24) * f);
    }
  }
  // 2^(127 - e); a page that was given a byte above 247 may need a subnormal
  const float up = e < 254 ? pow2i(127 - e) : __uint_as_float(0x00400000u >> (e - 254));
  for (int j0 = 0; j0 * RPS < n; j0 += STEPS) {
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const int at = (j0 + j) * RPS + step;
      if (at < n) {
        if (!kept) x[j].load(in, base + (size_t)at * stride);
        float f[8];
        x[j].values(f);
        uint2 o;
        o.x = to_e4m3x4(f[0] * up, f[1] * up, f[2] * up, f[3] * up);
        o.y = to_e4m3x4(f[4] * up, f[5] * up, f[6] * up, f[7] * up);
        *reinterpret_cast<uint2 *>(tile + (size_t)(held + at) * D + part * 8) = o;
      }
    }
  }
  if (tid == 0) exps[ph] = (uint8_t)e;
  if (kThreads > 32) __syncthreads();  // s_max is free again
}

template <int D, int TYPE, int kThreads, int STEPS>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvView c, const void *__restrict__ kin,
                                                            const void *__restrict__ vin, long long ks, long long vs,
                                                            const int32_t *__restrict__ starts, int rows, int per) {
  __shared__ int s_starts[kStarts + 1];
  __shared__ int s_row[kMaxRows], s_page[kMaxRows], s_slot[kMaxRows], s_count[kMaxRows];
  __shared__ int s_leaders[kMaxRows / 32];
  __shared__ float s_max[kThreads / 32];
  const int tid = threadIdx.x, head = blockIdx.y, values = blockIdx.z;
  const int row0 = blockIdx.x * per;
  const bool near = c.seqs <= kStarts;
  if (near) {
    for (int i = tid; i <= c.seqs; i += kThreads) s_starts[i] = __ldg(starts + i);
    __syncthreads();
  }
  auto start = [&](int s) { return near ? s_starts[s] : __ldg(starts + s); };
  int count = 0, page = -1, slot = 0;
  const int r = row0 + tid;
  if (tid < per && r < rows) {
    int lo = 0, hi = c.seqs;  // the last sequence that starts at or before the row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start(mid) <= r) lo = mid; else hi = mid;
    }
    const int a = max(start(lo), 0), b = min(start(lo + 1), rows);
    const long long pos = (long long)__ldg(c.lens + lo) - (b - a) + (r - a);  // position of the row
    if (r >= a && r < b && pos >= 0) {
      slot = (int)(pos & (c.page - 1));
      if (slot == 0 || r == a) {  // the first new position of its page
        const long long col = pos >> c.page_log2;
        if (col >= c.max_pages) {
          if (head == 0 && !values) atomicOr(c.status, MQA_KV_DEV_BAD_LENGTH);
        } else {
          page = __ldg(c.table + (size_t)lo * c.max_pages + col);
          if ((unsigned)page >= (unsigned)c.pages) {
            if (head == 0 && !values) atomicOr(c.status, MQA_KV_DEV_BAD_INDEX);
          } else {
            count = min(c.page - slot, b - r);
          }
        }
      }
    }
  }
  // the leaders, in order
  const uint32_t mine = __ballot_sync(~0u, count > 0);
  if ((tid & 31) == 0 && tid < kMaxRows) s_leaders[tid >> 5] = __popc(mine);
  __syncthreads();
  int leaders = 0, before = 0;
#pragma unroll
  for (int w = 0; w < (kThreads < kMaxRows ? kThreads : kMaxRows) / 32; ++w) {
    if (w < tid >> 5) before += s_leaders[w];
    leaders += s_leaders[w];
  }
  if (count > 0) {
    const int at = before + __popc(mine & lanemask_lt());
    s_row[at] = r, s_page[at] = page, s_slot[at] = slot, s_count[at] = count;
  }
  __syncthreads();
  const void *in = values ? vin : kin;
  const long long stride = values ? vs : ks;
  uint8_t *codes = values ? c.v : c.k;
  uint8_t *exps = values ? c.v_exps : c.k_exps;
  auto tile = [&](int i, auto group) {
    write_tile<D, TYPE, decltype(group)::value, STEPS>(c, in, stride, codes, exps, head, s_row[i], s_page[i], s_slot[i],
                                                       s_count[i], s_max);
  };
  // Few tiles: one after another by the whole CTA.  Many (single tokens of many
  // sequences): one per warp (2,048 tokens of 8 heads: 15.7 us, against 123).
  if (kThreads > 128 && leaders > 2) {
    for (int i = tid >> 5; i < leaders; i += kThreads / 32) tile(i, std::integral_constant<int, 32>());
  } else {
    for (int i = 0; i < leaders; ++i) tile(i, std::integral_constant<int, kThreads>());
  }
}

template <int D, int TYPE>
void launch(const KvView &c, const void *k, const void *v, long long ks, long long vs, const int32_t *starts, int rows,
            dim3 grid, int per, cudaStream_t stream) {
  if (per == 1)
    kv_append_kernel<D, TYPE, 128, 1><<<grid, 128, 0, stream>>>(c, k, v, ks, vs, starts, rows, per);
  else if (c.page <= 64)  // registers for a page's rows: of 64, or of 128 (9.3K rows: 16.8 us, with room for 128 17.9)
    kv_append_kernel<D, TYPE, 256, D / 32><<<grid, 256, 0, stream>>>(c, k, v, ks, vs, starts, rows, per);
  else
    kv_append_kernel<D, TYPE, 256, D / 16><<<grid, 256, 0, stream>>>(c, k, v, ks, vs, starts, rows, per);
}

template <int D>
cudaError_t launch(const KvView &c, const void *k, const void *v, long long ks, long long vs, int type,
                   const int32_t *starts, int rows, dim3 grid, int per, cudaStream_t stream) {
  switch (type) {
    case MQA_KV_BF16: launch<D, MQA_KV_BF16>(c, k, v, ks, vs, starts, rows, grid, per, stream); break;
    case MQA_KV_FP16: launch<D, MQA_KV_FP16>(c, k, v, ks, vs, starts, rows, grid, per, stream); break;
    default: launch<D, MQA_KV_FP32>(c, k, v, ks, vs, starts, rows, grid, per, stream);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvView &c, const void *k, const void *v, long long ks, long long vs, int type,
                             const int32_t *starts, int rows, int sms, cudaStream_t stream) {
  // Rows per CTA.  Few: one, by 128 threads (32 tokens of 8 heads 3.0 us, with 16 per
  // CTA 4.4).  More: 16, by 256 (512 tokens 5.8 us, with one 12.9, with a page of 64
  // 11; a prompt of 300 rows 3.6, 6.7 and 4.5).  Many: a page's, so that a prompt's
  // CTA has about one tile (2,000 rows 5.4 us, with 16 7.6).
  const long long work = (long long)rows * c.heads * 2;
  const int per = work <= 4LL * sms ? 1 : work <= 96LL * sms ? 16 : c.page;
  const dim3 grid((rows + per - 1) / per, c.heads, 2);
  return c.dim == 64 ? launch<64>(c, k, v, ks, vs, type, starts, rows, grid, per, stream)
                     : launch<128>(c, k, v, ks, vs, type, starts, rows, grid, per, stream);
}

}  // namespace mqa
