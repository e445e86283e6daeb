// Appending to the paged 8-bit cache (include/mqakv.h, mqa_kv_append).
//
// For a page, a head and keys or values, with new magnitudes up to a:
//     e = max(e_old if the page held earlier positions, min e: a <= 448 2^(e - 127))
//     code = RNE_e4m3(x 2^(127 - e));  earlier codes: RNE_e4m3(E(code) 2^(e_old - e))
// Scales are powers of two, so every product is exact and the only rounding is
// the one to e4m3 (half a step: 2^-4 of the value).
//
// Bound by memory: rows * heads * dim * (input bytes + 1), twice (K and V).  A
// CTA looks at a few consecutive rows, finds those that begin a page's new
// positions (its leaders) and writes each leader's tile: one pass for the
// magnitude, a second over the same bytes (from L1/L2) for the codes.
#include "kv_ptx.cuh"

#include <cuda_fp8.h>

namespace mqa {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxRows = 16;  // rows a CTA looks at

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

// 8 elements of a row as fp32 (bf16, fp16: one 16-byte load; fp32: two).
template <int TYPE>
__device__ __forceinline__ void load8(const void *base, size_t at, float (&f)[8]) {
  if (TYPE == MQA_KV_FP32) {
    const float4 *s = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + at);
    const float4 x = __ldg(s), y = __ldg(s + 1);
    f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
  } else {
    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + at));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = TYPE == MQA_KV_BF16 ? bf16x2_to_float2(ws[i]) : half2_to_float2(ws[i]);
      f[2 * i] = x.x, f[2 * i + 1] = x.y;
    }
  }
}

template <int D, int TYPE>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvView c, const void *__restrict__ kin,
                                                            const void *__restrict__ vin, long long ks, long long vs,
                                                            const int32_t *__restrict__ starts, int rows, int per) {
  __shared__ int s_page[kMaxRows], s_slot[kMaxRows], s_count[kMaxRows], s_held[kMaxRows];
  __shared__ float s_max[kThreads / 32];
  const int tid = threadIdx.x, head = blockIdx.y, values = blockIdx.z;
  const int row0 = blockIdx.x * per;
  if (tid < per) {
    const int r = row0 + tid;
    int count = 0, page = -1, slot = 0, held = 0;
    if (r < rows) {
      int lo = 0, hi = c.seqs;  // the last sequence that starts at or before the row
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(starts + mid) <= r) lo = mid; else hi = mid;
      }
      const int a = max(__ldg(starts + lo), 0), b = min(__ldg(starts + lo + 1), rows);
      const int len = __ldg(c.lens + lo);
      const long long pos = (long long)len - (b - a) + (r - a);  // position of the row
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
              held = slot;
            }
          }
        }
      }
    }
    s_page[tid] = page, s_slot[tid] = slot, s_count[tid] = count, s_held[tid] = held;
  }
  __syncthreads();
  const void *in = values ? vin : kin;
  const long long stride = values ? vs : ks;
  uint8_t *codes = values ? c.v : c.k;
  uint8_t *exps = values ? c.v_exps : c.k_exps;
  constexpr int LPR = D / 8, RPS = kThreads / LPR;  // lanes per row, rows per step
  const int part = tid % LPR, step = tid / LPR;
  for (int i = 0; i < per; ++i) {
    const int count = s_count[i];
    if (count == 0) continue;  // the same for the whole CTA
    const size_t base = (size_t)(row0 + i) * stride + (size_t)head * D + part * 8;
    float amax = 0.f;
#pragma unroll 4
    for (int r = step; r < count; r += RPS) {
      float f[8];
      load8<TYPE>(in, base + (size_t)r * stride, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = fabsf(f[j]);
        amax = a <= 3.402823466e38f ? fmaxf(amax, a) : amax;  // infinities and NaN do not set the scale
      }
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, x));
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    const size_t ph = (size_t)s_page[i] * c.heads + head;
    const int held = s_held[i], was = held ? exps[ph] : 0;
    __syncthreads();  // s_max written, the old exponent read by all
    amax = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const int e = max(needed_exp(amax), was);
    uint8_t *tile = codes + (ph << c.page_log2) * D;
    if (held && e > was) {  // earlier positions under the larger scale
      const float f = pow2i(max(was - e, -126));
      for (int j = tid; j < held * D / 4; j += kThreads) {
        uint32_t *w = reinterpret_cast<uint32_t *>(tile) + j;
        const uint32_t x = *w;
        *w = to_e4m3x4(from_e4m3(x & 255u) * f, from_e4m3(x >> 8 & 255u) * f, from_e4m3(x >> 16 & 255u) * f,
                       from_e4m3(x >> 24) * f);
      }
    }
    // 2^(127 - e); a page that was given a byte above 247 may need a subnormal
    const float up = e < 254 ? pow2i(127 - e) : __uint_as_float(0x00400000u >> (e - 254));
#pragma unroll 4
    for (int r = step; r < count; r += RPS) {
      float f[8];
      load8<TYPE>(in, base + (size_t)r * stride, f);
      uint2 o;
      o.x = to_e4m3x4(f[0] * up, f[1] * up, f[2] * up, f[3] * up);
      o.y = to_e4m3x4(f[4] * up, f[5] * up, f[6] * up, f[7] * up);
      *reinterpret_cast<uint2 *>(tile + (size_t)(s_slot[i] + r) * D + part * 8) = o;
    }
    if (tid == 0) exps[ph] = (uint8_t)e;
    __syncthreads();  // s_max is free again
  }
}

template <int D>
cudaError_t launch(const KvView &c, const void *k, const void *v, long long ks, long long vs, int type,
                   const int32_t *starts, int rows, dim3 grid, int per, cudaStream_t stream) {
  switch (type) {
    case MQA_KV_BF16:
      kv_append_kernel<D, MQA_KV_BF16><<<grid, kThreads, 0, stream>>>(c, k, v, ks, vs, starts, rows, per);
      break;
    case MQA_KV_FP16:
      kv_append_kernel<D, MQA_KV_FP16><<<grid, kThreads, 0, stream>>>(c, k, v, ks, vs, starts, rows, per);
      break;
    default: kv_append_kernel<D, MQA_KV_FP32><<<grid, kThreads, 0, stream>>>(c, k, v, ks, vs, starts, rows, per);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvView &c, const void *k, const void *v, long long ks, long long vs, int type,
                             const int32_t *starts, int rows, int sms, cudaStream_t stream) {
  // one row per CTA while the rows fit a few waves (decode: every row is a
  // leader); more rows per CTA for prompts, where one in page_size is
  const long long units = (long long)rows * c.heads * 2;
  int per = 1;
  while (per < kMaxRows && units / per > 32LL * sms) per *= 2;
  const dim3 grid((rows + per - 1) / per, c.heads, 2);
  return c.dim == 64 ? launch<64>(c, k, v, ks, vs, type, starts, rows, grid, per, stream)
                     : launch<128>(c, k, v, ks, vs, type, starts, rows, grid, per, stream);
}

}  // namespace mqa
