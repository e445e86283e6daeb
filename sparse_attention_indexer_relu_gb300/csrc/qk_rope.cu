// Norm and rotation of query and key heads in one pass (include/mqaqk.h,
// mqa_qk_norm_rope).
//
// Mathematics.  y = x rsqrt(mean x^2 + eps) w; each pair of y is turned by t = 2 pi
// frac(position * turns / 2^64).  The product is formed in 64-bit integers, whose
// wrap is the angle's, so the fraction is exact whatever the position; its upper
// 32 bits become the argument of sincospi.
//
// Split.  A unit is a head of a row, D / 8 lanes with 8 components each.  A CTA has
// consecutive units, all of whose loads are on their way while the angles of its
// rows are formed once for all heads into shared memory.
#include "../../include/mqaqk.h"
#include "kv_ptx.cuh"

#include <climits>

namespace {

using namespace mqa;

constexpr int kThreads = 256;

struct QkParams {
  mqa_qk_heads q, k;
  int rows, heads, half, interleaved, norm, weight_type, held;  // heads: of q and k; held: rows a CTA may touch
  unsigned units;
  float eps;
  const long long *turns;
  const int32_t *positions;
};

// 8 elements: 16 bytes, or 32 of fp32.
template <int TYPE>
struct Octet {
  uint4 w[TYPE == MQA_QK_FP32 ? 2 : 1];
  __device__ __forceinline__ void load(const void *base, size_t at) {
    if (TYPE == MQA_QK_FP32) {
      const uint4 *s = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(base) + at);
      w[0] = s[0], w[TYPE == MQA_QK_FP32 ? 1 : 0] = s[1];
    } else {
      w[0] = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + at);
    }
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (TYPE == MQA_QK_FP32) {
        const uint4 &v = w[TYPE == MQA_QK_FP32 ? i >> 1 : 0];
        f[2 * i] = __uint_as_float(i & 1 ? v.z : v.x), f[2 * i + 1] = __uint_as_float(i & 1 ? v.w : v.y);
      } else {
        const uint32_t v = i == 0 ? w[0].x : i == 1 ? w[0].y : i == 2 ? w[0].z : w[0].w;
        const float2 x = TYPE == MQA_QK_BF16 ? bf16x2_to_float2(v) : half2_to_float2(v);
        f[2 * i] = x.x, f[2 * i + 1] = x.y;
      }
    }
  }
  static __device__ __forceinline__ void store(void *base, size_t at, const float (&f)[8]) {
    if (TYPE == MQA_QK_FP32) {
      float4 *d = reinterpret_cast<float4 *>(reinterpret_cast<float *>(base) + at);
      d[0] = make_float4(f[0], f[1], f[2], f[3]);
      d[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = TYPE == MQA_QK_BF16 ? float2_to_bf162(f[2 * i], f[2 * i + 1]) : float2_to_half2(f[2 * i], f[2 * i + 1]);
      *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(base) + at) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
};

__device__ __forceinline__ void load_weight(const void *w, int type, int at, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 1.f;
  } else if (type == MQA_QK_FP32) {
    Octet<MQA_QK_FP32> o;
    o.load(w, at);
    o.values(f);
  } else if (type == MQA_QK_FP16) {
    Octet<MQA_QK_FP16> o;
    o.load(w, at);
    o.values(f);
  } else {
    Octet<MQA_QK_BF16> o;
    o.load(w, at);
    o.values(f);
  }
}

template <int LPH>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = LPH / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
template <int LPH>
__device__ __forceinline__ float max_lanes(float v) {
#pragma unroll
  for (int o = LPH / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}

// Squares that leave fp32's range: the head times a power of two first (the whole
// warp comes here; heads for which `odd` is false keep their factor).
template <int LPH, int D>
__device__ __noinline__ float rescued(float amax, float ss, float eps, bool odd, const float (&f)[8]) {
  amax = max_lanes<LPH>(amax);
  const int e = max(-100, min(100, exponent_of(amax)));
  const float down = pow2i(-e);
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = f[j] * down;
    s = fmaf(x, x, s);
  }
  s = sum_lanes<LPH>(s);
  const float r = rsqrtf(s * (1.f / D) + eps * down * down) * down;
  return odd && amax > 0.f && amax <= 3.402823466e38f ? r : rsqrtf(ss * (1.f / D) + eps);
}

// UNITS units per group of lanes.
template <int D, int TYPE, int UNITS>
__global__ void __launch_bounds__(kThreads) qk_kernel(const QkParams p) {
  constexpr int LPH = D / 8, GROUPS = kThreads / LPH;
  extern __shared__ float4 s_turn[];  // [row][pair of pairs j][lane of the head]: cos, sin, cos, sin
  const int lane = threadIdx.x % LPH, group = threadIdx.x / LPH;
  const unsigned first = blockIdx.x * (unsigned)(GROUPS * UNITS);
  const int row0 = (int)(first / (unsigned)p.heads);
  Octet<TYPE> x[UNITS];
  int row[UNITS], head[UNITS];
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const unsigned u = first + i * GROUPS + group;
    row[i] = (int)(u / (unsigned)p.heads);
    head[i] = (int)(u - (unsigned)row[i] * p.heads);
    const bool is_q = head[i] < p.q.heads;
    const mqa_qk_heads &h = is_q ? p.q : p.k;
    if (u < p.units)
      x[i].load(h.in, (size_t)row[i] * h.in_stride + (size_t)(is_q ? head[i] : head[i] - p.q.heads) * D + lane * 8);
    else
      x[i].w[0] = x[i].w[TYPE == MQA_QK_FP32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
  }
  // ---- angles of the rows: a lane of a head turns 8 pairs (halves, with the lane
  // that has the other component) or 4 (neighbours)
  const int ppl = p.interleaved ? 4 : 8, slots = p.half / ppl;
  for (int i = threadIdx.x; i < p.held * p.half; i += kThreads) {
    const int r = i / p.half, pair = i - r * p.half;
    if (row0 + r >= p.rows) break;
    const unsigned long long phase =
        (unsigned long long)(long long)__ldg(p.positions + row0 + r) * (unsigned long long)__ldg(p.turns + pair);
    float s, c;
    sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s, &c);
    float2 *at = reinterpret_cast<float2 *>(s_turn + r * (p.half / 2) + (pair % ppl >> 1) * slots + pair / ppl);
    at[pair & 1] = make_float2(c, s);
  }
  float wq[8], wk[8];
  load_weight(p.q.heads ? p.q.weight : nullptr, p.weight_type, lane * 8, wq);
  load_weight(p.k.heads ? p.k.weight : nullptr, p.weight_type, lane * 8, wk);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const unsigned u = first + i * GROUPS + group;
    float f[8];
    x[i].values(f);
    const bool is_q = head[i] < p.q.heads;
    if (p.norm) {
      float ss = 0.f, amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss), amax = fmaxf(amax, fabsf(f[j]));
      ss = sum_lanes<LPH>(ss);
      float rs = rsqrtf(ss * (1.f / D) + p.eps);
      const bool odd = !(ss <= 3e38f) || (ss < 0x1p-90f && p.eps < 0x1p-90f);
      if (__any_sync(~0u, odd)) rs = rescued<LPH, D>(amax, ss, p.eps, odd, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * rs * (is_q ? wq[j] : wk[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= is_q ? wq[j] : wk[j];
    }
    const float4 *turn = s_turn + (row[i] - row0) * (p.half / 2);
    if (p.interleaved) {
      if (lane < slots && u < p.units) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 t = turn[j * slots + lane];
          const float a = f[4 * j], b = f[4 * j + 1], c = f[4 * j + 2], d = f[4 * j + 3];
          f[4 * j] = a * t.x - b * t.y, f[4 * j + 1] = b * t.x + a * t.y;
          f[4 * j + 2] = c * t.z - d * t.w, f[4 * j + 3] = d * t.z + c * t.w;
        }
      }
    } else if (p.half) {
      const int base = threadIdx.x & 31 & ~(LPH - 1), mine = lane < slots ? lane : lane - slots;
      const int other = lane < slots ? lane + slots : lane < 2 * slots ? lane - slots : lane;
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = __shfl_sync(~0u, f[j], base + other);
      if (lane < 2 * slots && u < p.units) {
        const float sign = lane < slots ? -1.f : 1.f;  // (a cos - b sin, b cos + a sin)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 t = turn[j * slots + mine];
          f[2 * j] = f[2 * j] * t.x + sign * g[2 * j] * t.y;
          f[2 * j + 1] = f[2 * j + 1] * t.z + sign * g[2 * j + 1] * t.w;
        }
      }
    }
    if (u < p.units) {
      const mqa_qk_heads &h = is_q ? p.q : p.k;
      Octet<TYPE>::store(h.out, (size_t)row[i] * h.out_stride + (size_t)(is_q ? head[i] : head[i] - p.q.heads) * D +
                                    lane * 8, f);
    }
  }
}

template <int D, int TYPE>
cudaError_t launch(QkParams &p, int sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  auto run = [&](auto *kernel, int units) {
    const unsigned per = kGroups * units, ctas = (p.units + per - 1) / per;
    p.held = (int)((per - 1) / p.heads + 2);
    if (p.held > p.rows) p.held = p.rows;
    kernel<<<ctas, kThreads, (size_t)p.held * p.half * 8, stream>>>(p);
    return cudaGetLastError();
  };
  const bool few = p.units <= (unsigned)(sms * 4 * kGroups);
  return few ? run(qk_kernel<D, TYPE, 1>, 1) : run(qk_kernel<D, TYPE, 4>, 4);
}

template <int D>
cudaError_t launch(QkParams &p, int type, int sms, cudaStream_t stream) {
  return type == MQA_QK_BF16   ? launch<D, MQA_QK_BF16>(p, sms, stream)
         : type == MQA_QK_FP16 ? launch<D, MQA_QK_FP16>(p, sms, stream)
                               : launch<D, MQA_QK_FP32>(p, sms, stream);
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_heads(const mqa_qk_heads &h, int rows, int dim, int per16) {
  if (h.heads < 0 || h.heads > 65536) return MQA_ERR_INVALID_ARGUMENT;
  if (h.heads == 0) return MQA_OK;
  const long long width = (long long)h.heads * dim;
  if (!h.in || !h.out || (rows > 1 && (h.in_stride < width || h.out_stride < width))) return MQA_ERR_INVALID_ARGUMENT;
  if (!aligned(h.in, 16) || !aligned(h.out, 16) || !aligned(h.weight, 16) || h.in_stride % per16 ||
      h.out_stride % per16)
    return MQA_ERR_MISALIGNED;
  return MQA_OK;
}

}  // namespace

extern "C" int mqa_qk_norm_rope(const mqa_qk_heads *q, const mqa_qk_heads *k, int rows, int type, int weight_type,
                                int head_dim, int rotary, int interleaved, int norm, float eps, const int64_t *turns,
                                const int32_t *positions, void *stream) {
  if (!q || !k || rows < 0 || type < MQA_QK_BF16 || type > MQA_QK_FP32 || weight_type < MQA_QK_BF16 ||
      weight_type > MQA_QK_FP32 || (head_dim != 64 && head_dim != 128 && head_dim != 256) || rotary < 0 ||
      rotary > head_dim || rotary % 16 || !(eps >= 0.f && eps <= 3.402823466e38f))
    return MQA_ERR_INVALID_ARGUMENT;
  const int per16 = type == MQA_QK_FP32 ? 4 : 8;
  if (rows == 0 || q->heads + k->heads == 0) {
    return q->heads < 0 || k->heads < 0 ? MQA_ERR_INVALID_ARGUMENT : MQA_OK;
  }
  int rc = check_heads(*q, rows, head_dim, per16);
  if (rc == MQA_OK) rc = check_heads(*k, rows, head_dim, per16);
  if (rc != MQA_OK) return rc;
  if ((long long)rows * (q->heads + k->heads) > INT_MAX || (rotary && (!turns || !positions)))
    return MQA_ERR_INVALID_ARGUMENT;
  if (!aligned(turns, 8) || !aligned(positions, 4)) return MQA_ERR_MISALIGNED;
  int sms = 0;
  rc = require_device(&sms);
  if (rc != MQA_OK) return rc;
  QkParams p = {};
  p.q = *q;
  p.k = *k;
  p.rows = rows;
  p.heads = q->heads + k->heads;
  p.half = rotary / 2;
  p.interleaved = interleaved != 0;
  p.norm = norm != 0;
  p.weight_type = weight_type;
  p.units = (unsigned)rows * p.heads;
  p.eps = eps;
  p.turns = reinterpret_cast<const long long *>(turns);
  p.positions = positions;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = head_dim == 64    ? launch<64>(p, type, sms, s)
                        : head_dim == 128 ? launch<128>(p, type, sms, s)
                                          : launch<256>(p, type, sms, s);
  if (e == cudaSuccess) return MQA_OK;
  cudaGetLastError();
  return MQA_ERR_CUDA;
}
