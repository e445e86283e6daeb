// Norm and rotation of query and key heads in one pass (include/mqaqk.h,
// mqa_qk_norm_rope).
//
// Mathematics.  y = x rsqrt(mean x^2 + eps) w; each pair of y is turned by t = 2 pi
// frac(position * turns / 2^64).  The product is formed in 64-bit integers, whose
// wrap is the angle's, so the fraction is exact whatever the position; its upper
// 32 bits, rounded to fp32 (by at most 2^-26 of a turn), become the argument of sincospi.
//
// With r = rsqrt(...) and the weights taken in, a pair (a, b) becomes
//     (w_a cos) (r a) - (w_b sin) (r b),  (w_b cos) (r b) + (w_a sin) (r a):
// the four factors belong to the row, so they are formed once for all heads that a
// warp takes of it, and a component costs an unpacking, a square, a product by r, a product
// and a fused product, two components to an instruction.  (r first: |r a| is at most
// sqrt(D), so nothing leaves fp32's range that the answer does not.)
//
// Split.  A head is D / 8 lanes with four pairs each (of those that are not turned,
// any two components make a pair), a step of a warp 32 / (D / 8) heads of a row.  A warp
// takes a row's heads, q's, then k's, or a share of them where rows are few, with
// several steps' loads on their way; the angles of the CTA's rows are formed together
// into shared memory.
//
// What bounds it.  HBM: each component is read once and written once.  16,384 rows of
// 32 and 8 heads of 128 in bf16: 336 MB in 58.5 us, 5.74 TB/s, 85% of the measured copy
// rate; fp32, 8,192 rows: 5.9 TB/s.  Rows of few heads are bound by latency: a warp
// has two or three steps of work behind its CTA's chain positions -> angles -> barrier ->
// weights -> factors (60,000 rows of 2 and 1 heads of 128, 92 MB, 53 us, 1.7 TB/s; several
// rows to a warp, one after another, which keeps the chain: 59).  A kernel in which every head fetched its cosines from
// shared memory took 113 us (256 instructions per step of two heads, now 112).
#include "../../include/mqaqk.h"
#include "kv_ptx.cuh"

#include <climits>

namespace {

using namespace mqa;

// (16,384 rows of 32 and 8 heads of 128: 58.5 us with CTAs of 128 and six of them on an
// SM, 60.3 with three of 256, 67 with as many registers as the compiler likes; 64.5
// with two steps ahead and eight CTAs, 81 with one and ten.)
constexpr int kThreads = 128, kWarps = kThreads / 32;

struct QkParams {
  mqa_qk_heads q, k;
  int rows, half, norm, weight_type;
  int steps, q_steps;    // of a row, and those of its query heads
  int per_warp, shares;  // steps that a warp takes, warps that share a row
  float eps;
  const long long *turns;
  const int32_t *positions;
};

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Four elements: 8 bytes, or 16 of fp32.
template <int TYPE>
struct Four {
  static constexpr int words = TYPE == MQA_QK_FP32 ? 4 : 2;
  static constexpr int bytes = 4 * words;
  uint32_t w[words];
  __device__ __forceinline__ void load(const char *at) {
    if (TYPE == MQA_QK_FP32) {
      const uint4 v = *reinterpret_cast<const uint4 *>(at);
      w[0] = v.x, w[1] = v.y, w[words - 2] = v.z, w[words - 1] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2 *>(at);
      w[0] = v.x, w[1] = v.y;
    }
  }
  __device__ __forceinline__ void values(float (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (TYPE == MQA_QK_FP32) {
        f[2 * i] = __uint_as_float(w[(2 * i) % words]), f[2 * i + 1] = __uint_as_float(w[(2 * i + 1) % words]);
      } else {
        const float2 x = TYPE == MQA_QK_BF16 ? bf16x2_to_float2(w[i]) : half2_to_float2(w[i]);
        f[2 * i] = x.x, f[2 * i + 1] = x.y;
      }
    }
  }
  static __device__ __forceinline__ void store(char *at, float a, float b, float c, float d) {
    if (TYPE == MQA_QK_FP32)
      *reinterpret_cast<float4 *>(at) = make_float4(a, b, c, d);
    else
      *reinterpret_cast<uint2 *>(at) = TYPE == MQA_QK_BF16
                                           ? make_uint2(float2_to_bf162(a, b), float2_to_bf162(c, d))
                                           : make_uint2(float2_to_half2(a, b), float2_to_half2(c, d));
  }
};

template <int TYPE>
__device__ __forceinline__ void weights_of(const void *w, int at, float (&f)[4]) {
  Four<TYPE> o;
  o.load(reinterpret_cast<const char *>(w) + (size_t)at * (Four<TYPE>::bytes / 4));
  o.values(f);
}
__device__ __forceinline__ void load_weights(const void *w, int type, int at, float (&f)[4]) {
  if (!w) f[0] = f[1] = f[2] = f[3] = 1.f;
  else if (type == MQA_QK_FP32) weights_of<MQA_QK_FP32>(w, at, f);
  else if (type == MQA_QK_FP16) weights_of<MQA_QK_FP16>(w, at, f);
  else weights_of<MQA_QK_BF16>(w, at, f);
}
// From the order of memory (two runs of four) to pairs (a_0 .. a_3), (b_0 .. b_3), and back.
template <bool NEIGHBOURS>
__device__ __forceinline__ void to_pairs(const float (&x)[4], const float (&y)[4], uint64_t (&a)[2], uint64_t (&b)[2]) {
  a[0] = NEIGHBOURS ? pack2(x[0], x[2]) : pack2(x[0], x[1]);
  a[1] = NEIGHBOURS ? pack2(y[0], y[2]) : pack2(x[2], x[3]);
  b[0] = NEIGHBOURS ? pack2(x[1], x[3]) : pack2(y[0], y[1]);
  b[1] = NEIGHBOURS ? pack2(y[1], y[3]) : pack2(y[2], y[3]);
}

template <int LPH>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = LPH / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ float square_sum(const uint64_t (&f)[2], const uint64_t (&g)[2]) {
  float a, b;
  unpack2(fma2(g[1], g[1], fma2(g[0], g[0], fma2(f[1], f[1], mul2(f[0], f[0])))), a, b);
  return a + b;
}
__device__ __forceinline__ float rsqrt_of(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Heads whose squares leave fp32's range: the power of two that the components are
// multiplied with first, and r for those.  (The whole warp comes here; others keep
// theirs.)
template <int LPH, int D>
__device__ __noinline__ float2 rescued(uint64_t f0, uint64_t f1, uint64_t g0, uint64_t g1, float r, float eps, bool odd) {
  uint64_t f[4] = {f0, f1, g0, g1};
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2(f[i], a, b);
    amax = fmaxf(amax, fmaxf(fabsf(a), fabsf(b)));
  }
#pragma unroll
  for (int o = LPH / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  const bool able = odd && amax > 0.f && amax <= 3.402823466e38f;
  const float down = able ? pow2i(-max(-100, min(100, exponent_of(amax)))) : 1.f;
  uint64_t a[2], b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) a[i] = mul2(f[i], pack2(down, down)), b[i] = mul2(f[2 + i], pack2(down, down));
  const float s = sum_lanes<LPH>(square_sum(a, b));
  if (odd && amax == 0.f && eps > 0.f) return make_float2(1.f, 0.f);  // (rsqrt reads the least eps as zero)
  return make_float2(down, able ? rsqrt_of(s * (1.f / D) + eps * down * down) : r);
}

template <int D, int TYPE, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads, 6) qk_kernel(const QkParams p) {
  constexpr int LPH = D / 8, HEADS = 32 / LPH, AHEAD = TYPE == MQA_QK_FP32 ? 2 : 4;
  constexpr int SIZE = Four<TYPE>::bytes / 4, STEP = HEADS * D * SIZE;  // bytes of an element and from step to step
  extern __shared__ float4 s_angles[];                                  // [row][pair]: cos, sin
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane % LPH, sub = lane / LPH;
  const unsigned item0 = blockIdx.x * kWarps, item = item0 + warp, shares = p.shares;
  const int row0 = (int)(item0 / shares), row = (int)(item / shares);
  const int begin = (int)(item - row * shares) * p.per_warp;
  const int end = row < p.rows ? min(begin + p.per_warp, p.steps) : begin;
  // the lane's two runs of four components
  const bool turned = part < p.half / 4;
  const int lo = NEIGHBOURS || !turned ? part * 8 : part * 4, hi = NEIGHBOURS || !turned ? lo + 4 : lo + p.half;
  const float tiny = p.eps < 0x1p-90f ? 0x1p-90f : 0.f;
  Four<TYPE> x[AHEAD], y[AHEAD];
  // steps [s0, s1) of a row's heads of one kind, s1 - s0 of which hold one for the lane's part of the warp
  struct Run {
    const char *in;
    char *out;
    int steps, mine;
  };
  auto run_of = [&](const mqa_qk_heads &h, int s0, int s1) {
    Run r;
    const int head = s0 * HEADS + sub;
    r.in = reinterpret_cast<const char *>(h.in) + ((size_t)row * h.in_stride + (size_t)head * D + lo) * SIZE;
    r.out = reinterpret_cast<char *>(h.out) + ((size_t)row * h.out_stride + (size_t)head * D + lo) * SIZE;
    r.steps = max(s1 - s0, 0);
    r.mine = min(r.steps, (h.heads - head + HEADS - 1) / HEADS);
    return r;
  };
  const int apart = (hi - lo) * SIZE;
  auto load = [&](const Run &r, int i, int step) {
    if (step < r.mine) {
      x[i].load(r.in + (size_t)step * STEP);
      y[i].load(r.in + (size_t)step * STEP + apart);
    } else {
#pragma unroll
      for (int k = 0; k < Four<TYPE>::words; ++k) x[i].w[k] = y[i].w[k] = 0;
    }
  };
  const Run q = run_of(p.q, min(begin, p.q_steps), min(end, p.q_steps));
  const Run k = run_of(p.k, max(begin - p.q_steps, 0), end - p.q_steps);
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load(q.steps ? q : k, i, i);
  const int rows_here = min((int)((item0 + kWarps - 1) / shares), p.rows - 1) - row0 + 1;
  for (int i = threadIdx.x; i < rows_here * p.half; i += kThreads) {
    const int r = i / p.half, pair = i - r * p.half;
    const unsigned long long phase =
        (unsigned long long)(long long)__ldg(p.positions + row0 + r) * (unsigned long long)__ldg(p.turns + pair);
    float s, c;
    sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s, &c);
    reinterpret_cast<float2 *>(s_angles)[i] = make_float2(c, s);
  }
  __syncthreads();
  auto work = [&](const mqa_qk_heads &h, const Run &r) {
    uint64_t ca[2], sa[2], cb[2], sb[2];  // a' = ca (r a) + sa (r b), b' = cb (r b) + sb (r a)
    {
      float u[4], v[4], c[4], s[4];
      uint64_t wa[2], wb[2];
      load_weights(h.weight, p.weight_type, lo, u);
      load_weights(h.weight, p.weight_type, hi, v);
      to_pairs<NEIGHBOURS>(u, v, wa, wb);
      const float4 *t = s_angles + ((row - row0) * p.half + part * 4) / 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 cs = turned ? t[i] : make_float4(1.f, 0.f, 1.f, 0.f);
        c[2 * i] = cs.x, s[2 * i] = cs.y, c[2 * i + 1] = cs.z, s[2 * i + 1] = cs.w;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t c2 = pack2(c[2 * i], c[2 * i + 1]), s2 = pack2(s[2 * i], s[2 * i + 1]);
        ca[i] = mul2(wa[i], c2), cb[i] = mul2(wb[i], c2);
        sb[i] = mul2(wa[i], s2), sa[i] = mul2(wb[i], pack2(-s[2 * i], -s[2 * i + 1]));
      }
    }
    for (int step = 0; step < r.steps; step += AHEAD) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (step + i >= r.steps) break;
        float u[4], v[4];
        uint64_t a[2], b[2];
        x[i].values(u);
        y[i].values(v);
        to_pairs<NEIGHBOURS>(u, v, a, b);
        load(r, i, step + i + AHEAD);
        float f = 1.f;
        if (p.norm) {
          const float ss = sum_lanes<LPH>(square_sum(a, b));
          f = rsqrt_of(fmaf(ss, 1.f / D, p.eps));
          const bool odd = !(ss <= 3e38f) || ss < tiny;
          if (__any_sync(~0u, odd)) {
            const float2 by = rescued<LPH, D>(a[0], a[1], b[0], b[1], f, p.eps, odd);
            f = by.y;
#pragma unroll
            for (int j = 0; j < 2; ++j) a[j] = mul2(a[j], pack2(by.x, by.x)), b[j] = mul2(b[j], pack2(by.x, by.x));
          }
        }
        float e[4], g[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          a[j] = mul2(a[j], pack2(f, f)), b[j] = mul2(b[j], pack2(f, f));
          uint64_t aa = mul2(ca[j], a[j]), bb = mul2(cb[j], b[j]);
          if (turned) aa = fma2(sa[j], b[j], aa), bb = fma2(sb[j], a[j], bb);
          unpack2(aa, e[2 * j], e[2 * j + 1]);
          unpack2(bb, g[2 * j], g[2 * j + 1]);
        }
        if (step + i < r.mine) {
          char *out = r.out + (size_t)(step + i) * STEP;
          if (NEIGHBOURS) {
            Four<TYPE>::store(out, e[0], g[0], e[1], g[1]);
            Four<TYPE>::store(out + apart, e[2], g[2], e[3], g[3]);
          } else {
            Four<TYPE>::store(out, e[0], e[1], e[2], e[3]);
            Four<TYPE>::store(out + apart, g[0], g[1], g[2], g[3]);
          }
        }
      }
    }
  };
  if (q.steps) work(p.q, q);
  if (k.steps) {
    if (q.steps) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) load(k, i, i);
    }
    work(p.k, k);
  }
}

template <int D, int TYPE>
cudaError_t launch(QkParams &p, bool neighbours, int sms, cudaStream_t stream) {
  constexpr int kHeads = 32 / (D / 8);
  p.q_steps = (p.q.heads + kHeads - 1) / kHeads;
  p.steps = p.q_steps + (p.k.heads + kHeads - 1) / kHeads;
  // a row for each warp, or so many that every SM has 32
  const long long want = (32LL * sms + p.rows - 1) / p.rows;
  p.shares = (int)(want < p.steps ? want : p.steps);
  p.per_warp = (p.steps + p.shares - 1) / p.shares;
  p.shares = (p.steps + p.per_warp - 1) / p.per_warp;
  const long long items = (long long)p.rows * p.shares, ctas = (items + kWarps - 1) / kWarps;
  const size_t smem = (size_t)((kWarps - 1) / p.shares + 2) * p.half * sizeof(float2);
  if (neighbours)
    qk_kernel<D, TYPE, true><<<(unsigned)ctas, kThreads, smem, stream>>>(p);
  else
    qk_kernel<D, TYPE, false><<<(unsigned)ctas, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(QkParams &p, int type, bool neighbours, int sms, cudaStream_t stream) {
  return type == MQA_QK_BF16   ? launch<D, MQA_QK_BF16>(p, neighbours, sms, stream)
         : type == MQA_QK_FP16 ? launch<D, MQA_QK_FP16>(p, neighbours, sms, stream)
                               : launch<D, MQA_QK_FP32>(p, neighbours, sms, stream);
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
  p.half = rotary / 2;
  p.norm = norm != 0;
  p.weight_type = weight_type;
  p.eps = eps;
  p.turns = reinterpret_cast<const long long *>(turns);
  p.positions = positions;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = head_dim == 64    ? launch<64>(p, type, interleaved != 0, sms, s)
                        : head_dim == 128 ? launch<128>(p, type, interleaved != 0, sms, s)
                                          : launch<256>(p, type, interleaved != 0, sms, s);
  if (e == cudaSuccess) return MQA_OK;
  cudaGetLastError();
  return MQA_ERR_CUDA;
}
