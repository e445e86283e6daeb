// Device helpers of the paged key/value cache's kernels: asynchronous copies,
// fp16 matrix products, powers of two and row conversions.
#pragma once
#include "kv_internal.h"
#include "ptx.cuh"

#include <atomic>
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace mqa {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// floor(log2 |x|) of a finite nonzero fp32 (subnormals read as -127).
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }
// Scale of a UE8M0 byte, 1 <= e <= 254: the fp32 with bit pattern e << 23 (0 and
// 255, which are not scales, read as their neighbours: never 0 or infinity).
__device__ __forceinline__ float exp_byte(uint32_t e) { return __uint_as_float(min(max(e, 1u), 254u) << 23); }

// Kernels of one call follow each other by programmatic dependent launch: each
// lets the next one's blocks be scheduled at once, and waits for the one before
// (its writes included) before it reads what that one wrote.  What a kernel
// writes before it waits, no earlier kernel of the call touches: the split
// kernel, which waits at its end, has rows, descriptions and slots of its own.
// Every block waits, so that a kernel's end means its predecessors' end too.
__device__ __forceinline__ void grid_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Factor of a product's scores: what a column's are multiplied with times a
// block's scale.  Never zero, which would turn a masked score (-inf) into NaN
// (the least normal number that is added changes no factor above 2^-101).
__device__ __forceinline__ float score_factor(float column, float block) { return fmaf(column, block, 0x1p-126f); }

// e4m3 code pair (low 16 bits) to fp16 pair.
__device__ __forceinline__ uint32_t cvt2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t cvt2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Four fp32 to four e4m3 codes (nearest even, saturating, NaN kept).
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tmov.b32 %0, {x, 0};\n\t}"
      : "=r"(lo)
      : "f"(a), "f"(b));
  asm("{\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tmov.b32 %0, {x, 0};\n\t}"
      : "=r"(hi)
      : "f"(c), "f"(d));
  return lo | hi << 16;
}
// Bytes of w that hold a NaN code (0x7F or 0xFF), as 0x80 bits.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), fp16 operands.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit values held two per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Barrier among `threads` threads of the CTA.
__device__ __forceinline__ void named_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// 32 lanes x 16 columns of 32-bit TMEM.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 16 bytes global -> shared without registers; zeros where !ok (nothing is read then).
__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
               "l"(__cvta_generic_to_global(src)), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Ordinary accesses to shared memory before, copies and MMAs after.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t w) {
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}
__device__ __forceinline__ uint32_t float2_to_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
__device__ __forceinline__ uint32_t float2_to_bf162(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}

// Wait for a barrier's phase: true once it is complete.  Once a wait of the CTA
// has run out (2 s), every wait for what has not come returns false at once.
// The warps that issue copies then leave: a barrier never counts the bytes of
// more than one phase, and the last phase's can be waited for (drain).  The
// others may run to their end, on whatever lies in shared memory: none of it
// may reach an address unchecked.  (A vote per wait that lets them leave, too,
// costs the tiled kernel 5% of a chunk of 32K positions.)
// S::test: compilation for tests, with a limit of its own.
constexpr unsigned long long kWaitNs = 2000000000ULL;
template <typename S>
__device__ __forceinline__ bool bounded_wait(S &sm, uint64_t *bar, uint32_t parity, const AttnParams &p) {
  if (mbar_try_wait(bar, parity)) return true;
  unsigned long long t0 = 0;
  for (int i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 15) == 15) {
      if (*reinterpret_cast<volatile int *>(&sm.dead)) return false;
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > (S::test ? p.wait_ns : kWaitNs)) {
        *reinterpret_cast<volatile int *>(&sm.dead) = 1;
        atomicOr(p.c.status, MQA_KV_DEV_WAIT_TIMEOUT);
        return false;
      }
    }
  }
}
// The same for the whole warp; what its lanes wrote before, all of them see (a
// vote alone orders no memory).
template <typename S>
__device__ __forceinline__ bool warp_wait(S &sm, uint64_t *bar, uint32_t parity, const AttnParams &p) {
  const bool ok = __all_sync(~0u, bounded_wait(sm, bar, parity, p));
  __syncwarp();
  return ok;
}
// For copies and products under way, also after a wait has run out.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < kWaitNs) {
  }
}

template <typename... Params, typename... Args>
inline cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                bool follows, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &a;
  cfg.numAttrs = follows ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}
// A kernel's dynamic shared memory limit, raised once per device.
typedef std::atomic<unsigned long long> DeviceFlags;
template <typename K>
inline cudaError_t allow_smem(K *kernel, size_t bytes, DeviceFlags &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ULL << dev, std::memory_order_release);
  return e;
}

template <int CB, int D>
__host__ __device__ constexpr size_t attn_slot_floats_dev() {
  return (size_t)CB * (D + 4);
}

// One warp writes a row of a head, a lane E consecutive components: acc = sum
// 2^(s + lv - w) E(v), ls = sum 2^(s - m), so the result is acc / ls * 2^(w - m);
// zeros where nothing was seen (m = -inf and no NaN).
template <int E>
__device__ __forceinline__ void finish_lane(const AttnParams &p, int row, int head, int lane, const float (&acc)[E],
                                            float m, float w, float ls) {
  const bool none = m == -INFINITY && ls == 0.f;
  const float f = none ? 0.f : ls != ls ? NAN : ex2(w - m) / ls;
  const size_t at = (size_t)row * p.q_heads + head;
  uint32_t *o = reinterpret_cast<uint32_t *>(p.out) + (at * 32 + lane) * (E / 2);
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float a = none ? 0.f : acc[e] * f, b = none ? 0.f : acc[e + 1] * f;
    o[e / 2] = p.bf16 ? float2_to_bf162(a, b) : float2_to_half2(a, b);
  }
  if (p.lse && lane == 0) p.lse[at] = none ? -INFINITY : (m + log2f(ls)) * 0.693147180559945309f;
}

}  // namespace mqa
