// Attention over the paged 8-bit cache for many query columns per key/value
// head (prompts and their chunks) on the tcgen05 tensor cores.
// (include/mqakv.h, mqa_kv_attention; the mathematics is kv_attn.cu's.)
//
// A CTA holds 256 columns of an item (query row x query head of one key/value
// head) as two 128-row tiles and walks over 128-key tiles:
//     S = Q K^T (Q, K fp16 in shared memory, S fp32 in TMEM),
//     P = 2^(s + lv - w) rounded to fp16, written back over S in TMEM,
//     O += P V (P from TMEM, V fp16 in shared memory, O fp32 in TMEM).
// While one tile's scores are turned into weights the tensor cores work on the
// other tile.  Roles: 2 x 4 softmax warps (a thread per column; it also moves
// its references and rescales its row of O when a score passes them by 2^8),
// 2 x 4 converter warps (codes from global memory to fp16 in the swizzled
// layouts that the MMAs read: K with its components contiguous, V as it lies,
// which the MMA reads transposed), one issuing warp.
// Every wait has a time limit; once one has run out, all of them return at
// once and the kernel runs to its end on whatever it finds in shared memory.
//
// Work is cut like kv_attn.cu's: the key tiles of all items in one line, even
// parts per CTA, partial results in two slots per CTA and a joining pass.  The
// position of a part is found from the exact number of tiles that causal
// column blocks need (a sum of floors).
#include "kv_ptx.cuh"

#include <cfloat>

namespace mqa {

namespace {

constexpr int kThreads = 640;
constexpr int kKeys = 128;                // keys per tile
constexpr int kCols = kTiledCols;         // columns per item
constexpr int kStagesKV = 2;
constexpr int kMeta = 4;                  // tile descriptions in flight (softmax is at most 3 behind)
constexpr float kSlack = 8.0f;
constexpr long long kWaitNs = 2000000000LL;
constexpr int kConverters = 128;
constexpr int kBarConv = 1;               // named barriers of the two converter groups

// sum over 0 <= i < n of floor((a i + b) / m); a, b >= 0, m > 0.  Whole parts
// first; what is left below the line is counted along the other axis.
template <typename T>
__device__ __forceinline__ long long floor_sum_as(long long n, T m, T a, T b) {
  long long sum = 0;
  while (true) {
    const T qa = a / m, qb = b / m;
    sum += n * (n - 1) / 2 * (long long)qa + n * (long long)qb;
    a -= qa * m;
    b -= qb * m;
    const T top = a * (T)n + b;
    if (top < m) return sum;
    n = (long long)(top / m);
    b = top - (T)n * m;
    const T x = a;
    a = m;
    m = x;
  }
}
__device__ __forceinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  // all that is divided is at most a n + b: 32-bit division where that fits
  if (n < (1 << 20) && a * n + b < (1LL << 32)) return floor_sum_as<uint32_t>(n, (uint32_t)m, (uint32_t)a, (uint32_t)b);
  return floor_sum_as<unsigned long long>(n, m, a, b);
}

// Shape of a sequence's work.
struct Seq {
  int r0, n, len, blocks;
};
__device__ __forceinline__ Seq seq_of(const AttnParams &p, int s) {
  Seq q;
  q.r0 = min(max(p.starts[s], 0), p.rows);
  q.n = max(min(p.starts[s + 1], p.rows) - q.r0, 0);
  q.len = min(max(p.c.lens[s], 0), p.c.max_pages << p.c.page_log2);
  const long long cols = (long long)q.n * p.group;
  q.blocks = cols > p.max_cols ? (int)((cols + kCols - 1) / kCols) : 0;
  return q;
}
__device__ __forceinline__ int tiles_for(int lim) { return max(1, (lim + kKeys - 1) / kKeys); }
// Positions that the last column of a block sees.
__device__ __forceinline__ int block_limit(const AttnParams &p, const Seq &q, int block) {
  const int last = min(q.n - 1, (block * kCols + kCols - 1) / p.group);
  return p.causal ? min(max(q.len - q.n + last + 1, 0), q.len) : q.len;
}
// Tiles of a block, and of all blocks before it.  (More rows than positions:
// every block counts as the whole length.)
__device__ __forceinline__ int block_tiles(const AttnParams &p, const Seq &q, int block) {
  return tiles_for(p.causal && q.len >= q.n ? block_limit(p, q, block) : q.len);
}
__device__ long long tiles_before(const AttnParams &p, const Seq &q, int block) {
  if (!p.causal || q.len < q.n) return (long long)block * tiles_for(q.len);
  const int inner = min(block, q.blocks - 1);  // the last block may be cut short
  const long long g = p.group;
  long long sum = floor_sum(inner, kKeys * g, kCols, kCols - 1 + g * (q.len - q.n + kKeys));
  if (block > inner) sum += tiles_for(q.len);
  return sum;
}

struct Part {  // a part of an item: tiles [t0, t1) of tiles
  int seq, head, block, tiles, t0, t1;
  Seq q;
};

// The CTA's parts, one after another.  Each warp walks by itself; its state lies
// in shared memory, where lane 0 moves it on (in registers it would crowd out
// the tiles that are on their way).
struct Walk {
  long long at, end;
  Part x;
  __device__ __forceinline__ bool valid() const { return at < end; }
  __device__ void fit() { x.t1 = (int)min((long long)x.tiles, x.t0 + (end - at)); }
  __device__ void next(const AttnParams &p) {
    at += x.t1 - x.t0;
    if (at >= end) return;
    x.t0 = 0;
    if (++x.block == x.q.blocks) {
      x.block = 0;
      if (++x.head == p.c.heads) {
        x.head = 0;
        do x.q = seq_of(p, ++x.seq);
        while (x.q.blocks == 0);
      }
    }
    x.tiles = block_tiles(p, x.q, x.block);
    fit();
  }
  // key tiles that hold a key some column sees
  __device__ __forceinline__ int needed(const AttnParams &p) const {
    const int lim = block_limit(p, x.q, x.block);
    return max(0, min(x.t1, (lim + kKeys - 1) / kKeys) - x.t0);
  }
  __device__ __forceinline__ int cols(const AttnParams &p) const {
    return (int)min((long long)kCols, (long long)x.q.n * p.group - (long long)x.block * kCols);
  }
};

struct TileMeta {
  float ks[8], lv[8];    // per 16 keys: key scale, log2 of the value scale
  uint32_t hide[4];      // keys that no column sees (a page outside the pool)
  uint32_t nan[4];       // keys whose values hold a NaN code
};

template <int D>
struct Smem {
  uint8_t q[2][128 * D * 2];
  uint8_t k[kStagesKV][kKeys * D * 2];
  uint8_t v[kStagesKV][kKeys * D * 2];
  float cs[2][kCols];
  TileMeta meta[kMeta];
  int row[2][kMeta][8];  // keys', values': first row of each 16 keys in the pool, below 0: none
  uint64_t q_full, q_empty, k_full[kStagesKV], k_empty[kStagesKV], v_full[kStagesKV], v_empty[kStagesKV];
  uint64_t s_full[2], p_full[2], o_full[2], done;
  Walk walk[kThreads / 32];
  uint32_t tmem;
  int dead;
  int found_seq;
  long long found_at, scan[kThreads / 32];
};

__device__ __forceinline__ void step_on(const AttnParams &p, Walk &w) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) w.next(p);
  __syncwarp();
}

// ------------------------------------------------------------------ waits
template <int D>
__device__ __forceinline__ void wait(Smem<D> &sm, uint64_t *bar, uint32_t parity, int32_t *status) {
  if (mbar_try_wait(bar, parity)) return;
  unsigned long long t0 = 0;
  for (int i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if ((i & 15) == 15) {
      if (*reinterpret_cast<volatile int *>(&sm.dead)) return;
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitNs) {
        *reinterpret_cast<volatile int *>(&sm.dead) = 1;
        atomicOr(status, MQA_KV_DEV_WAIT_TIMEOUT);
        return;
      }
    }
  }
}

// ------------------------------------------------------------------ tcgen05
// K-major operand: 128-byte rows of 64 fp16, 8-row groups of 1024 bytes.
// MN-major (transposed) operand: the same bytes with the 64 contiguous values
// along N: 1024 bytes between groups of 8 k, `block` bytes between blocks of 64 n.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t block) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(block >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// kind::f16, fp16 x fp16 -> fp32.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <int R>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

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
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Byte offset of 16-byte chunk c (8 fp16) of row r in a [128][D] operand:
// halves of 64 values, rows of 128 bytes, chunks exchanged within 8 rows.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// ------------------------------------------------------------------ converters
// One group of 4 warps converts the keys, another the values; each also loads
// half of an item's queries.  A warp's load covers whole 128-byte lines; its
// lanes are laid out so that 8 of them store to 8 different bank groups (4
// chunks of two rows whose exchanges differ in the lowest bit).
template <int D, bool VALUES>
__device__ void convert_role(const AttnParams &p, Smem<D> &sm) {
  Walk &w = sm.walk[threadIdx.x >> 5];
  constexpr int CH = D / 16;              // 16-byte chunks of a code row
  constexpr int RPS = kConverters / CH;   // rows per step: 16 (D = 128) or 32
  constexpr int STEPS = kKeys / RPS;
  const int tid = threadIdx.x & (kConverters - 1), lane = tid & 31;
  const int ch = D == 128 ? (lane & 3) | (lane >> 4) << 2 : lane & 3;
  const int r0 = D == 128 ? (tid >> 5) * 4 + (lane >> 2 & 3) : (tid >> 5) * 8 + (lane >> 2);
  const int heads = p.c.heads;
  const uint8_t *codes = VALUES ? p.c.v : p.c.k;
  uint64_t *full = VALUES ? sm.v_full : sm.k_full, *empty = VALUES ? sm.v_empty : sm.k_empty;
  int(*rows)[8] = sm.row[VALUES];
  constexpr int kBar = kBarConv + VALUES;
  uint32_t tile_no = 0, q_no = 0;
  for (; w.valid(); step_on(p, w)) {
    const int nt = w.needed(p), ncols = w.cols(p);
    const int lim = block_limit(p, w.x.q, w.x.block), first = w.x.t0 * kKeys + tid * 16, head = w.x.head;
    const int32_t *table = p.c.table + (size_t)w.x.seq * p.c.max_pages;
    if (nt == 0) continue;  // softmax reads nothing either
    // lookups: threads 0 .. 7 hold 16 keys each, pages three tiles ahead, exponents two
    auto load_page = [&](int t) -> int {
      const int pos = first + t * kKeys;
      return tid < 8 && t < nt && pos < lim ? __ldg(table + (pos >> p.c.page_log2)) : -1;
    };
    auto row_of = [&](int t, int page) -> int {
      const int pos = first + t * kKeys;
      if (tid >= 8 || t >= nt || pos >= lim) return -2;  // nothing there
      if ((unsigned)page >= (unsigned)p.c.pages) {
        if (VALUES) atomicOr(p.c.status, MQA_KV_DEV_BAD_INDEX);
        return -1;
      }
      return ((page * heads + head) << p.c.page_log2) + (pos & (p.c.page - 1));
    };
    // nothing is computed from a loaded value before it is published, an iteration later
    uint32_t ke1 = 127, ve1 = 127;
    auto load_exps = [&](int row) {
      if (!VALUES || row < 0) return;
      const int ph = row >> p.c.page_log2;
      ke1 = __ldg(p.c.k_exps + ph);
      ve1 = __ldg(p.c.v_exps + ph);
    };
    auto publish = [&](uint32_t no, int row) {
      const int m = no % kMeta;
      if (tid < 8) {
        rows[m][tid] = row;
        if (VALUES) {
          sm.meta[m].ks[tid] = exp_byte(ke1);
          sm.meta[m].lv[tid] = (float)(int)ve1 - 127.f;
          const uint32_t bad = __ballot_sync(0xFFu, row == -1);
          if (tid < 4) {
            sm.meta[m].hide[tid] = (bad >> (2 * tid) & 1 ? 0xFFFFu : 0u) | (bad >> (2 * tid + 1) & 1 ? 0xFFFF0000u : 0u);
            sm.meta[m].nan[tid] = 0;
          }
        }
      }
    };
    uint4 x[STEPS];
    auto load = [&](uint32_t no, int i) {
      const int r = i * RPS + r0;
      const int row = rows[no % kMeta][r >> 4];
      x[i] = make_uint4(0, 0, 0, 0);
      if (row >= 0) x[i] = __ldg(reinterpret_cast<const uint4 *>(codes + (size_t)(row + (r & 15)) * D + ch * 16));
    };
    int pg2 = load_page(0);
    int row1 = row_of(0, pg2);
    load_exps(row1);
    pg2 = load_page(1);
    publish(tile_no, row1);
    row1 = row_of(1, pg2), load_exps(row1), pg2 = load_page(2);
    named_bar(kBar, kConverters);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) load(tile_no, i);

    for (int t = 0; t < nt; ++t, ++tile_no) {
      const int stage = tile_no % kStagesKV;
      const uint32_t round = tile_no / kStagesKV;
      if (t + 1 < nt) publish(tile_no + 1, row1);
      row1 = row_of(t + 2, pg2), load_exps(row1), pg2 = load_page(t + 3);
      named_bar(kBar, kConverters);
      wait(sm, &empty[stage], (round & 1) ^ 1, p.c.status);
      uint8_t *dst = VALUES ? sm.v[stage] : sm.k[stage];
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int r = i * RPS + r0;
        uint32_t ws[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        if (VALUES) {
          const uint32_t odd = nan_bytes(ws[0]) | nan_bytes(ws[1]) | nan_bytes(ws[2]) | nan_bytes(ws[3]);
          if (odd) {  // taken out here; the scores of the columns that see the key become NaN
            atomicOr(&sm.meta[tile_no % kMeta].nan[r >> 5], 1u << (r & 31));
#pragma unroll
            for (int b = 0; b < 4; ++b) ws[b] &= ~((nan_bytes(ws[b]) >> 7) * 255u);
          }
        }
        *reinterpret_cast<uint4 *>(dst + chunk_at(r, 2 * ch)) =
            make_uint4(cvt2(ws[0]), cvt2_hi(ws[0]), cvt2(ws[1]), cvt2_hi(ws[1]));
        *reinterpret_cast<uint4 *>(dst + chunk_at(r, 2 * ch + 1)) =
            make_uint4(cvt2(ws[2]), cvt2_hi(ws[2]), cvt2(ws[3]), cvt2_hi(ws[3]));
        if (t + 1 < nt) load(tile_no + 1, i);  // on its way while the rest is converted
      }
      fence_async_smem();
      mbar_arrive(&full[stage]);
      if (t == 0) {
        // ---- this group's 128 query rows (the previous part's last scores must be
        // done): 8 components per lane, a row's largest magnitude by exchange
        wait(sm, &sm.q_empty, (q_no & 1) ^ 1, p.c.status);
        constexpr int LPR = D / 8, QR = 32 / LPR;  // lanes per row, rows per warp step
        const int part = lane % LPR;
#pragma unroll 1
        for (int b = 0; b < 32 / QR; b += 8) {
          uint4 u[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = (tid >> 5) * 32 + (b + i) * QR + lane / LPR, col = VALUES * 128 + r;
            const int cc = w.x.block * kCols + col;
            u[i] = make_uint4(0, 0, 0, 0);
            if (col < ncols)
              u[i] = __ldg(reinterpret_cast<const uint4 *>(
                  reinterpret_cast<const uint16_t *>(p.q) + (size_t)(w.x.q.r0 + cc / p.group) * p.q_stride +
                  (size_t)(w.x.head * p.group + cc % p.group) * D + part * 8));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = (tid >> 5) * 32 + (b + i) * QR + lane / LPR;
            const uint32_t ws[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
            float2 f[4];
            float amax = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f[j] = p.bf16 ? bf16x2_to_float2(ws[j]) : half2_to_float2(ws[j]);
              amax = fmaxf(amax, fmaxf(fabsf(f[j].x), fabsf(f[j].y)));
            }
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
            int e = 0;
            if (amax > 0.f && amax <= FLT_MAX) e = 10 - exponent_of(amax);
            e = max(-100, min(100, e));
            const float up = pow2i(e);
            if (part == 0) sm.cs[q_no & 1][VALUES * 128 + r] = p.scale_log2 * pow2i(-e);
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = float2_to_half2(f[j].x * up, f[j].y * up);
            *reinterpret_cast<uint4 *>(sm.q[VALUES] + chunk_at(r, part)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        fence_async_smem();
        mbar_arrive(&sm.q_full);
      }
    }
    ++q_no;
  }
}

// ------------------------------------------------------------------ MMA issue
template <int D>
__device__ void mma_role(const AttnParams &p, Smem<D> &sm) {
  Walk &w = sm.walk[threadIdx.x >> 5];
  const uint32_t tmem = sm.tmem;
  const bool lead = (threadIdx.x & 31) == 0;
  constexpr uint32_t kQk = idesc_f16(128, kKeys, false), kPv = idesc_f16(128, D, true);
  uint32_t tile_no = 0, q_no = 0, p_no = 0;
  auto qk = [&](int x, int stage, bool on) {
    if (!lead) return;
    const uint32_t a = smem_u32(sm.q[x]), b = smem_u32(sm.k[stage]);
    if (on) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
        umma_ss(tmem + 256 + x * 128, sw128_kmajor_desc(a + off), sw128_kmajor_desc(b + off), kQk, kk > 0);
      }
    }
    umma_commit(&sm.s_full[x]);
  };
  auto pv = [&](int x, int stage, bool first) {
    if (!lead) return;
    const uint32_t b = smem_u32(sm.v[stage]);
#pragma unroll
    for (int kk = 0; kk < kKeys / 16; ++kk)
      umma_ts(tmem + x * 128, tmem + 256 + x * 128 + kk * 8, desc_mn(b + kk * 2048, 128 * 128), kPv,
              !first || kk > 0);
  };
  for (; w.valid(); step_on(p, w)) {
    const int nt = w.needed(p);
    const bool two = w.cols(p) > 128;
    if (nt == 0) continue;
    for (int t = -1; t < nt; ++t) {
      // scores of tile t + 1, weights times values of tile t
      const uint32_t kn = tile_no + t + 1, vn = tile_no + t;
      const int ks = kn % kStagesKV, vs = vn % kStagesKV;
      const bool more = t + 1 < nt;
      if (more) wait(sm, &sm.k_full[ks], kn / kStagesKV & 1, p.c.status);
      if (t < 0) wait(sm, &sm.q_full, q_no & 1, p.c.status);
      else wait(sm, &sm.v_full[vs], vn / kStagesKV & 1, p.c.status);
      for (int x = 0; x < 2; ++x) {
        const bool on = x == 0 || two;
        if (t >= 0) {
          wait(sm, &sm.p_full[x], p_no++ >> 1 & 1, p.c.status);
          __syncwarp();
          tc_fence_after();
          if (on) pv(x, vs, t == 0);
          if (on && !more && lead) umma_commit(&sm.o_full[x]);
        }
        tc_fence_after();
        if (more) qk(x, ks, on);
      }
      if (lead) {
        if (t >= 0) umma_commit(&sm.v_empty[vs]);
        if (more) umma_commit(&sm.k_empty[ks]);
        if (t + 2 == nt) umma_commit(&sm.q_empty);  // the last scores are under way
      }
      __syncwarp();
    }
    tile_no += nt;
    ++q_no;
  }
  if (lead) {
    umma_commit(&sm.done);
    wait(sm, &sm.done, 0, p.c.status);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ softmax
// How a tile's scores are read: as they are; cut at the keys the column sees;
// or with every rare case (pages outside the pool, NaN values, scales far apart).
enum Mode { kPlain, kCut, kRare };

template <int MODE>
__device__ __forceinline__ void hide_keys(uint32_t (&s)[32], const TileMeta &meta, int j, int room) {
  if (MODE == kPlain) return;
  if (MODE == kRare) {
    const uint32_t hide = meta.hide[j], nan = meta.nan[j];
#pragma unroll
    for (int b = 0; b < 32; ++b) {
      if (nan >> b & 1) s[b] = 0x7FC00000u;
      if (hide >> b & 1) s[b] = 0xFF800000u;  // -inf
    }
  }
  const int n = room - 32 * j;
#pragma unroll
  for (int b = 0; b < 32; ++b)
    if (b >= n) s[b] = 0xFF800000u;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, uint32_t c) { return max3(a, b, __uint_as_float(c)); }
__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
  return max3(__uint_as_float(a), __uint_as_float(b), c);
}

// A column's largest score of the tile, and largest score plus value exponent.
// The next 32 columns are on their way from TMEM while 32 are looked at.
template <int MODE>
__device__ __forceinline__ void scan_scores(uint32_t ts, const TileMeta &meta, int room, float cs, float &top,
                                            float &topw) {
  auto look = [&](uint32_t(&s)[32], int j) {
    hide_keys<MODE>(s, meta, j, room);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint32_t *v = s + 16 * g;
      const float a = max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), v[6]);
      const float b = max3(max3(v[7], v[8], v[9]), max3(v[10], v[11], v[12]), v[13]);
      const float x = max3(fmaxf(a, __uint_as_float(v[14])), b, v[15]) * (cs * meta.ks[2 * j + g]);
      top = fmaxf(top, x);
      topw = fmaxf(topw, x + meta.lv[2 * j + g]);
    }
  };
  uint32_t s0[32], s1[32];
  tmem_ld_32x32b_x32(ts, s0);
#pragma unroll 1
  for (int j = 0; j < 4; j += 2) {
    tmem_ld_wait();
    tmem_ld_32x32b_x32(ts + 32 * j + 32, s1);
    look(s0, j);
    tmem_ld_wait();
    if (j == 0) tmem_ld_32x32b_x32(ts + 64, s0);
    look(s1, j + 1);
  }
}

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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Scores to weights, in place (fp16 over the first half of the fp32 columns);
// returns the column's sum with this tile's.  A weight in the sum is 2^back of
// the one that enters the product.
template <int MODE>
__device__ __forceinline__ float weigh(uint32_t ts, const TileMeta &meta, int room, float cs, float mr, float ww,
                                       float l) {
  auto turn = [&](uint32_t(&s)[32], int j) {
    hide_keys<MODE>(s, meta, j, room);
    uint32_t h[16];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float f = cs * meta.ks[2 * j + g], lv = meta.lv[2 * j + g];
      const float b = lv - ww, back = ww - lv - mr;
      const uint64_t f2 = pack2(f, f), b2 = pack2(b, b);
      if (MODE == kRare && back > 64.f) {
#pragma unroll
        for (int k = 0; k < 16; ++k) l += ex2(__uint_as_float(s[16 * g + k]) * f - mr);
      }
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float y, z;
        unpack2(fma2(pack2(__uint_as_float(s[16 * g + 2 * k]), __uint_as_float(s[16 * g + 2 * k + 1])), f2, b2), y, z);
        y = ex2(y), z = ex2(z);
        sum[k & 1] = add2(sum[k & 1], pack2(y, z));
        h[8 * g + k] = float2_to_half2(y, z);
      }
      float y, z;
      unpack2(add2(sum[0], sum[1]), y, z);
      if (MODE != kRare || !(back > 64.f)) l = fmaf(y + z, ex2(back), l);
    }
    tmem_st16(ts + 16 * j, h);
  };
  uint32_t s0[32], s1[32];
  tmem_ld_32x32b_x32(ts, s0);
#pragma unroll 1
  for (int j = 0; j < 4; j += 2) {
    tmem_ld_wait();
    tmem_ld_32x32b_x32(ts + 32 * j + 32, s1);
    turn(s0, j);
    tmem_ld_wait();
    if (j == 0) tmem_ld_32x32b_x32(ts + 64, s0);
    turn(s1, j + 1);
  }
  return l;
}

template <int D>
__device__ void softmax_role(const AttnParams &p, Smem<D> &sm, long long per) {
  Walk &w = sm.walk[threadIdx.x >> 5];
  const int x = threadIdx.x >> 7;        // tile of columns
  const int r = threadIdx.x & 127;       // its column
  const uint32_t lanes = (uint32_t)(r & ~31) << 16;
  const uint32_t ts = sm.tmem + 256 + x * 128 + lanes, to = sm.tmem + x * 128 + lanes;
  uint32_t tile_no = 0, q_no = 0, s_no = 0, o_no = 0;
  for (; w.valid(); step_on(p, w)) {
    const int nt = w.needed(p), ncols = w.cols(p);
    const int col = x * 128 + r;
    if (ncols <= x * 128) {  // this half is empty: it keeps step, so that it meets every phase of the barriers
      if (nt) wait(sm, &sm.q_full, q_no++ & 1, p.c.status);
      for (int t = 0; t < nt; ++t, ++tile_no) {
        wait(sm, &sm.v_full[tile_no % kStagesKV], tile_no / kStagesKV & 1, p.c.status);
        wait(sm, &sm.s_full[x], s_no++ & 1, p.c.status);  // without it this half could run ahead of the issuing warp
        mbar_arrive(&sm.p_full[x]);
      }
      continue;
    }
    const int c = w.x.block * kCols + col;
    const int i = c / p.group;
    const int lim = col < ncols ? (p.causal ? min(max(w.x.q.len - w.x.q.n + i + 1, 0), w.x.q.len) : w.x.q.len) : 0;
    float m = -INFINITY, wr = -INFINITY, l = 0.f;
    float cs = 0.f;
    const int room0 = lim - w.x.t0 * kKeys;
    if (nt) {
      wait(sm, &sm.q_full, q_no & 1, p.c.status);
      cs = sm.cs[q_no & 1][col];
      ++q_no;
    }
    for (int t = 0; t < nt; ++t, ++tile_no) {
      const int stage = tile_no % kStagesKV;
      wait(sm, &sm.v_full[stage], tile_no / kStagesKV & 1, p.c.status);
      wait(sm, &sm.s_full[x], s_no++ & 1, p.c.status);
      __syncwarp();
      tc_fence_after();
      const TileMeta &meta = sm.meta[tile_no % kMeta];
      const int room = room0 - t * kKeys;  // keys of the tile that the column sees
      uint32_t odd = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) odd |= meta.hide[j] | meta.nan[j];
      const bool cut = __any_sync(~0u, room < kKeys);
      // largest score, and largest score with the value scale
      float top = -INFINITY, topw = -INFINITY;
      if (odd) scan_scores<kRare>(ts, meta, room, cs, top, topw);
      else if (cut) scan_scores<kCut>(ts, meta, room, cs, top, topw);
      else scan_scores<kPlain>(ts, meta, room, cs, top, topw);
      const bool move = top > m + kSlack || topw > wr + kSlack;
      if (__any_sync(~0u, move)) {
        const float mn = fmaxf(m, top), wn = fmaxf(wr, topw);
        const float fl = mn == m ? 1.f : ex2(m - mn), fo = wn == wr ? 1.f : ex2(wr - wn);
        m = mn, wr = wn;
        l *= fl;
        if (t > 0) {
#pragma unroll 1
          for (int j = 0; j < D; j += 16) {
            uint32_t o[16];
            tmem_ld16(to + j, o);
            tmem_ld_wait();
#pragma unroll
            for (int b = 0; b < 16; ++b) o[b] = __float_as_uint(__uint_as_float(o[b]) * fo);
            tmem_st16(to + j, o);
          }
        }
      }
      const float mr = m == -INFINITY ? 0.f : m, ww = wr == -INFINITY ? 0.f : wr;
      // values so small that their weights would leave fp32's range before they
      // are scaled back: the sum takes a power of two of its own
      bool far = false;
#pragma unroll
      for (int g = 0; g < 8; ++g) far |= ww - meta.lv[g] - mr > 64.f;
      if (odd || __any_sync(~0u, far)) l = weigh<kRare>(ts, meta, room, cs, mr, ww, l);
      else if (cut) l = weigh<kCut>(ts, meta, room, cs, mr, ww, l);
      else l = weigh<kPlain>(ts, meta, room, cs, mr, ww, l);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sm.p_full[x]);
    }
    // ---- the part's result
    if (nt) {
      wait(sm, &sm.o_full[x], o_no++ & 1, p.c.status);
      __syncwarp();
      tc_fence_after();
    }
    const bool whole = w.x.t0 == 0 && w.x.t1 == w.x.tiles;
    const bool none = m == -INFINITY && l == 0.f;
    const float f = none ? 0.f : l != l ? NAN : ex2(wr - m) / l;
    const int row = w.x.q.r0 + i, head = w.x.head * p.group + c % p.group;
    float *slot = p.slots + ((size_t)blockIdx.x * 2 + (w.x.t0 == 0 ? 1 : 0)) * ((size_t)kCols * (D + 4));
    uint4 *out = reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p.out) + ((size_t)row * p.q_heads + head) * D);
#pragma unroll 1
    for (int j = 0; j < D; j += 16) {
      uint32_t o[16];
      if (nt) {
        tmem_ld16(to + j, o);
        tmem_ld_wait();
      }
#pragma unroll
      for (int b = 0; b < 16; ++b) o[b] = none ? 0u : o[b];
      if (col < ncols) {
        if (whole) {
          uint32_t h[8];
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const float y = __uint_as_float(o[2 * b]) * f, z = __uint_as_float(o[2 * b + 1]) * f;
            h[b] = none ? 0u : p.bf16 ? float2_to_bf162(y, z) : float2_to_half2(y, z);
          }
          out[j / 8] = make_uint4(h[0], h[1], h[2], h[3]);
          out[j / 8 + 1] = make_uint4(h[4], h[5], h[6], h[7]);
        } else {
          float4 *d = reinterpret_cast<float4 *>(slot + (size_t)col * D + j);
#pragma unroll
          for (int b = 0; b < 4; ++b)
            d[b] = make_float4(__uint_as_float(o[4 * b]), __uint_as_float(o[4 * b + 1]), __uint_as_float(o[4 * b + 2]),
                               __uint_as_float(o[4 * b + 3]));
        }
      }
    }
    if (col < ncols) {
      if (whole) {
        if (p.lse)
          p.lse[(size_t)row * p.q_heads + head] = none ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
      } else {
        slot[(size_t)kCols * D + col] = m;
        slot[(size_t)kCols * D + kCols + col] = wr;
        slot[(size_t)kCols * D + 2 * kCols + col] = l;
      }
    }
    if (threadIdx.x == 0 && !whole && w.x.t0 == 0) {
      const long long rest = w.x.tiles - (w.x.t1 - w.x.t0);
      p.desc[blockIdx.x] = make_int4(w.x.q.r0, w.x.head, w.x.block * kCols,
                                     (int)((rest + per - 1) / per) | ncols << 20);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(const AttnParams p) {
  extern __shared__ uint8_t raw[];
  Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw + ((1024 - (smem_u32(raw) & 1023)) & 1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // ---- this CTA's part of the line
  const int per_thread = (p.c.seqs + kThreads - 1) / kThreads;
  long long mine = 0;
  for (int i = 0; i < per_thread; ++i) {
    const int s = tid * per_thread + i;
    if (s >= p.c.seqs) break;
    const Seq q = seq_of(p, s);
    if (q.blocks) mine += p.c.heads * tiles_before(p, q, q.blocks);
    if (blockIdx.x == 0 && p.c.lens[s] != q.len) atomicOr(p.c.status, MQA_KV_DEV_BAD_LENGTH);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  long long total = 0, before = incl - mine;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += sm.scan[i];
    total += sm.scan[i];
  }
  const long long per = max((total + gridDim.x - 1) / gridDim.x, (long long)kTiledMinTiles);
  Walk w;
  w.at = blockIdx.x * per;
  w.end = min(total, w.at + per);
  if (tid == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (w.at >= w.end) return;  // the whole CTA leaves together
  if (w.at >= before && w.at < before + mine) {
    long long b = before;
    for (int i = 0; i < per_thread; ++i) {
      const int s = tid * per_thread + i;
      const Seq q = seq_of(p, s);
      const long long u = q.blocks ? p.c.heads * tiles_before(p, q, q.blocks) : 0;
      if (w.at < b + u) {
        sm.found_seq = s;
        sm.found_at = w.at - b;
        break;
      }
      b += u;
    }
  }
  if (tid == 0) {
    sm.dead = 0;
    mbar_init(&sm.q_full, 2 * kConverters);
    mbar_init(&sm.q_empty, 1);
    for (int i = 0; i < kStagesKV; ++i) {
      mbar_init(&sm.k_full[i], kConverters);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], kConverters);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 128);
      mbar_init(&sm.o_full[i], 1);
    }
    mbar_init(&sm.done, 1);
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  {
    w.x.seq = sm.found_seq;
    w.x.q = seq_of(p, w.x.seq);
    const long long per_head = tiles_before(p, w.x.q, w.x.q.blocks);
    w.x.head = (int)(sm.found_at / per_head);
    const long long rest = sm.found_at - w.x.head * per_head;
    int lo = 0, hi = w.x.q.blocks;  // the last block that begins at or before `rest`
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tiles_before(p, w.x.q, mid) <= rest) lo = mid; else hi = mid;
    }
    w.x.block = lo;
    w.x.tiles = block_tiles(p, w.x.q, lo);
    w.x.t0 = (int)(rest - tiles_before(p, w.x.q, lo));
    w.fit();
  }
  if (lane == 0) sm.walk[warp] = w;
  __syncwarp();
  // registers: 256 x 128 + 256 x 88 + 128 x 48 = 640 x 96, what the block was launched with
  if (warp < 8) {
    reg_inc<128>();
    softmax_role<D>(p, sm, per);
  } else if (warp < 12) {
    reg_dec<88>();
    convert_role<D, false>(p, sm);
  } else if (warp < 16) {
    reg_dec<88>();
    convert_role<D, true>(p, sm);
  } else {
    reg_dec<48>();
    if (warp == 16) mma_role<D>(p, sm);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) tmem_dealloc(sm.tmem, 512);
}

// Join split items: block (c, y) adds the parts of 32 columns of the item that
// CTA c began; a warp per column in turn.
template <int D>
__global__ void __launch_bounds__(256) kv_prefill_join_kernel(const AttnParams p) {
  const int4 d = p.desc[blockIdx.x];
  const int more = d.w & 0xFFFFF, ncols = d.w >> 20;
  if (more == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float acc[8][D];
  constexpr size_t pitch = (size_t)kCols * (D + 4);
  auto slot = [&](int i) { return p.slots + ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * pitch; };
  for (int col = blockIdx.y * 32 + warp; col < min(ncols, (int)blockIdx.y * 32 + 32); col += 8) {
    float mx = -INFINITY, wx = -INFINITY, ls = 0.f, o[D / 32];
    for (int i = lane; i <= more; i += 32) {
      const float *s = slot(i) + (size_t)kCols * D;
      mx = fmaxf(mx, s[col]);
      wx = fmaxf(wx, s[kCols + col]);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, k));
      wx = fmaxf(wx, __shfl_xor_sync(~0u, wx, k));
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int i = 0; i <= more; ++i) {
      const float *s = slot(i), *t = s + (size_t)kCols * D;
      const float m = t[col], w = t[kCols + col];
      ls += t[2 * kCols + col] * (m == mx ? 1.f : ex2(m - mx));
      const float f = w == wx ? 1.f : ex2(w - wx);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] += f * s[(size_t)col * D + lane + 32 * e];
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[warp][lane + 32 * e] = o[e];
    __syncwarp();
    const int c = d.z + col;
    finish<D>(p, d.x + c / p.group, d.y * p.group + c % p.group, lane, acc[warp], mx, wx, ls);
    __syncwarp();
  }
}

template <int D>
cudaError_t launch(const AttnParams &p, int ctas, cudaStream_t stream) {
  constexpr int bytes = (int)sizeof(Smem<D>) + 1024;
  auto *k = kv_prefill_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  k<<<ctas, kThreads, bytes, stream>>>(p);
  const cudaError_t le = cudaGetLastError();
  if (le != cudaSuccess) return le;
  kv_prefill_join_kernel<D><<<dim3(ctas, kCols / 32), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_prefill(const AttnParams &p, int ctas, cudaStream_t stream) {
  return p.c.dim == 64 ? launch<64>(p, ctas, stream) : launch<128>(p, ctas, stream);
}

}  // namespace mqa
