// Attention over the paged 8-bit cache for many query columns per key/value
// head (prompts and their chunks) on the tcgen05 tensor cores.
// (include/mqakv.h, mqa_kv_attention; the mathematics is kv_attn.cu's.)
//
// A CTA holds 256 columns of an item (query row x query head of one key/value
// head) as two 128-row halves and walks over 128-key tiles:
//     S = Q K^T (kind::f8f6f4: the keys' codes as they lie in the pool, brought
//         by TMA; each query value as a sum of e4m3 terms, below; S fp32 in TMEM),
//     P = 2^(s + lv - w) rounded to fp16, written back over S in TMEM,
//     O += P V (kind::f16: P from TMEM, V converted to fp16 in shared memory, O
//         fp32 in TMEM).
// Query terms: a row is multiplied by the power of two that brings its largest
// magnitude to (224, 448]; x = t1 + t2 (+ t3), each term the e4m3 rounding of
// what is left.  Two terms hold a bf16's 8 bits and three an fp16's 11 exactly,
// down to e4m3's smallest step of 2^-9: what is lost is at most 2^-10 of 224,
// 2^-17.8 of the row's largest value, and only in values below 2^-10 (bf16) or
// 2^-7 (fp16) of it.  The products with two terms take as long as one fp16
// product would, and no key has to be converted or stored twice.
// While one half's scores are turned into weights the tensor cores work on the
// other half.  Roles: 2 x 4 softmax warps (a thread per column; it also moves
// its references and rescales its row of O when a score passes them too far),
// 4 converter warps (values to fp16, which the MMA reads transposed), one warp
// that looks pages up and issues the queries' and keys' copies, one that issues
// the MMAs.  The query terms are formed once per call by a kernel of their own
// (in the main kernel they cost 20,000 cycles per item), laid out so that an
// item's columns are consecutive rows.
// Every wait has a time limit; once one has run out, all of them return at
// once: the lookup warp leaves after the copies it has under way, and the other
// roles run to their end on whatever they find in shared memory (rows are
// checked before they are read).
//
// What bounds it: a half's chain of weights (about 1,750 cycles for 128 x 128),
// their product and the next scores (1,024), 3,100 cycles per tile with its
// waits, against 2,048 of both halves' MMAs.  (Scores of 64 keys per MMA, the
// upper ones ahead of the product, would break the chain, but then the queries
// are read from shared memory twice as often: 894 us instead of 718.)
// 2,048 rows at the end of 32K positions (32 heads, 8 key/value heads of 128):
// 735 to 745 us a pass, 1.43 to 1.45 PFLOP/s, 74% of the measured bf16 rate; fp16
// queries, whose third term lengthens the scores' product by half, 831 us in a
// run where bf16 took 725.  Five prompts of up to 1,531 rows: 90 us, of which 13
// for the query terms, 5 to find the parts, 7 until the first scores are there, 9
// to join.
//
// Work is cut like kv_attn.cu's: the key tiles of all items in one line, even
// parts per CTA, partial results in two slots per CTA and a joining pass.  The
// position of a part is found from the exact number of tiles that causal
// column blocks need (a sum of floors).
#include "kv_ptx.cuh"

#include <cfloat>

namespace mqa {

namespace {

constexpr int kThreads = 512;
constexpr int kKeys = 128;                // keys per tile
constexpr int kCols = kTiledCols;         // columns per item
constexpr int kStagesK = 3, kStagesV = 2;
constexpr int kMeta = 8;                  // tile descriptions in flight
constexpr int kTerms = kQueryTerms;       // e4m3 terms of a query value (bf16: 2)
// Tiles by which a part's end may move to its item's: partial results and their
// joining cost about as much.  (Up to an eighth of the part made the chunk of 32K
// positions 16% slower, for want of balance.)
constexpr int kNear = 2;
constexpr int kConverters = 128;

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

// Where an end of a CTA's part lies: `off` tiles into the item of x.
struct Cut {
  Part x;
  int off;
};

struct TileMeta {
  float2 kv[8];          // per 16 keys: key scale, log2 of the value scale
  float lv_min;          // least of the latter,
  float spread;          // and how far it lies below the largest of the part so far
  uint32_t odd;          // nonzero where hide or nan is
  uint32_t hide[4];      // keys that no column sees (a page outside the pool)
  uint32_t nan[4];       // keys whose values hold a NaN code
  int row[8];            // first row of each 16 keys in the pool; -1: page outside the pool, -2: no key needed
};


template <int D, bool TEST>
struct Smem {
  static constexpr bool test = TEST;
  uint8_t q[2][kTerms][128 * D];
  uint8_t k[kStagesK][kKeys * D];
  uint8_t v[kStagesV][kKeys * D * 2];
  TileMeta meta[kMeta];
  uint64_t q_full, q_empty, k_full[kStagesK], k_empty[kStagesK], v_full[kStagesV], v_empty[kStagesV];
  uint64_t m_full[kMeta], m_empty[kMeta], n_full[kMeta], s_full[2], p_full[2], o_full[2], done;
  uint64_t never[kStagesK];  // tests: nothing arrives here
  Walk walk[kThreads / 32];
  uint32_t tmem;
  int dead;
  int found_seq[2];
  long long found_at[2], found_per_head[2], scan[kThreads / 32];
  Cut cut[2];
};

__device__ __forceinline__ void step_on(const AttnParams &p, Walk &w) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) w.next(p);
  __syncwarp();
}

// ------------------------------------------------------------------ tcgen05
// Shared-memory operand descriptors, in two words.  The low one is the address
// in units of 16 bytes and the leading byte offset; it is all that changes from
// one MMA to the next.  High word: stride byte offset, version, swizzle.
//  codes (K-major): rows of D bytes (128: 128-byte swizzle, 64: 64-byte swizzle),
//  8-row groups;
//  values (transposed): 128-byte rows of 64 fp16 along N, 1024 bytes between
//  groups of 8 k, 128 * 128 bytes between blocks of 64 n.
template <int D>
struct Desc {
  static constexpr uint32_t codes_hi = ((8u * D) >> 4) | 1u << 14 | (D == 128 ? 2u : 4u) << 29;
  static constexpr uint32_t values_hi = (1024u >> 4) | 1u << 14 | 2u << 29;
  static __device__ __forceinline__ uint32_t codes_lo(const void *p) {
    return ((smem_u32(p) & 0x3FFFFu) >> 4) | 1u << 16;
  }
  static __device__ __forceinline__ uint32_t values_lo(const void *p) {
    return ((smem_u32(p) & 0x3FFFFu) >> 4) | (128u * 128 >> 4) << 16;
  }
};
// kind::f16, fp16 x fp16 -> fp32.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void umma_codes(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, "
      "%3};\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_weights(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                             uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

__device__ __forceinline__ void store32(void *p, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(__cvta_generic_to_global(p)), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// 32 bytes of the caller's rows.  `out` is 16-byte aligned; where it is 32-byte
// aligned (rows are a multiple of 32 bytes), one store writes a whole sector: ragged
// prompts of up to 1,531 rows take 87.4 us so, and 94.9 in two stores of 16 bytes.
__device__ __forceinline__ void store_out(uint8_t *p, const uint32_t *v, bool wide) {
  if (wide) {
    store32(p, v);
  } else {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
template <int R>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}


// Byte offset of 16-byte chunk c (8 fp16) of row r in a [128][D] operand:
// halves of 64 values, rows of 128 bytes, chunks exchanged within 8 rows.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Byte offset of 16-byte chunk c of row r in a [128][D] operand of codes.
template <int D>
__device__ __forceinline__ uint32_t code_at(int r, int c) {
  return (uint32_t)(r * D + ((c ^ (D == 128 ? r & 7 : r >> 1 & 3)) << 4));
}

// ------------------------------------------------------------------ lookups and key copies
// Four tiles at a time (lane = tile x 16 keys): page, row in the pool and
// scales; then, tile by tile, the description and the keys' copies, one box
// per page.
template <int D, bool TEST>
__device__ void lookup_role(const AttnParams &p, const CUtensorMap &map, const CUtensorMap &q_map, Smem<D, TEST> &sm) {
  Walk &w = sm.walk[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31, g = lane & 7, heads = p.c.heads;
  const int box = min(p.c.page, kKeys), per_box = box >> 4;
  uint32_t tile_no = 0, q_no = 0;
  const uint64_t keep = policy_evict_last(), once = policy_evict_first();  // other CTAs read the same keys
  const int terms = p.bf16 ? 2 : 3, planes = p.rows * p.group;  // rows of a head in a term's plane
  auto walk = [&] {
    for (; w.valid(); step_on(p, w)) {
      const int nt = w.needed(p);
      const int lim = block_limit(p, w.x.q, w.x.block), first = w.x.t0 * kKeys + g * 16, head = w.x.head;
      const int32_t *table = p.c.table + (size_t)w.x.seq * p.c.max_pages;
      float lv_max = -128.f;
      auto ask = [&] {  // the part's queries
        const int halves = w.cols(p) > 128 ? 2 : 1, at = w.x.q.r0 * p.group + w.x.block * kCols;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&sm.q_full, (uint32_t)(terms * halves * 128 * D));
        __syncwarp();
        if (lane < terms * halves) {
          const int x = lane / terms, term = lane % terms;
          tma_load_2d(sm.q[x][term], &q_map, &sm.q_full, 0, (term * heads + head) * planes + at + 128 * x, once);
        }
        ++q_no;
      };
      const bool begins = q_no == 0;
      if (begins && nt > 0) ask();  // the first part's before anything is looked up
      for (int tb = 0; tb < nt; tb += 4) {
        const int t = tb + (lane >> 3), pos = first + t * kKeys;
        int row = -2;
        float ks = 1.f, lv = 0.f;
        if (t < nt && pos < lim) {
          const int page = __ldg(table + (pos >> p.c.page_log2));
          if ((unsigned)page < (unsigned)p.c.pages) {
            const int ph = page * heads + head;
            row = (ph << p.c.page_log2) + (pos & (p.c.page - 1));
            ks = exp_byte(__ldg(p.c.k_exps + ph));
            lv = (float)(int)__ldg(p.c.v_exps + ph) - 127.f;
          } else {
            row = -1;
            atomicOr(p.c.status, MQA_KV_DEV_BAD_INDEX);
          }
        }
        float lv_min = lv;  // of the tile; groups that hold no key do not count
        if (row < 0) lv_min = 128.f;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) lv_min = fminf(lv_min, __shfl_xor_sync(~0u, lv_min, o));
        lv_max = fmaxf(lv_max, row < 0 ? -128.f : lv);  // over four tiles at once: never less than it must be
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) lv_max = fmaxf(lv_max, __shfl_xor_sync(~0u, lv_max, o));
        const uint32_t bad = __ballot_sync(~0u, row == -1);
        const uint32_t copies = __ballot_sync(~0u, row >= 0 && g % per_box == 0);
        for (int u = 0; u < min(4, nt - tb); ++u, ++tile_no) {
          const int slot = tile_no % kMeta, stage = tile_no % kStagesK;
          if (!warp_wait(sm, &sm.m_empty[slot], (tile_no / kMeta & 1) ^ 1, p)) return;
          TileMeta &meta = sm.meta[slot];
          if (lane >> 3 == u) {
            meta.row[g] = row;
            meta.kv[g] = make_float2(ks, lv);
            if (g < 4) {
              const uint32_t two = bad >> (8 * u + 2 * g);
              meta.hide[g] = (two & 1 ? 0xFFFFu : 0u) | (two & 2 ? 0xFFFF0000u : 0u);
              meta.nan[g] = 0;
            }
            if (g == 0) {
              meta.lv_min = lv_min;
              meta.spread = lv_max - lv_min;
              meta.odd = (bad >> (8 * u) & 255u) != 0;
            }
          }
          const uint32_t mine = copies >> (8 * u) & 255u;
          if (!warp_wait(sm, &sm.k_empty[stage], (tile_no / kStagesK & 1) ^ 1, p)) return;
          if (lane == 0) {
            mbar_arrive(&sm.m_full[slot]);
            mbar_arrive_expect_tx(&sm.k_full[stage], (uint32_t)(__popc(mine) * box * D));
          }
          __syncwarp();
          if (lane >> 3 == u && (mine >> g & 1))
            tma_load_2d(sm.k[stage] + g * 16 * D, &map, &sm.k_full[stage], 0, row, keep);
          if (tb + u == 0 && !begins) {  // once the previous part's last scores are done
            if (!warp_wait(sm, &sm.q_empty, (q_no & 1) ^ 1, p)) {
              ++tile_no;  // its copies are under way
              return;
            }
            ask();
          }
        }
      }
    }
  };
  if (!TEST || p.stall != 2 || warp_wait(sm, &sm.never[0], 0, p)) walk();
  // the copies must have landed before the CTA leaves
  if (q_no) drain(&sm.q_full, (q_no - 1) & 1);
  for (int i = 1; i <= kStagesK; ++i)
    if (tile_no >= (uint32_t)i) drain(&sm.k_full[(tile_no - i) % kStagesK], (tile_no - i) / kStagesK & 1);
  __syncwarp();
}

// ------------------------------------------------------------------ converters
template <int STEPS, int RPS>
__device__ void take_nan_out(uint4 (&x)[STEPS], TileMeta &meta, int r0) {
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    uint32_t *w = &x[i].x;
    uint32_t odd = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t n = nan_bytes(w[b]);
      odd |= n;
      w[b] &= ~((n >> 7) * 255u);
    }
    if (odd) {
      const int r = i * RPS + r0;
      atomicOr(&meta.nan[r >> 5], 1u << (r & 31));
      meta.odd = 1;
    }
  }
}
// A warp's load covers whole 128-byte lines; its lanes are laid out so that 8
// of them store to 8 different bank groups (4 chunks of two rows whose
// exchanges differ in the lowest bit).
template <int D, bool TEST>
__device__ void convert_role(const AttnParams &p, Smem<D, TEST> &sm) {
  Walk &w = sm.walk[threadIdx.x >> 5];
  constexpr int CH = D / 16;              // 16-byte chunks of a code row
  constexpr int RPS = kConverters / CH;   // rows per step: 16 (D = 128) or 32
  constexpr int STEPS = kKeys / RPS;
  const int tid = threadIdx.x & (kConverters - 1), lane = tid & 31;
  const int ch = D == 128 ? (lane & 3) | (lane >> 4) << 2 : lane & 3;
  const int r0 = D == 128 ? (tid >> 5) * 4 + (lane >> 2 & 3) : (tid >> 5) * 8 + (lane >> 2);
  const uint32_t last_row = ((uint32_t)p.c.pages * p.c.heads << p.c.page_log2) - 16;  // begins the pool's last 16 rows
  uint32_t tile_no = 0;
  uint4 x[STEPS];
  auto load = [&](uint32_t no, int i) {
    const int r = i * RPS + r0;
    const int row = sm.meta[no % kMeta].row[r >> 4];
    x[i] = make_uint4(0, 0, 0, 0);
    // (past the L1, of which shared memory leaves little: spills live there, and the
    // chunk of 32K positions takes 799 us so and 920 with loads that allocate in it)
    if ((uint32_t)row <= last_row)
      x[i] = __ldcg(reinterpret_cast<const uint4 *>(p.c.v + (size_t)(row + (r & 15)) * D + ch * 16));
  };
  for (; w.valid(); step_on(p, w)) {
    const int nt = w.needed(p);
    if (nt == 0) continue;  // nothing is read
    bounded_wait(sm, &sm.m_full[tile_no % kMeta], tile_no / kMeta & 1, p);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) load(tile_no, i);

    for (int t = 0; t < nt; ++t, ++tile_no) {
      const int stage = tile_no % kStagesV;
      // NaN codes are taken out; the scores of the columns that see their key become
      // NaN.  The softmax waits for this, not for the stage.
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        any |= nan_bytes(x[i].x) | nan_bytes(x[i].y) | nan_bytes(x[i].z) | nan_bytes(x[i].w);
      if (any) take_nan_out<STEPS, RPS>(x, sm.meta[tile_no % kMeta], r0);
      mbar_arrive(&sm.n_full[tile_no % kMeta]);
      if (t + 1 < nt) bounded_wait(sm, &sm.m_full[(tile_no + 1) % kMeta], (tile_no + 1) / kMeta & 1, p);
      bounded_wait(sm, &sm.v_empty[stage], (tile_no / kStagesV & 1) ^ 1, p);
      uint8_t *dst = sm.v[stage];
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int r = i * RPS + r0;
        const uint32_t ws[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        *reinterpret_cast<uint4 *>(dst + chunk_at(r, 2 * ch)) =
            make_uint4(cvt2(ws[0]), cvt2_hi(ws[0]), cvt2(ws[1]), cvt2_hi(ws[1]));
        *reinterpret_cast<uint4 *>(dst + chunk_at(r, 2 * ch + 1)) =
            make_uint4(cvt2(ws[2]), cvt2_hi(ws[2]), cvt2(ws[3]), cvt2_hi(ws[3]));
        if (t + 1 < nt) load(tile_no + 1, i);  // on its way while the rest is converted
      }
      fence_async_smem();
      mbar_arrive(&sm.v_full[stage]);
    }
  }
}

// ------------------------------------------------------------------ MMA issue
// The warp waits together, one elected lane issues, and the others wait for it
// before the next barrier: lanes that poll hold up the one that issues.
template <int D, bool TEST>
__device__ void mma_role(const AttnParams &p, Smem<D, TEST> &sm) {
  Walk &w = sm.walk[threadIdx.x >> 5];
  const uint32_t tmem = sm.tmem;
  constexpr uint32_t kQk = idesc_f8_e4m3_f32(128, kKeys), kPv = idesc_f16(128, D, true);
  const int terms = p.bf16 ? 2 : 3;
  uint64_t *const k_full = TEST && p.stall == 1 ? sm.never : sm.k_full;
  uint32_t tile_no = 0, q_no = 0, p_no = 0;
  const uint32_t q0 = Desc<D>::codes_lo(sm.q[0][0]), k0 = Desc<D>::codes_lo(sm.k[0]),
                 v0 = Desc<D>::values_lo(sm.v[0]);
  auto qk = [&](int x, int stage) {
    uint32_t a = q0 + x * (kTerms * 128 * D / 16);
    const uint32_t b = k0 + stage * (kKeys * D / 16), d = tmem + 256 + x * 128;
#pragma unroll 1
    for (int term = 0; term < terms; ++term, a += 128 * D / 16) {
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) umma_codes(d, a + kk * 2, b + kk * 2, Desc<D>::codes_hi, kQk, term | kk);
    }
  };
  auto pv = [&](int x, int stage, bool first) {
    const uint32_t b = v0 + stage * (kKeys * D * 2 / 16), d = tmem + x * 128, a = tmem + 256 + x * 128;
#pragma unroll
    for (int kk = 0; kk < kKeys / 16; ++kk)
      umma_weights(d, a + kk * 8, b + kk * (2048 / 16), Desc<D>::values_hi, kPv, kk ? 1u : !first);
  };
  for (; w.valid(); step_on(p, w)) {
    const int nt = w.needed(p);
    const bool two = w.cols(p) > 128;
    if (nt == 0) continue;
    for (int t = -1; t < nt; ++t) {
      // scores of tile t + 1, weights times values of tile t
      const uint32_t kn = tile_no + t + 1, vn = tile_no + t;
      const int ks = kn % kStagesK, vs = vn % kStagesV;
      const bool more = t + 1 < nt;
      if (more) bounded_wait(sm, k_full + ks, kn / kStagesK & 1, p);
      if (t < 0) bounded_wait(sm, &sm.q_full, q_no & 1, p);
      else bounded_wait(sm, &sm.v_full[vs], vn / kStagesV & 1, p);
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        const bool on = x == 0 || two;
        if (t >= 0) bounded_wait(sm, &sm.p_full[x], p_no++ >> 1 & 1, p);
        __syncwarp();
        tc_fence_after();
        if (elect_one()) {
          if (t >= 0 && on) {
            pv(x, vs, t == 0);
            if (!more) umma_commit(&sm.o_full[x]);
          }
          if (more && on) qk(x, ks);
          if (more) umma_commit(&sm.s_full[x]);
          if (x == 1) {
            if (t >= 0) {
              umma_commit(&sm.v_empty[vs]);
              umma_commit(&sm.m_empty[vn % kMeta]);
            }
            if (more) umma_commit(&sm.k_empty[ks]);
            if (t + 2 == nt) umma_commit(&sm.q_empty);  // the last scores are under way
          }
        }
        __syncwarp();
      }
    }
    tile_no += nt;
    ++q_no;
  }
  if (elect_one()) umma_commit(&sm.done);
  __syncwarp();
  drain(&sm.done, 0);  // no product is under way when the CTA leaves
  __syncwarp();
}

// ------------------------------------------------------------------ softmax
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, uint32_t c) { return max3(a, b, __uint_as_float(c)); }
__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
  return max3(__uint_as_float(a), __uint_as_float(b), c);
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

// Rare tiles, through TMEM so that their code stays small.  Scores of keys in a
// page outside the pool become -inf, of keys with a NaN value NaN.
__device__ __noinline__ void hide_keys(uint32_t ts, const TileMeta &meta) {
#pragma unroll 1
  for (int j = 0; j < kKeys / 16; ++j) {
    uint32_t s[16];
    tmem_ld16(ts + 16 * j, s);
    const uint32_t nan = meta.nan[j >> 1] >> (16 * (j & 1)), hide = meta.hide[j >> 1] >> (16 * (j & 1));
    tmem_ld_wait();
#pragma unroll
    for (int b = 0; b < 16; ++b) {
      if (nan >> b & 1) s[b] = 0x7FC00000u;
      if (hide >> b & 1) s[b] = 0xFF800000u;  // -inf
    }
    tmem_st16(ts + 16 * j, s);
  }
  tmem_st_wait();
}
// A column's largest score of 16 keys, and the largest with their value exponent.
__device__ __forceinline__ void largest(const uint32_t *v, float f, float lv, float &top, float &topw) {
  const float a = max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), v[6]);
  const float b = max3(max3(v[7], v[8], v[9]), max3(v[10], v[11], v[12]), v[13]);
  const float y = max3(fmaxf(a, __uint_as_float(v[14])), b, v[15]) * f;
  top = fmaxf(top, y);
  topw = fmaxf(topw, y + lv);
}

// New references for a tile, the sum and the row of O brought to them.
// A weight in the sum is 2^(w - lv - m) of the one that enters the product.
// Where that is large (kFar), the values are so small that the latter may leave
// fp32's range; w - m is at most the largest lv so far (plus the slack of the
// references), so a tile's spread of lv tells when to look.
constexpr float kFar = 64.f;
template <int D>
__device__ __forceinline__ void settle(uint32_t ts, uint32_t to, const TileMeta &meta, float cs, bool has_o,
                                    float &m, float &w, float &l) {
  float top = -INFINITY, topw = -INFINITY;
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    uint32_t s[64];
    tmem_ld_32x32b_x32(ts + 64 * j, *reinterpret_cast<uint32_t(*)[32]>(s));
    tmem_ld_32x32b_x32(ts + 64 * j + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
    tmem_ld_wait();
#pragma unroll
    for (int g = 0; g < 4; ++g) largest(s + 16 * g, score_factor(cs, meta.kv[4 * j + g].x), meta.kv[4 * j + g].y, top, topw);
  }
  const float mn = fmaxf(m, top), wn = fmaxf(w, topw);
  const float fl = mn == m ? 1.f : ex2(m - mn), fo = wn == w ? 1.f : ex2(w - wn);
  m = mn, w = wn;
  l *= fl;
  if (has_o) {
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
// Weights of a tile whose value scales are that far apart, 16 keys at a time.
__device__ __noinline__ float weigh_far(uint32_t ts, const TileMeta &meta, float cs, float m, float w, float l) {
  const float mr = m == -INFINITY ? 0.f : m, wr = w == -INFINITY ? 0.f : w;
#pragma unroll 1
  for (int g = 0; g < 8; ++g) {
    uint32_t s[16];
    tmem_ld16(ts + 16 * g, s);
    const float f = score_factor(cs, meta.kv[g].x), lv = meta.kv[g].y;
    tmem_ld_wait();
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float y[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float x = __uint_as_float(s[2 * k + b]) * f;
        l += ex2(x - mr);
        y[b] = ex2(x + (lv - wr));
      }
      h[k] = float2_to_half2(y[0], y[1]);
    }
    tmem_st8(ts + 8 * g, h);
  }
  return l;
}

// Scores of keys at or behind the column's limit, in TMEM.
__device__ __noinline__ void hide_behind(uint32_t ts, int room) {
#pragma unroll 1
  for (int j = 0; j < kKeys; j += 32) {
    if (__all_sync(~0u, room >= j + 32)) continue;
    uint32_t s[32];
    tmem_ld_32x32b_x32(ts + j, s);
    tmem_ld_wait();
#pragma unroll
    for (int b = 0; b < 32; ++b)
      if (j + b >= room) s[b] = 0xFF800000u;
    tmem_st32(ts + j, s);
  }
  tmem_st_wait();
}

template <int D, bool TEST>
__device__ void softmax_role(const AttnParams &p, Smem<D, TEST> &sm, long long per, long long near) {
  Walk &w = sm.walk[threadIdx.x >> 5];
  const int x = threadIdx.x >> 7;        // tile of columns
  const int r = threadIdx.x & 127;       // its column
  const uint32_t lanes = (uint32_t)(r & ~31) << 16;
  const uint32_t ts = sm.tmem + 256 + x * 128 + lanes, to = sm.tmem + x * 128 + lanes;
  uint32_t tile_no = 0, s_no = 0, o_no = 0;
  for (; w.valid(); step_on(p, w)) {
    const int nt = w.needed(p), ncols = w.cols(p);
    const int col = x * 128 + r;
    if (ncols <= x * 128) {  // this half is empty: it keeps step, so that it meets every phase of the barriers
      for (int t = 0; t < nt; ++t, ++tile_no) {
        bounded_wait(sm, &sm.n_full[tile_no % kMeta], tile_no / kMeta & 1, p);
        bounded_wait(sm, &sm.s_full[x], s_no++ & 1, p);  // without it this half could run ahead of the issuing warp
        mbar_arrive(&sm.p_full[x]);
      }
      continue;
    }
    float m = -INFINITY, wr = -INFINITY, l = 0.f, cs = 0.f;
    int room0 = 0;  // keys that the column sees from the part's first tile on
    if (col < ncols) {
      const int c = w.x.block * kCols + col;
      room0 = p.causal ? min(max(w.x.q.len - w.x.q.n + c / p.group + 1, 0), w.x.q.len) : w.x.q.len;
      cs = __ldcg(p.q_scale + (size_t)w.x.head * p.rows * p.group + (size_t)w.x.q.r0 * p.group + c);
    }
    room0 -= w.x.t0 * kKeys;
    const int whole_tiles = __reduce_min_sync(~0u, room0) / kKeys;  // tiles every column of the warp sees whole
    for (int t = 0; t < nt; ++t, ++tile_no) {
      bounded_wait(sm, &sm.n_full[tile_no % kMeta], tile_no / kMeta & 1, p);
      bounded_wait(sm, &sm.s_full[x], s_no++ & 1, p);
      __syncwarp();
      tc_fence_after();
      const TileMeta &meta = sm.meta[tile_no % kMeta];
      const int room = room0 - t * kKeys;  // keys of the tile that the column sees
      if (meta.odd) hide_keys(ts, meta);
      if (t >= whole_tiles) hide_behind(ts, room);  // (not below: 128 live scores and a branch spill)
      // The weights are formed with the references as they stand.  A tile in which
      // 16 of them sum to more than 2^12 (or the scores pass m by as much) is done
      // again with new references: its scores are still in TMEM then.  The first
      // tile has its references set first.
      const bool look = meta.spread > kFar - 16.f;
      for (bool anew = t == 0;; anew = true) {
        if (anew) settle<D>(ts, to, meta, cs, t > 0, m, wr, l);
        if (look && __any_sync(~0u, wr - meta.lv_min - m > kFar)) {
          if (!anew) continue;
          l = weigh_far(ts, meta, cs, m, wr, l);
          break;
        }
        uint32_t s[128];
        {
#pragma unroll
          for (int j = 0; j < 2; ++j) tmem_ld_32x32b_x32(ts + 32 * j, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * j));
          tmem_ld_wait();
#pragma unroll
          for (int j = 2; j < 4; ++j) tmem_ld_32x32b_x32(ts + 32 * j, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * j));
          const float mr = m == -INFINITY ? 0.f : m, ww = wr == -INFINITY ? 0.f : wr;
          float lt = 0.f, most = 0.f;
          // Pairs of scores pass through three steps, kLag pairs apart (4, 6 or 8
          // are alike within 1%), so that the
          // exponentials of one overlap the products of another and the sums and
          // roundings of a third: product and offset; 2^x; sum and fp16.
          constexpr int kLag = 6;
          uint64_t e[64], sum[2] = {0, 0};
          uint64_t f2 = 0, b2 = 0;
          float back[8];
#pragma unroll
          for (int i = 0; i < 64 + 2 * kLag; ++i) {
            if (i < 64) {
              if (i == 32) tmem_ld_wait();
              if (i % 8 == 0) {
                const float2 kv = meta.kv[i / 8];
                const float f = score_factor(cs, kv.x), b = kv.y - ww;
                f2 = pack2(f, f), b2 = pack2(b, b);
                back[i / 8] = ex2(-b - mr);
              }
              e[i] = fma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), f2, b2);
            }
            if (i >= kLag && i < 64 + kLag) {
              float y, z;
              unpack2(e[i - kLag], y, z);
              e[i - kLag] = pack2(ex2(y), ex2(z));
            }
            if (i >= 2 * kLag) {
              const int k = i - 2 * kLag;
              float y, z;
              unpack2(e[k], y, z);
              s[k] = float2_to_half2(y, z);
              sum[k & 1] = k % 8 < 2 ? e[k] : add2(sum[k & 1], e[k]);
              if (k % 8 == 7) {
                unpack2(add2(sum[0], sum[1]), y, z);
                y += z;
                most = fmaxf(most, y);
                lt = fmaf(y, back[k / 8], lt);
              }
            }
          }
          if (!anew && __any_sync(~0u, fmaxf(most, lt * 0.125f) > 4096.f)) continue;
          l += lt;
        }
        tmem_st32(ts, s);
        tmem_st32(ts + 32, s + 32);
        break;
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sm.p_full[x]);
    }
    // ---- the part's result
    if (nt) {
      bounded_wait(sm, &sm.o_full[x], o_no++ & 1, p);
      __syncwarp();
      tc_fence_after();
    }
    const bool whole = w.x.t0 == 0 && w.x.t1 == w.x.tiles;
    const bool none = m == -INFINITY && l == 0.f;
    const float f = none ? 1.f : l != l ? NAN : ex2(wr - m) / l;
    const int c = w.x.block * kCols + col, ncols_now = w.cols(p);
    const int row = w.x.q.r0 + c / p.group, head = w.x.head * p.group + c % p.group;
    float *slot = p.slots + ((size_t)blockIdx.x * 2 + (w.x.t0 == 0 ? 1 : 0)) * ((size_t)kCols * (D + 4));
    uint8_t *out = reinterpret_cast<uint8_t *>(p.out) + ((size_t)row * p.q_heads + head) * D * 2;
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
#pragma unroll 1
    for (int j = 0; j < D; j += 32) {
      uint32_t o[32];
      if (nt) {
        tmem_ld_32x32b_x32(to + j, o);
        tmem_ld_wait();
      }
      if (none) {
#pragma unroll
        for (int b = 0; b < 32; ++b) o[b] = 0;
      }
      if (col < ncols_now) {
        // a lane writes its row by itself, in whole 32-byte sectors (the slots are aligned to them)
        if (whole) {
#pragma unroll
          for (int k = 0; k < 32; k += 16) {
            uint32_t h[8];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              const float y = __uint_as_float(o[k + 2 * b]) * f, z = __uint_as_float(o[k + 2 * b + 1]) * f;
              h[b] = p.bf16 ? float2_to_bf162(y, z) : float2_to_half2(y, z);
            }
            store_out(out + 2 * (j + k), h, wide);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; k += 8) store32(slot + (size_t)col * D + j + k, o + k);
        }
      }
    }
    if (col < ncols_now) {
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
      // ends of parts that lie inside the item behind this one, each the beginning of
      // a following CTA's part
      const long long rest = w.x.tiles - w.x.t1 - near;
      p.desc[blockIdx.x] = make_int4(w.x.q.r0, w.x.head, w.x.block * kCols,
                                     (int)((rest + per - 1) / per) | ncols_now << 20);
    }
  }
}

template <int D, bool TEST>
__global__ void __launch_bounds__(kThreads, 1)
    kv_prefill_kernel(const AttnParams p, const __grid_constant__ CUtensorMap map,
                      const __grid_constant__ CUtensorMap q_map) {
  grid_dependents();
  extern __shared__ uint8_t raw[];
  using S = Smem<D, TEST>;
  S &sm = *reinterpret_cast<S *>(raw + ((1024 - (smem_u32(raw) & 1023)) & 1023));
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
  // (One tile is enough for a part: a prompt of 128 rows takes 15 us so, 21 with two
  // tiles or more and 31 with four.)
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  // Even ends; one that lies within kNear tiles of an item's own end is
  // moved there, which saves the item's partial results and their joining.
  const long long near = min(per / 8, (long long)kNear), cut0 = min(blockIdx.x * per, total), cut1 = min(cut0 + per, total);
  if (tid == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (cut0 >= cut1) grid_wait();
  if (cut0 >= cut1) return;  // the whole CTA leaves together
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const long long cut = k ? cut1 : cut0;
    if (cut >= before && cut < before + mine) {
      long long b = before;
      for (int i = 0; i < per_thread; ++i) {
        const int s = tid * per_thread + i;
        const Seq q = seq_of(p, s);
        const long long per_head = q.blocks ? tiles_before(p, q, q.blocks) : 0, u = p.c.heads * per_head;
        if (cut < b + u) {
          sm.found_seq[k] = s;
          sm.found_per_head[k] = per_head;
          sm.found_at[k] = b;
          break;
        }
        b += u;
      }
    }
  }
  if (tid == 0) {
    sm.dead = 0;
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int i = 0; i < kStagesK; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < kStagesV; ++i) {
      mbar_init(&sm.v_full[i], kConverters);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < kMeta; ++i) {
      mbar_init(&sm.m_full[i], 1);
      mbar_init(&sm.m_empty[i], 1);
      mbar_init(&sm.n_full[i], kConverters);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 128);
      mbar_init(&sm.o_full[i], 1);
    }
    mbar_init(&sm.done, 1);
    for (int i = 0; i < kStagesK; ++i) mbar_init(&sm.never[i], 1);
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // a warp finds the item of each end (each warp by itself took 11,000 cycles for both)
  if (warp == 0 || (warp == 1 && cut1 < total)) {
    Cut c;
    c.x.seq = sm.found_seq[warp];
    c.x.q = seq_of(p, c.x.seq);
    long long rest = (warp ? cut1 : cut0) - sm.found_at[warp], begins = 0;
    const long long per_head = sm.found_per_head[warp];
    c.x.head = (int)(rest / per_head);
    rest -= c.x.head * per_head;
    int lo = 0, hi = c.x.q.blocks;  // the last block that begins at or before `rest`: 32 candidates at a time
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const long long v = at < hi ? tiles_before(p, c.x.q, at) : 0;
      const int pick = 31 - __clz(__ballot_sync(~0u, at < hi && v <= rest));  // lane 0's candidate always is one
      begins = __shfl_sync(~0u, v, pick);
      lo += pick * step;
      hi = min(hi, lo + step);
    }
    c.x.block = lo;
    c.x.tiles = block_tiles(p, c.x.q, lo);
    c.off = (int)(rest - begins);
    if (lane == 0) sm.cut[warp] = c;
  }
  __syncthreads();
  if (lane == 0) {
    Walk w;
    const Cut &c = sm.cut[0], &e = sm.cut[1];
    w.end = cut1;
    if (cut1 < total) {
      const int to_end = e.x.tiles - e.off;
      w.end = e.off <= near ? cut1 - e.off : to_end <= near ? cut1 + to_end : cut1;
    }
    w.at = cut0;
    w.x = c.x;
    w.x.t0 = c.off;
    if (c.off <= near) {
      w.at = cut0 - c.off;
      w.x.t0 = 0;
    } else if (c.x.tiles - c.off <= near) {
      w.x.t1 = c.x.tiles;
      w.next(p);
    }
    if (w.valid()) w.fit();
    sm.walk[warp] = w;
  }
  __syncwarp();
  grid_wait();  // the query terms
  // Registers: 256 x 192 + 128 x 80 + 128 x 48 = 512 x 128, what the block was
  // launched with.  (Chunk of 32K positions, at the time: 720 us; with 184, 96 and 48
  // 735; with 200, 72 and 40 the converters spill: 1,360 instead of 799.)
  if (warp < 8) {
    reg_inc<192>();
    softmax_role<D, TEST>(p, sm, per, near);
  } else if (warp < 12) {
    reg_dec<80>();
    convert_role<D, TEST>(p, sm);
  } else {
    reg_dec<48>();
    if (warp == 12) mma_role<D, TEST>(p, sm);
    if (warp == 13) lookup_role<D, TEST>(p, map, q_map, sm);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) tmem_dealloc(sm.tmem, 512);
}

// Query terms: D / 8 lanes per (row, head), 8 values each (90K rows of 128: 13.4 us, 3.4
// TB/s).  Terms go to planes
// [term][key/value head][row][head of the group][D], factors to [key/value
// head][row][head of the group].
template <int D>
__device__ __forceinline__ void terms_of(const AttnParams &p, const uint4 u, bool on, int row, int head, int part,
                                         uint8_t *__restrict__ q8, float *__restrict__ factor) {
  constexpr int LPR = D / 8;
  const uint32_t ws[4] = {u.x, u.y, u.z, u.w};
  float f[8];
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 y = p.bf16 ? bf16x2_to_float2(ws[j]) : half2_to_float2(ws[j]);
    f[2 * j] = y.x, f[2 * j + 1] = y.y;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!(fabsf(f[j]) <= FLT_MAX)) f[j] = NAN;  // infinities too: no softmax of theirs is a number
    amax = fmaxf(amax, fabsf(f[j]));
  }
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if (!on) return;
  // power of two that brings the largest magnitude to (224, 448]
  int e = 0;
  if (amax > 0.f) e = ((__float_as_uint(amax) & 0x7FFFFFu) > 0x600000u ? 7 : 8) - exponent_of(amax);
  e = max(-110, min(110, e));
  const float up = pow2i(e);
  // (exact: head < 2^16, so the quotient's error is below half of 1 / group)
  const int kv_head = (int)(((float)head + 0.5f) * __frcp_rn((float)p.group));
  const size_t at = ((size_t)kv_head * p.rows + row) * p.group + (head - kv_head * p.group);
  if (part == 0) factor[at] = p.scale_log2 * pow2i(-e);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] *= up;
  const size_t plane = (size_t)p.rows * p.q_heads * D;
  const int terms = p.bf16 ? 2 : 3;
  for (int term = 0;;) {
    uint2 c;
    c.x = to_e4m3x4(f[0], f[1], f[2], f[3]);
    c.y = to_e4m3x4(f[4], f[5], f[6], f[7]);
    *reinterpret_cast<uint2 *>(q8 + term * plane + at * D + part * 8) = c;
    if (++term == terms) break;
    const uint32_t back[4] = {cvt2(c.x), cvt2_hi(c.x), cvt2(c.y), cvt2_hi(c.y)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = half2_to_float2(back[j]);
      f[2 * j] -= y.x, f[2 * j + 1] -= y.y;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(256) kv_query_terms_kernel(const AttnParams p, uint8_t *__restrict__ q8,
                                                            float *__restrict__ factor) {
  grid_dependents();
  constexpr int LPR = D / 8, PER = 256 / LPR, BATCH = 4;  // lanes per row, rows per CTA and step, steps
  const int part = threadIdx.x % LPR;
  const int from = min(max(p.starts[0], 0), p.rows) * p.q_heads;  // rows of no sequence are not read
  const int last = min(max(p.starts[p.c.seqs], 0), p.rows) * p.q_heads;
  const int first = blockIdx.x * PER * BATCH + threadIdx.x / LPR;
  uint4 u[BATCH];
  int row[BATCH], head[BATCH];
#pragma unroll
  for (int i = 0; i < BATCH; ++i) {
    const int at = first + i * PER;
    if (i == 0 || p.q_heads < PER) {
      row[i] = at / p.q_heads, head[i] = at - row[i] * p.q_heads;
    } else {
      row[i] = row[i - 1], head[i] = head[i - 1] + PER;
      if (head[i] >= p.q_heads) ++row[i], head[i] -= p.q_heads;
    }
    u[i] = make_uint4(0, 0, 0, 0);
    if (at >= from && at < last)
      u[i] = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(p.q) +
                                                   (size_t)row[i] * p.q_stride + (size_t)head[i] * D + part * 8));
  }
#pragma unroll
  for (int i = 0; i < BATCH; ++i) {
    const int at = first + i * PER;
    terms_of<D>(p, u[i], at >= from && at < last, row[i], head[i], part, q8, factor);
  }
}

template <int D, bool TEST>
cudaError_t launch(const AttnParams &p, const CUtensorMap &map, const CUtensorMap &q_map, uint8_t *q8, float *factor,
                   int ctas, cudaStream_t stream) {
  constexpr size_t bytes = sizeof(Smem<D, TEST>) + 1024;
  static DeviceFlags done{0};
  cudaError_t e = allow_smem(kv_prefill_kernel<D, TEST>, bytes, done);
  if (e != cudaSuccess) return e;
  const int rows = p.rows * p.q_heads, per = 4 * 256 / (D / 8);
  e = launch_after(kv_query_terms_kernel<D>, dim3((rows + per - 1) / per), 256, 0, stream, false, p, q8, factor);
  if (e != cudaSuccess) return e;
  return launch_after(kv_prefill_kernel<D, TEST>, dim3(ctas), kThreads, bytes, stream, true, p, map, q_map);
}

}  // namespace

cudaError_t launch_kv_prefill(const AttnParams &p, const CUtensorMap &map, const CUtensorMap &q_map, uint8_t *q8,
                              float *factor, int ctas, cudaStream_t stream) {
  if (p.test)
    return p.c.dim == 64 ? launch<64, true>(p, map, q_map, q8, factor, ctas, stream)
                         : launch<128, true>(p, map, q_map, q8, factor, ctas, stream);
  return p.c.dim == 64 ? launch<64, false>(p, map, q_map, q8, factor, ctas, stream)
                       : launch<128, false>(p, map, q_map, q8, factor, ctas, stream);
}

}  // namespace mqa
