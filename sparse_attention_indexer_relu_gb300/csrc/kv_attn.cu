// Attention over the paged 8-bit cache for few query columns per key/value
// head: single tokens, short runs of them, and rows that each read their own
// selected keys.  (include/mqakv.h, mqa_kv_attention.)
//
// Mathematics.  The columns of an item are (query row, query head) pairs that
// read the same key/value head.  With c = scale * log2(e) and s = c * 2^(ke -
// 127) * q . E(k), in base 2,
//     out = sum_t 2^(s_t - m) 2^(ve_t - 127) E(v_t) / sum_t 2^(s_t - m).
// The codes are exact in fp16, so both products run on the tensor cores in
// fp16 with fp32 accumulation: q enters times a power of two that brings its
// column's largest magnitude to 2^10 (exact for bf16 and fp16 down to 2^-34 of
// it), and the weights enter as p' = 2^(s + lv - w), lv = ve - 127, with a
// running reference w of their own, so that a weight is rounded to fp16
// relative to the largest weight TIMES scale that its column has seen (11
// bits; a weight 2^-24 below it still has one).  The sum of the softmax is
// kept in fp32 from unrounded weights against a second reference m.  Both
// references move only when a weight passes 2^12.
//
// Layout.  S^T = K Q^T and O^T = V^T P^T: keys are the M dimension of the
// first product and head components that of the second, so 8 columns fill an
// MMA's N.  The order of the contraction index is free as long as both
// operands agree, so a lane takes 32 contiguous bytes of a key row (K) and 16
// contiguous components of 4 keys (V), converts them in registers and needs no
// transposed loads; P passes from one product to the other by an 8 x 8
// transpose of registers.
//
// Split.  All items' key tiles form one line that is cut evenly between the
// CTAs of a fixed grid, whatever the lengths; a CTA's range begins and ends
// inside items, for which it leaves partial results in its two workspace
// slots, and a second kernel joins them in a fixed order.
//
// Windows and trees (MQA_KV_KIND) are this kernel with other limits.  A window's items
// have the tiles of the first positions and those from its sequence's first row's
// window on, one number of tiles for the whole sequence; a tree's rows see what
// their masks say behind the sequence's rows.  Sub-tiles that no column sees are not
// read, and only those that some column sees in part look at limits or masks.
//
// What bounds it.  Single tokens over long caches: HBM (32 sequences of 16K to
// 64K positions, 8 key/value heads of 128: 2.68 GB in 400 us, 6.7 TB/s, 99% of
// the measured copy rate; 323 instructions per 16 keys, issue slots 44% busy; 128 with
// a window of 4,096 over up to 32K positions: 1.08 GB in 168 us, 6.4 TB/s, 95%).  One
// token with a window of 1,024: 10.6 us in a graph, two dependent kernels' latencies.
// More columns, or keys picked one by one: instructions and their latencies at
// the 12 warps per SM that the accumulators leave room for (16 x 5 fp16 rows, 4
// heads per key/value head of 64: 591 per 16 keys and 24 columns, 33 us, 1.33
// TB/s; 2,505 rows with 512 selected keys each, 16 heads per key/value head of
// 128: 683 per 16 keys, issue slots 52% busy, 180 us, 116 TFLOP/s out of L2).
#include "kv_internal.h"
#include "kv_ptx.cuh"

#include <cfloat>

// Compiled once for dense and selected attention (with the joining kernels), once
// for windows and once for trees.
#ifndef MQA_KV_KIND
#define MQA_KV_KIND 0
#endif

namespace mqa {

namespace {

constexpr int kWarps = kAttnThreads / 32;
constexpr int kTile = 16 * kWarps;  // keys per unit of work: one 16-key sub-tile per warp
// Sub-tiles in flight per warp: 2 x 16 warps x 4 KB ahead on an SM.  Long caches
// take 396 us with three stages and 429 with two (or with five CTAs of two: 460).
constexpr int kStages = 3;

// CTAs per SM: what its registers allow without much spilling in the loop (16
// columns of 128, four CTAs of 128 registers instead of three: 180 -> 275 us for
// selected prompts; 24 of 64, four instead of three: 34 -> 38 us).
template <int D, int NB>
struct Cfg {
  static constexpr int ctas = D == 64 ? (NB == 1 ? 5 : NB <= 3 ? 3 : 2) : (NB == 1 ? 4 : NB == 2 ? 3 : 2);
};

template <int D>
__host__ __device__ constexpr int stage_bytes() {
  return 2 * 16 * D;
}

// Per-warp stage descriptions: scale, exponent and position of its keys.
struct Meta {
  float ks[kStages][16];
  float lv[kStages][16];
  int pos[kStages][16];
  int any[kStages];
};

template <int D, int NB, int KIND, bool TEST>
struct Smem {
  static constexpr bool test = TEST;
  union {
    uint8_t ring[kWarps][kStages][2 * 16 * D];  // 16 rows of keys, 16 of values
    float merge[kWarps][8 * (NB < 2 ? NB : 2)][D + 4];
  };
  Meta meta[kWarps];
  uint64_t full[kWarps][kStages];
  uint64_t never[kStages];      // tests: nothing arrives here
  int dead;                     // a wait has run out
  float cs[8 * NB];             // per column: scale * log2(e) / (power of two q was multiplied with)
  int lim[8 * NB];              // positions the column sees: [0, lim)
  int lo[KIND >= kWindow ? 8 * NB : 1];  // windows: where the column's begins; trees: its row (-1: none)
  float wm[kWarps][8 * NB], ww[kWarps][8 * NB], wl[kWarps][8 * NB];
  uint4 qf[NB][D / 32][32];     // q fragments
  long long scan[kWarps];
  int found[2];
  long long found_at;
};

struct Item {
  int seq, head, cb;   // sequence (or row, for selected keys), key/value head, column block
  int tiles;           // key tiles of the item
};

}  // namespace

#if MQA_KV_KIND == 0
int attn_ctas_per_sm(int nb, int dim) {
  if (dim == 64) return nb == 1 ? Cfg<64, 1>::ctas : nb == 2 ? Cfg<64, 2>::ctas : nb == 3 ? Cfg<64, 3>::ctas : Cfg<64, 4>::ctas;
  return nb == 1 ? Cfg<128, 1>::ctas : nb == 2 ? Cfg<128, 2>::ctas : nb == 3 ? Cfg<128, 3>::ctas : Cfg<128, 4>::ctas;
}
size_t attn_slot_floats(int nb, int dim) { return (size_t)8 * nb * (dim + 4); }
#endif

namespace {

template <int D, int NB, int KIND, bool TEST>
__global__ void __launch_bounds__(kAttnThreads, Cfg<D, NB>::ctas)
    kv_attn_kernel(const AttnParams p, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map) {
  grid_dependents();
  extern __shared__ uint8_t smem_raw[];
  constexpr bool SEL = KIND == kSelected, WIN = KIND == kWindow, TREE = KIND == kTree;
  using S = Smem<D, NB, KIND, TEST>;
  S &sm = *reinterpret_cast<S *>(smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
  constexpr int CB = 8 * NB;
  constexpr int KW = D / 16;   // words of a K row per lane (8 or 4)
  constexpr int VW = D / 32;   // words of a V row per lane (4 or 2)
  constexpr int MT = D / 16;   // 16-component tiles of O^T
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int heads = p.c.heads, group = p.group;
  const int nsel_tiles = SEL ? max(1, (p.n_selected + kTile - 1) / kTile) : 1;
  const int ncb_sel = (group + CB - 1) / CB;

  const uint64_t policy = policy_evict_first();  // every key is read once, or few times
  // ---- this CTA's range of the line of work
  // sequence s: rows [r0, r1), length; units = heads * column blocks * tiles
  auto rows_of = [&](int s, int &r0, int &n) {
    r0 = min(max(p.starts[s], 0), p.rows);
    n = max(min(p.starts[s + 1], p.rows) - r0, 0);
  };
  auto length_of = [&](int s) { return min(max(p.c.lens[s], 0), p.c.max_pages << p.c.page_log2); };
  auto shape_of = [&](int s, int &ncb, int &tiles) {  // column blocks and tiles per item of sequence s
    int r0, n;
    rows_of(s, r0, n);
    const long long cols = (long long)n * group;
    ncb = cols > p.max_cols ? 0 : (int)((cols + CB - 1) / CB);
    const int len = length_of(s);
    tiles = ncb ? max(1, (len + kTile - 1) / kTile - (WIN ? skipped_tiles<kTile>(p, len - n + 1) : 0)) : 0;
  };
  long long total;
  // a warp has a run of sequences, 32 at a time
  const int per_warp = (p.c.seqs + kAttnThreads - 1) / kAttnThreads * 32, s0 = warp * per_warp + lane;
  auto units_of = [&](int s) -> long long {
    int ncb = 0, tiles = 0;
    if (s < p.c.seqs) shape_of(s, ncb, tiles);
    return (long long)heads * ncb * tiles;
  };
  long long mine = 0, before = 0;  // of the warp, and of the warps before it
  int first = 0;                   // selected keys: the first row of a sequence
  if (SEL) {
    first = min(max(p.starts[0], 0), p.rows);
    const int last = min(max(p.starts[p.c.seqs], first), p.rows);
    total = (long long)(last - first) * heads * ncb_sel * nsel_tiles;
  } else {
#pragma unroll 4
    for (int i = 0; i < per_warp; i += 32) mine += units_of(s0 + i);
#pragma unroll
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
    if (lane == 0) sm.scan[warp] = mine;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm.scan[w];
      total += sm.scan[w];
    }
  }
  // (Windows and trees: two tiles at least, for fewer parts to join.  A window of 1,024:
  // one token 10.8 us with one, 10.6 with two, 11.0 with three and 13.9 with four, 9
  // rows 15.1, 14.0, 14.4 and 17.5; a window of 4,096 15.0, 13.0, 13.0 and 15.5.)
  const long long per = max((total + gridDim.x - 1) / gridDim.x, WIN || TREE ? 2LL : 1LL);
  long long at = blockIdx.x * per;
  const long long end = min(total, at + per);
  if (tid == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (at >= end) grid_wait();
  if (at >= end) return;  // the whole CTA leaves together
  if (tid == 0) {
    sm.dead = 0;
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(&sm.full[0][0] + i, 1);
    for (int i = 0; i < kStages; ++i) mbar_init(sm.never + i, 1);
    fence_mbar_init();
  }
  uint32_t copies = 0;  // sub-tiles whose copies this warp has issued, in all segments
  uint64_t *const full = TEST && p.stall ? sm.never : sm.full[warp];  // what it waits for
  Item it;
  int tile;  // first tile of the current segment
  if (SEL) {
    const long long item = at / nsel_tiles;
    it.tiles = nsel_tiles;
    tile = (int)(at - item * nsel_tiles);
    it.cb = (int)(item % ncb_sel);
    it.head = (int)(item / ncb_sel % heads);
    it.seq = first + (int)(item / ((long long)ncb_sel * heads));  // the row
  } else {
    if (at >= before && at < before + mine) {
      long long b = before;
      for (int i = 0; i < per_warp && b <= at; i += 32) {
        const long long u = units_of(s0 + i);
        long long incl = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(~0u, incl, o);
          if (lane >= o) incl += v;
        }
        if (at >= b + incl - u && at < b + incl) {
          sm.found[0] = s0 + i;
          sm.found_at = at - (b + incl - u);
        }
        b += __shfl_sync(~0u, incl, 31);
      }
    }
    __syncthreads();
    it.seq = sm.found[0];
    int ncb;
    shape_of(it.seq, ncb, it.tiles);
    const long long item = sm.found_at / it.tiles;
    tile = (int)(sm.found_at - item * it.tiles);
    it.cb = (int)(item % ncb);
    it.head = (int)(item / ncb);
  }

  Meta &meta = sm.meta[warp];
  while (at < end) {
    const int t0 = tile, t1 = (int)min((long long)it.tiles, t0 + (end - at));
    // ---- the item's rows, columns and limits
    int r0, n, seq = it.seq, ncb;
    if (SEL) {
      int lo = 0, hi = p.c.seqs;  // the last sequence that starts at or before the row
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.starts[mid] <= it.seq) lo = mid; else hi = mid;
      }
      seq = lo;
      ncb = ncb_sel;
    }
    rows_of(seq, r0, n);
    const int len = length_of(seq);
    if (!SEL) ncb = (int)(((long long)n * group + CB - 1) / CB);
    const int32_t *table = p.c.table + (size_t)seq * p.c.max_pages;
    const int c0 = it.cb * CB;                          // first column of the block
    const int ncols = min(CB, (SEL ? group : n * group) - c0);
    if (tid == 0 && p.c.lens[seq] != len) atomicOr(p.c.status, MQA_KV_DEV_BAD_LENGTH);
    fence_async_smem();  // copies into what was read and written with ordinary accesses
    __syncthreads();     // the previous segment's readers of cs / lim / merge are done
    if (tid < CB) {
      int lim = SEL ? 0 : INT32_MAX;  // columns behind the last take part like the others (a query of zeros)
      int lo = TREE ? -1 : INT32_MIN;
      if (tid < ncols) {
        const int i = SEL ? it.seq - r0 : (c0 + tid) / group;
        lim = p.causal ? min(max(len - n + i + 1, 0), len) : len;
        if (SEL && (i < 0 || i >= n)) lim = 0;
        if (WIN) lo = lim - p.window;
        if (TREE) lo = r0 + i;
      }
      sm.lim[tid] = lim;
      if (WIN || TREE) sm.lo[tid] = lo;
    }
    __syncthreads();
    int lim_max = 0, lim_min = INT32_MAX;
    int lo_max = 0, lo_min = INT32_MAX;  // windows
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      lim_max = max(lim_max, i < ncols ? sm.lim[i] : 0);
      lim_min = min(lim_min, i < ncols ? sm.lim[i] : INT32_MAX);
      if (WIN) {
        lo_max = max(lo_max, i < ncols ? sm.lo[i] : 0);
        lo_min = min(lo_min, i < ncols ? sm.lo[i] : INT32_MAX);
      }
    }
    const int own0 = len - n;  // trees: position of the sequence's first row
    // first position of the warp's 16 in tile i of the segment
    const int sinks_end = WIN ? sink_tiles<kTile>(p) : 0, skip = WIN ? skipped_tiles<kTile>(p, len - n + 1) : 0;
    auto base_of = [&](int i) {
      const int t = t0 + i;
      return (WIN && t >= sinks_end ? t + skip : t) * kTile + warp * 16;
    };
    const int32_t *sel = SEL ? p.selected + (size_t)it.seq * p.n_selected : nullptr;
    // the tiles this item needs: later ones hold no key that a column sees
    const int t1e = SEL ? t1 : min(t1, (lim_max + kTile - 1) / kTile - skip);
    const int iters = max(0, t1e - t0);
    // ---- loads, 16 rows of keys and of values per sub-tile, the 16-byte chunks
    // of a row exchanged so that both products' reads spread over the banks:
    // whole rows by TMA, whose swizzle is the same, selected ones 16 bytes per
    // lane (as TMA gathers, 8 instructions of one lane each, they held their
    // warp up for 1,200 cycles).  Nothing is computed from a loaded index
    // before the refresh after the one that loaded it.
    // Dense: lane j holds sub-tile i + j's first row and exponents.
    int d_row = -1;
    // Selected: 32 entries per refresh (two sub-tiles): position, page, exponents.
    int s_raw = -1, s_pos1 = -1, s_pg1 = -1, s_pos2 = -1, s_row2 = -1, s_pos = -1, s_row = -1;
    uint32_t ke = 127, ve = 127;
    float s_ks = 0.f, s_lv = 0.f;
    auto load_raw = [&](int i) {  // the lane's entry among sub-tiles i, i + 1
      const int k = (t0 + i + (lane >> 4)) * kTile + warp * 16 + (lane & 15);
      s_raw = i + (lane >> 4) < iters && k < p.n_selected ? __ldg(sel + k) : -1;
    };
    auto load_page = [&](int pos) -> int { return pos < 0 ? -1 : __ldg(table + (pos >> p.c.page_log2)); };
    auto row_of = [&](int pos, int pg) -> int {
      if (pos < 0) return -1;
      if ((unsigned)pg >= (unsigned)p.c.pages) {
        atomicOr(p.c.status, MQA_KV_DEV_BAD_INDEX);
        return -1;
      }
      return ((pg * heads + it.head) << p.c.page_log2) + (pos & (p.c.page - 1));
    };
    auto load_exps = [&](int row) {
      if (row < 0) return;
      const int ph = row >> p.c.page_log2;
      ke = __ldg(p.c.k_exps + ph);
      ve = __ldg(p.c.v_exps + ph);
    };
    auto step_sel = [&](int i) {  // entries of sub-tile i enter the chain
      s_pos = s_pos2, s_row = s_row2;
      s_ks = exp_byte(ke), s_lv = (float)(int)ve - 127.f;
      s_pos2 = s_pos1, s_row2 = row_of(s_pos1, s_pg1), load_exps(s_row2);
      s_pos1 = (unsigned)s_raw < (unsigned)lim_max ? s_raw : -1, s_pg1 = load_page(s_pos1);
      load_raw(i);
    };
    // the first indices are on their way while the queries are turned into terms
    auto begin = [&] {
      if (SEL) {
        step_sel(0);
        step_sel(2);
        step_sel(4);
      }
    };
    begin();
    auto issue = [&](int i) {
      if (i >= iters) {
        if (SEL) cp_async_commit();
        return;
      }
      const uint32_t no = copies++;
      const int stage = no % kStages;
      uint64_t *bar = &sm.full[warp][stage];
      uint8_t *kd = sm.ring[warp][stage], *vd = kd + 16 * D;
      if (SEL) {
        if ((i & 1) == 0) step_sel(i + 6);
        const int half = 16 * (i & 1);
        const uint32_t ok = __ballot_sync(~0u, s_row >= 0) >> half & 0xFFFFu;
        if ((lane >> 4) == (i & 1)) {
          meta.ks[stage][lane & 15] = s_ks;
          meta.lv[stage][lane & 15] = s_lv;
          meta.pos[stage][lane & 15] = s_row < 0 ? INT32_MAX : s_pos;
        }
        if (lane == 0) meta.any[stage] = ok != 0;
        constexpr int CH = D / 16;  // chunks per row
        const int ch = lane % CH, rl = lane / CH;
        if (ok) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const int r = c * (32 / CH) + rl;
            const int row = __shfl_sync(~0u, s_row, half + r);
            const size_t src = (size_t)(unsigned)max(row, 0) * D + ch * 16;
            const int dst = r * D + ((ch ^ (D == 128 ? r & 7 : r >> 1 & 3)) << 4);
            cp_async16(kd + dst, p.c.k + src, row >= 0);  // zeros for entries that name no visible key
            cp_async16(vd + dst, p.c.v + src, row >= 0);
          }
        }
        cp_async_commit();
      } else {
        if ((i & 31) == 0) {
          const int pos = base_of(i + lane);
          const bool want = i + lane < iters && pos < lim_max && (!WIN || pos < p.sinks || pos + 16 > lo_min);
          d_row = want ? row_of(pos, load_page(pos)) : -1;
          load_exps(d_row);
        }
        if (lane == (i & 31)) {
          meta.ks[stage][0] = exp_byte(ke);
          meta.lv[stage][0] = (float)(int)ve - 127.f;
          meta.any[stage] = d_row >= 0;
        }
        const int row = __shfl_sync(~0u, d_row, i & 31);
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, row >= 0 ? 2 * 16 * D : 0);
          if (row >= 0) {
            tma_load_2d(kd, &k_map, bar, 0, row, policy);
            tma_load_2d(vd, &v_map, bar, 0, row, policy);
          }
        }
      }
    };
    // ---- q: column g of each 8-column block, the lane's components
    // k-step j: b0 = components KW*4*t + 4j, +1; b1 = +2, +3 (t's 4*KW bytes of a key row)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (nb % kWarps != warp) continue;  // one warp loads a block for all
      const int col = nb * 8 + g;
      float f[4 * KW];
      float amax = 0.f;
      if (col < ncols) {
        const int row = SEL ? it.seq : r0 + (c0 + col) / group;
        const int h = it.head * group + (SEL ? c0 + col : (c0 + col) % group);
        const size_t off = (size_t)row * p.q_stride + (size_t)h * D + 4 * KW * t;
        const uint4 *src = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(p.q) + off);
#pragma unroll
        for (int j = 0; j < KW / 2; ++j) {
          const uint4 w = __ldg(src + j);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            float2 x = p.bf16 ? bf16x2_to_float2(ws[b]) : half2_to_float2(ws[b]);
            f[8 * j + 2 * b] = x.x;
            f[8 * j + 2 * b + 1] = x.y;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4 * KW; ++j) f[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4 * KW; ++j) {
        if (!(fabsf(f[j]) <= FLT_MAX)) f[j] = NAN;  // infinities too: no softmax of theirs is a number
        amax = fmaxf(amax, fabsf(f[j]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
      // power of two that brings the column's largest magnitude to [2^10, 2^11)
      int e = 0;
      if (amax > 0.f) e = 10 - exponent_of(amax);
      e = max(-100, min(100, e));
      const float up = pow2i(e);
      if (t == 0) sm.cs[col] = p.scale_log2 * pow2i(-e);
#pragma unroll
      for (int j = 0; j < KW / 2; ++j)
        sm.qf[nb][j][lane] = make_uint4(
            float2_to_half2(f[8 * j] * up, f[8 * j + 1] * up), float2_to_half2(f[8 * j + 2] * up, f[8 * j + 3] * up),
            float2_to_half2(f[8 * j + 4] * up, f[8 * j + 5] * up), float2_to_half2(f[8 * j + 6] * up, f[8 * j + 7] * up));
    }
    __syncthreads();
    uint4 qr[KW / 2];  // 8 columns: in registers; more are read with each sub-tile
    if (NB == 1) {
#pragma unroll
      for (int j = 0; j < KW / 2; ++j) qr[j] = sm.qf[0][j][lane];
    }
    float cs[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        cs[nb][c] = sm.cs[nb * 8 + 2 * t + c];
      }

    float m[NB][2], w[NB][2], l[NB][2];
    float o[MT][NB][4];

    bool lost = false;  // a wait has run out
    // A masked weight is zero, but zero times a NaN value is NaN: where the
    // result has one, the segment runs again with NaN codes of V taken out and
    // every visible key that has one scored NaN.
    for (int careful = 0; careful < 2; ++careful) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 2; ++c) m[nb][c] = w[nb][c] = -INFINITY, l[nb][c] = 0.f;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][nb][i] = 0.f;

      if (careful) begin();
      uint32_t done = copies;  // sub-tiles worked on
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) issue(i);

      for (int i = 0; i < iters; ++i, ++done) {
        const int stage = done % kStages;
        if (SEL) {
          cp_async_wait<kStages - 2>();
          __syncwarp();
        } else if (!warp_wait(sm, full + stage, done / kStages & 1, p)) {
          lost = true;
          break;
        }
        if (!meta.any[stage]) {  // no key of the sub-tile is seen
          __syncwarp();
          issue(i + kStages - 1);
          continue;
        }
        const uint8_t *kd = sm.ring[warp][stage], *vd = kd + 16 * D;
        // ---- S^T = K Q^T
        float acc[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[nb][j] = 0.f;
        uint32_t ka[KW], kb[KW];  // rows g and g + 8
#pragma unroll
        for (int h = 0; h < KW / 4; ++h) {
          const int ch = t * (KW / 4) + h;
          const int sa = D == 128 ? (g & 7) : ((g >> 1) & 3), sb = D == 128 ? (g & 7) : (((g + 8) >> 1) & 3);
          const uint4 x = *reinterpret_cast<const uint4 *>(kd + g * D + ((ch ^ sa) << 4));
          const uint4 y = *reinterpret_cast<const uint4 *>(kd + (g + 8) * D + ((ch ^ sb) << 4));
          ka[4 * h] = x.x, ka[4 * h + 1] = x.y, ka[4 * h + 2] = x.z, ka[4 * h + 3] = x.w;
          kb[4 * h] = y.x, kb[4 * h + 1] = y.y, kb[4 * h + 2] = y.z, kb[4 * h + 3] = y.w;
        }
#pragma unroll
        for (int j = 0; j < KW; j += 2) {
          const uint32_t a[4] = {cvt2(ka[j]), cvt2(kb[j]), cvt2_hi(ka[j]), cvt2_hi(kb[j])};
          const uint32_t b[4] = {cvt2(ka[j + 1]), cvt2(kb[j + 1]), cvt2_hi(ka[j + 1]), cvt2_hi(kb[j + 1])};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint4 q = NB == 1 ? qr[j / 2] : sm.qf[nb][j / 2][lane];
            mma_f16(acc[nb], a, q.x, q.y);
            mma_f16(acc[nb], b, q.z, q.w);
          }
        }
        // ---- V words: keys 2t, 2t + 1, 2t + 8, 2t + 9, components 4 * VW * g ...
        uint32_t v[4][VW];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const int r = 2 * t + (kk & 1) + 8 * (kk >> 1);
          const int sw = D == 128 ? (r & 7) : ((r >> 1) & 3);
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4 *>(vd + r * D + ((g ^ sw) << 4));
            v[kk][0] = x.x, v[kk][1] = x.y, v[kk][VW - 2] = x.z, v[kk][VW - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(vd + r * D + (((g >> 1) ^ sw) << 4) + 8 * (g & 1));
            v[kk][0] = x.x, v[kk][1] = x.y;
          }
        }
        uint32_t bad_keys = 0;
        if (careful) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int j = 0; j < VW; ++j) {
              const uint32_t nb8 = nan_bytes(v[kk][j]);
              if (nb8) {
                bad_keys |= 1u << (2 * t + (kk & 1) + 8 * (kk >> 1));
                v[kk][j] &= ~((nb8 >> 7) * 255u);
              }
            }
          bad_keys = __reduce_or_sync(~0u, bad_keys);
        }
        // ---- weights: formed with the references as they stand; a sub-tile in which
        // one passes 2^12 (or that finds no references yet) moves them and starts over
        uint32_t pf[NB][2];
        float pl[NB][2][2];
        {
          float ks[2], lv[2], none[2];
          int room[2];  // by how much a column's limit lies behind the key
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int k = SEL ? g + 8 * r : 0, pos = SEL ? meta.pos[stage][k] : base_of(i);
            ks[r] = meta.ks[stage][k];
            lv[r] = meta.lv[stage][k];
            none[r] = SEL && pos == INT32_MAX ? -INFINITY : 0.f;  // an entry that names no visible key
            room[r] = SEL ? 0 : pos + g + 8 * r;
          }
          if (SEL) {
            if (bad_keys) {
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (bad_keys >> (g + 8 * r) & 1) {
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb) acc[nb][2 * r] = acc[nb][2 * r + 1] = NAN;
                }
            }
          } else if (bad_keys || base_of(i) + 16 > (TREE ? own0 : lim_min) ||
                     (WIN && base_of(i) < lo_max && base_of(i) + 16 > p.sinks)) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  if (bad_keys >> (g + 8 * r) & 1) acc[nb][2 * r + c] = NAN;
                  // (scales are positive: -inf stays -inf)
                  const int col = nb * 8 + 2 * t + c;
                  if (room[r] >= min(sm.lim[col], lim_max)) acc[nb][2 * r + c] = -INFINITY;
                  if (WIN && room[r] < sm.lo[col] && room[r] >= p.sinks) acc[nb][2 * r + c] = -INFINITY;
                  if (TREE && sm.lo[col] >= 0 &&
                      !(tree_bits(p.tree + (size_t)sm.lo[col] * p.tree_words, p.tree_words, room[r] - own0) & 1))
                    acc[nb][2 * r + c] = -INFINITY;
                }
          }
          for (bool anew = false;; anew = true) {
            bool move = false, far = false;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              float p2[2][2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float mc = m[nb][c], wc = w[nb][c], mr = mc == -INFINITY ? 0.f : mc, wr = mc == -INFINITY ? 0.f : wc;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const float f = score_factor(cs[nb][c], ks[r]);
                  p2[r][c] = ex2(fmaf(acc[nb][2 * r + c], f, none[r] + (lv[r] - wr)));
                  pl[nb][c][r] = SEL ? ex2(fmaf(acc[nb][2 * r + c], f, none[r] - mr)) : p2[r][c];
                }
                // dense: both keys have one value scale, and the weight in the sum is
                // 2^back of the one that enters the product
                const float back = wr - lv[0] - mr;
                if (!SEL) {
                  pl[nb][c][0] = (pl[nb][c][0] + pl[nb][c][1]) * ex2(back);
                  pl[nb][c][1] = 0.f;
                  far |= back > 64.f;
                }
                move |= fmaxf(fmaxf(p2[0][c], p2[1][c]), fmaxf(pl[nb][c][0], pl[nb][c][1]) * 0.125f) > 4096.f ||
                        mc == -INFINITY;
              }
#pragma unroll
              for (int r = 0; r < 2; ++r) pf[nb][r] = float2_to_half2(p2[r][0], p2[r][1]);
            }
            if (!__any_sync(~0u, move || far) || anew) {
              if (!SEL && __any_sync(~0u, far)) {
                // values so small that their weights may have left fp32's range
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const float f = score_factor(cs[nb][c], ks[0]), mr = m[nb][c] == -INFINITY ? 0.f : m[nb][c];
                    pl[nb][c][0] = ex2(fmaf(acc[nb][c], f, -mr)) + ex2(fmaf(acc[nb][2 + c], f, -mr));
                  }
              }
              break;
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float s0 = fmaf(acc[nb][c], score_factor(cs[nb][c], ks[0]), none[0]);
                const float s1 = fmaf(acc[nb][2 + c], score_factor(cs[nb][c], ks[1]), none[1]);
                float a = fmaxf(s0, s1), b = fmaxf(s0 + lv[0], s1 + lv[1]);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                  a = fmaxf(a, __shfl_xor_sync(~0u, a, x));
                  b = fmaxf(b, __shfl_xor_sync(~0u, b, x));
                }
                a = fmaxf(a, m[nb][c]), b = fmaxf(b, w[nb][c]);
                const float fl = m[nb][c] == a ? 1.f : ex2(m[nb][c] - a), fo = w[nb][c] == b ? 1.f : ex2(w[nb][c] - b);
                m[nb][c] = a, w[nb][c] = b;
                l[nb][c] *= fl;
#pragma unroll
                for (int j = 0; j < MT; ++j) o[j][nb][c] *= fo, o[j][nb][2 + c] *= fo;
              }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int c = 0; c < 2; ++c) l[nb][c] += pl[nb][c][0] + pl[nb][c][1];
#pragma unroll
            for (int r = 0; r < 2; ++r) pf[nb][r] = transpose8x8(pf[nb][r]);
          }
        }
        // ---- O^T += V^T P^T; tile j holds components 4 * VW * g + 2j and + 2j + 1 in rows g and g + 8
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          const uint32_t a01 = __byte_perm(v[0][j], v[1][j], 0x5140), b01 = __byte_perm(v[0][j], v[1][j], 0x7362);
          const uint32_t a23 = __byte_perm(v[2][j], v[3][j], 0x5140), b23 = __byte_perm(v[2][j], v[3][j], 0x7362);
          const uint32_t x[4] = {cvt2(a01), cvt2_hi(a01), cvt2(a23), cvt2_hi(a23)};
          const uint32_t y[4] = {cvt2(b01), cvt2_hi(b01), cvt2(b23), cvt2_hi(b23)};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma_f16(o[2 * j][nb], x, pf[nb][0], pf[nb][1]);
            mma_f16(o[2 * j + 1][nb], y, pf[nb][0], pf[nb][1]);
          }
        }
        __syncwarp();
        issue(i + kStages - 1);
      }
      if (SEL) cp_async_wait<0>();
      bool bad = false;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) bad |= o[j][nb][i] != o[j][nb][i];
      if (careful || lost || !__any_sync(~0u, bad)) break;
    }

    // ---- join the warps: common references, then sums in warp order
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nb][c] += __shfl_xor_sync(~0u, l[nb][c], x);
        if (g == 0) {
          sm.wm[warp][nb * 8 + 2 * t + c] = m[nb][c];
          sm.ww[warp][nb * 8 + 2 * t + c] = w[nb][c];
          sm.wl[warp][nb * 8 + 2 * t + c] = l[nb][c];
        }
      }
    __syncthreads();  // every warp is done with its ring
    const bool whole = t0 == 0 && t1 == it.tiles;
    float *slot = p.slots + ((size_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * attn_slot_floats_dev<CB, D>();
    // two blocks of columns at a time: every warp leaves its part, then a warp adds a column's
    constexpr int NP = NB < 2 ? NB : 2;
    for (int n0 = 0; n0 < NB; n0 += NP) {
      if (n0) __syncthreads();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (nb < n0 || nb >= n0 + NP) continue;
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<float2 *>(&sm.merge[warp][(nb - n0) * 8 + 2 * t + c][4 * VW * g + 2 * j]) =
                make_float2(o[j][nb][c], o[j][nb][2 + c]);
      }
      __syncthreads();
      for (int col = n0 * 8 + warp; col < min(ncols, (n0 + NP) * 8); col += kWarps) {
        float mx = -INFINITY, wx = -INFINITY, ls = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) mx = fmaxf(mx, sm.wm[x][col]), wx = fmaxf(wx, sm.ww[x][col]);
#pragma unroll
        for (int x = 0; x < kWarps; ++x)
          ls += sm.wl[x][col] * (sm.wm[x][col] == mx ? 1.f : ex2(sm.wm[x][col] - mx));
        constexpr int E = D / 32;  // components per lane
        float sum[E];
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
          const float f = sm.ww[x][col] == wx ? 1.f : ex2(sm.ww[x][col] - wx);
          const float *part = &sm.merge[x][col - n0 * 8][lane * E];
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(part + e);
            sum[e] += f * v.x, sum[e + 1] += f * v.y;
          }
        }
        if (whole) {
          const int row = SEL ? it.seq : r0 + (c0 + col) / group;
          const int h = it.head * group + (SEL ? c0 + col : (c0 + col) % group);
          finish_lane<E>(p, row, h, lane, sum, mx, wx, ls);
        } else {
#pragma unroll
          for (int e = 0; e < E; e += 2)
            *reinterpret_cast<float2 *>(slot + col * D + lane * E + e) = make_float2(sum[e], sum[e + 1]);
          if (lane == 0) {
            slot[CB * D + col] = mx;
            slot[CB * D + CB + col] = wx;
            slot[CB * D + 2 * CB + col] = ls;
          }
        }
      }
    }
    if (!whole && t0 == 0 && tid == 0) {
      // the CTAs that hold the item's other parts follow this one
      const long long rest = it.tiles - (t1 - t0);
      p.desc[blockIdx.x] = make_int4(SEL ? it.seq : r0, it.head, SEL ? -c0 - 1 : c0, (int)((rest + per - 1) / per) |
                                     ncols << 20);
    }
    // ---- next item (none after a wait that has run out: every warp sees that, as
    // none waits between the barriers above and the next item's)
    at += t1 - t0;
    tile = 0;
    if (at >= end || (!SEL && *reinterpret_cast<volatile int *>(&sm.dead))) break;
    if (++it.cb == ncb) {
      it.cb = 0;
      if (++it.head == heads) {
        it.head = 0;
        if (SEL) {
          ++it.seq;
        } else {
          int nn = 0;
          do {
            ++it.seq;
            shape_of(it.seq, nn, it.tiles);
          } while (nn == 0);
        }
      }
    }
  }
  if (!SEL)  // the copies have landed before the CTA leaves, also where a wait has run out
    for (uint32_t i = 1; i <= kStages && i <= copies; ++i)
      drain(&sm.full[warp][(copies - i) % kStages], (copies - i) / kStages & 1);
  grid_wait();
}

}  // namespace

#if MQA_KV_KIND == 0
// Join split items: a block adds the parts of two columns of the item that CTA
// `cta` of the kernel before began.  One long sequence is cut into one part
// per CTA, so four warps share a column's parts, each its own in CTA order, and
// are added in warp order: results do not depend on the timing.
namespace {
template <int D>
__device__ __forceinline__ void join_many(const AttnParams &p, int cb, int cta) {
  constexpr int WPC = 4, kJoinCols = 8 / WPC;
  const int4 d = p.desc[cta];
  const int more = d.w & 0xFFFFF, ncols = d.w >> 20;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, share = warp % WPC;
  const int col = blockIdx.y * kJoinCols + warp / WPC;
  if (more == 0 || blockIdx.y * kJoinCols >= ncols) return;
  __shared__ float acc[8][D];
  __shared__ float red[8];
  const bool on = col < ncols;
  const size_t pitch = (size_t)cb * (D + 4);
  auto slot = [&](int i) { return p.slots + ((size_t)(cta + i) * 2 + (i == 0 ? 1 : 0)) * pitch; };
  float mx = -INFINITY, wx = -INFINITY;
  constexpr int E = D / 32;
  float o[E], ls = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  if (on) {
    for (int i = lane; i <= more; i += 32) {
      const float *s = slot(i) + (size_t)cb * D;
      mx = fmaxf(mx, s[col]);
      wx = fmaxf(wx, s[cb + col]);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, x));
      wx = fmaxf(wx, __shfl_xor_sync(~0u, wx, x));
    }
#pragma unroll 8
    for (int i = share; i <= more; i += WPC) {
      const float *s = slot(i), *t = s + (size_t)cb * D;
      const float m = t[col], w = t[cb + col];
      ls += t[2 * cb + col] * (m == mx ? 1.f : ex2(m - mx));
      const float f = w == wx ? 1.f : ex2(w - wx);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v = *reinterpret_cast<const float2 *>(s + (size_t)col * D + lane * E + e);
        o[e] += f * v.x, o[e + 1] += f * v.y;
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[warp][lane * E + e] = o[e];
    if (lane == 0) red[warp] = ls;
  }
  __syncthreads();
  if (!on || share) return;
#pragma unroll
  for (int k = 1; k < WPC; ++k) {
    ls += red[warp + k];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += acc[warp + k][lane * E + e];
  }
  const bool sel = d.z < 0;
  const int c = (sel ? -d.z - 1 : d.z) + col;
  const int row = sel ? d.x : d.x + c / p.group, h = d.y * p.group + (sel ? c : c % p.group);
  finish_lane<E>(p, row, h, lane, o, mx, wx, ls);
}

// The same for the tiled kernel's items: many columns.  A warp has kFewCols columns,
// PARTS parts' loads of all of them in flight.  Mostly there are two or three parts,
// and registers decide (9 us after 5 prompts of up to 1,531 rows; with two in flight
// 12).  Calls of few items are cut into many parts: 18 drafts of 141 rows x 2 heads
// after 8K positions take 47 us with three in flight, 48 with two, 54 with four and 51
// with one; 3 of 58 rows x 16 heads of 64 after 30K 53, 55, 51 and 64.
constexpr int kFewCols = 4, kManyParts = 3;
template <int D, int PARTS>
__device__ __forceinline__ void join_few(const AttnParams &p) {
  const int4 d = p.desc[blockIdx.x];
  const int more = d.w & 0xFFFFF, ncols = d.w >> 20;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = (blockIdx.y * 8 + warp) * kFewCols;
  if (more == 0 || c0 >= ncols) return;
  constexpr int E = D / 32, CB = kTiledCols;
  constexpr size_t pitch = (size_t)CB * (D + 4);
  auto slot = [&](int i) { return p.slots + ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * pitch; };
  float mx[kFewCols], wx[kFewCols], ls[kFewCols], o[kFewCols][E];
#pragma unroll
  for (int k = 0; k < kFewCols; ++k) {
    mx[k] = wx[k] = -INFINITY, ls[k] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[k][e] = 0.f;
  }
  for (int i0 = 0; i0 <= more; i0 += PARTS) {
    float m[PARTS][4], w[PARTS][4], l[PARTS][4];
    float2 v[PARTS][kFewCols][E / 2];
#pragma unroll
    for (int b = 0; b < PARTS; ++b) {
      if (i0 + b > more) break;
      const float *s = slot(i0 + b), *t = s + (size_t)CB * D + c0;  // columns behind the last hold anything: not used
      *reinterpret_cast<float4 *>(m[b]) = *reinterpret_cast<const float4 *>(t);
      *reinterpret_cast<float4 *>(w[b]) = *reinterpret_cast<const float4 *>(t + CB);
      *reinterpret_cast<float4 *>(l[b]) = *reinterpret_cast<const float4 *>(t + 2 * CB);
#pragma unroll
      for (int k = 0; k < kFewCols; ++k)
#pragma unroll
        for (int e = 0; e < E / 2; ++e)
          v[b][k][e] = *reinterpret_cast<const float2 *>(s + (size_t)(c0 + k) * D + lane * E + 2 * e);
    }
#pragma unroll
    for (int b = 0; b < PARTS; ++b) {
      if (i0 + b > more) break;
#pragma unroll
      for (int k = 0; k < kFewCols; ++k) {  // references move as larger ones come; fmaf: the same bits for any PARTS
        const float pm = m[b][k], pw = w[b][k], pl = l[b][k];
        const float mn = fmaxf(mx[k], pm), wn = fmaxf(wx[k], pw);
        const float fa = mx[k] == mn ? 1.f : ex2(mx[k] - mn), fb = pm == mn ? 1.f : ex2(pm - mn);
        const float ga = wx[k] == wn ? 1.f : ex2(wx[k] - wn), gb = pw == wn ? 1.f : ex2(pw - wn);
        ls[k] = fmaf(ls[k], fa, pl * fb);
        mx[k] = mn, wx[k] = wn;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          o[k][2 * e] = fmaf(o[k][2 * e], ga, v[b][k][e].x * gb);
          o[k][2 * e + 1] = fmaf(o[k][2 * e + 1], ga, v[b][k][e].y * gb);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kFewCols; ++k) {
    const int c = d.z + c0 + k;
    if (c0 + k < ncols) finish_lane<E>(p, d.x + c / p.group, d.y * p.group + c % p.group, lane, o[k], mx[k], wx[k], ls[k]);
  }
}


template <int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const AttnParams p, int cb) {
  grid_wait();
  join_many<D>(p, cb, blockIdx.x);
}
template <int D, int PARTS>
__global__ void __launch_bounds__(256) kv_join_few_kernel(const AttnParams p) {
  grid_wait();
  join_few<D, PARTS>(p);
}
// Of a call that ran both kernels: the first `tiled` blocks of a row join the tiled
// one's items.  (In a launch of their own the split kernel's, of which such a call may
// have none, took 3 us more.)
template <int D, int PARTS>
__global__ void __launch_bounds__(256) kv_join_both_kernel(const AttnParams t, const AttnParams p, int tiled, int cb) {
  grid_wait();
  if ((int)blockIdx.x < tiled) join_few<D, PARTS>(t);
  else join_many<D>(p, cb, blockIdx.x - tiled);
}
}  // namespace

cudaError_t launch_kv_join(const AttnParams &p, int nb, int ctas, cudaStream_t stream) {
  const dim3 grid(ctas, 4 * nb);
  return p.c.dim == 64 ? launch_after(kv_join_kernel<64>, grid, 256, 0, stream, true, p, 8 * nb)
                       : launch_after(kv_join_kernel<128>, grid, 256, 0, stream, true, p, 8 * nb);
}

cudaError_t launch_kv_join_tiled(const AttnParams &p, int ctas, bool many, cudaStream_t stream) {
  const dim3 grid(ctas, kTiledCols / (8 * kFewCols));
  auto run = [&](auto *kernel) { return launch_after(kernel, grid, 256, 0, stream, true, p); };
  if (p.c.dim == 64) return many ? run(kv_join_few_kernel<64, kManyParts>) : run(kv_join_few_kernel<64, 1>);
  return many ? run(kv_join_few_kernel<128, kManyParts>) : run(kv_join_few_kernel<128, 1>);
}

cudaError_t launch_kv_join_both(const AttnParams &t, int tiled_ctas, bool many, const AttnParams &p, int nb, int ctas,
                                cudaStream_t stream) {
  constexpr int kRows = kTiledCols / (8 * kFewCols);
  const dim3 grid(tiled_ctas + ctas, kRows > 4 * nb ? kRows : 4 * nb);
  auto run = [&](auto *kernel) { return launch_after(kernel, grid, 256, 0, stream, true, t, p, tiled_ctas, 8 * nb); };
  if (p.c.dim == 64) return many ? run(kv_join_both_kernel<64, kManyParts>) : run(kv_join_both_kernel<64, 1>);
  return many ? run(kv_join_both_kernel<128, kManyParts>) : run(kv_join_both_kernel<128, 1>);
}

#endif  // MQA_KV_KIND == 0

namespace {

template <int D, int NB>
cudaError_t launch(const AttnParams &p, const CUtensorMap &k_map, const CUtensorMap &v_map, int ctas, bool follows,
                   cudaStream_t stream) {
  constexpr size_t bytes = sizeof(Smem<D, NB, MQA_KV_KIND, false>) + 1024;
  static DeviceFlags done[3];
  auto run = [&](auto *kernel, DeviceFlags &flags) {
    const cudaError_t e = allow_smem(kernel, bytes, flags);
    return e != cudaSuccess ? e
                            : launch_after(kernel, dim3(ctas), kAttnThreads, bytes, stream, follows, p, k_map, v_map);
  };
#if MQA_KV_KIND == 0
  return p.selected ? run(kv_attn_kernel<D, NB, kSelected, false>, done[0])
         : p.test   ? run(kv_attn_kernel<D, NB, kDense, true>, done[1])
                    : run(kv_attn_kernel<D, NB, kDense, false>, done[2]);
#else
  return run(kv_attn_kernel<D, NB, MQA_KV_KIND, false>, done[0]);
#endif
}

template <int D>
cudaError_t launch_d(const AttnParams &p, const CUtensorMap &k_map, const CUtensorMap &v_map, int nb, int ctas,
                     bool follows, cudaStream_t stream) {
  switch (nb) {
    case 1: return launch<D, 1>(p, k_map, v_map, ctas, follows, stream);
    case 2: return launch<D, 2>(p, k_map, v_map, ctas, follows, stream);
    case 3: return launch<D, 3>(p, k_map, v_map, ctas, follows, stream);
    default: return launch<D, 4>(p, k_map, v_map, ctas, follows, stream);
  }
}
}  // namespace

template <>
cudaError_t launch_kv_attention<MQA_KV_KIND>(const AttnParams &p, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                             int nb, int ctas, bool follows, cudaStream_t stream) {
  return p.c.dim == 64 ? launch_d<64>(p, k_map, v_map, nb, ctas, follows, stream)
                       : launch_d<128>(p, k_map, v_map, nb, ctas, follows, stream);
}

}  // namespace mqa
