// kvq_tree.cu -- attention of drafted tokens over the 8-bit pool: split-K, flash-shaped, on the tcgen05 tensor cores.
//
// The last n_b stored tokens of sequence b are drafted; query row (i, h) sees every token before them and those
// drafted tokens whose bit is set in its mask:
//   out[i][h] = sum_t softmax_t(sm_scale q[i][h].K[t]) V[t]   over t < L - n, and t = L - n + j with bit j set.
// Rows are few (n_b times the heads of a kv head) and contexts long, so the work is reading K and V once:
// 2 * Hkv * D * 17/16 bytes per token.  Blocks of 128 rows of one (sequence, kv head) share every dequantized tile:
//   S[128 rows][T keys] = Q . Kd^T,   O[128 rows][D] += P . Vd      (T = 128 at D = 128, 64 at D = 256)
// Q, S, P (over the S it was made from) and O are in tensor memory, one row per lane; K and V are bf16 tiles in 128-byte
// swizzled shared memory, two of each.  MMAs of different accumulators are not ordered among themselves, so the QK
// that next writes an S buffer waits for the PV that reads the P in it.
//
// Work split.  A unit is one tile of T keys for one block of rows; units are numbered by (sequence, row block,
// kv head, tile), and CTA c of C takes the units [c U / C, (c + 1) U / C): every CTA gets the same number of tiles to
// within one, whatever the lengths, and reads a contiguous run of each sequence.  The run is cut into segments, one
// per (sequence, row block, kv head); only a CTA's first and last segment can be parts of a block, so two partial
// slots per CTA suffice.  A segment that is a whole block writes its output; the others write (m, l, O) and
// the merge kernel (a programmatic dependent) joins the segments of each row.
//
// Masks.  Visibility of a half tile's keys is one 64-bit word per row: ones before the drafted tokens, the
// row's mask bits among them, zeros behind the end, and zeros for masked pages.  Where a row of a warp does not see a
// key, its score is set to -inf first; the passes of the softmax have one variant.
//
// Roles of a CTA's 28 warps: 0-7 softmax (two per lane quarter, each on half of a tile's keys; quarters without a row
// only keep the barriers' counts), 8-15 dequantize K and 16-23 V, 26 looks up pages, 27 issues the MMAs.
//
// Measured: 32 sequences of 3..16 drafted tokens over 0.7k..8k, 4 heads per kv head (q8_0): 113 us in a graph, 2.9
// TB/s; 4 x 32 over 64k at head_dim 256, 8 heads per kv head (two blocks): 162 us, 847 TFLOP/s.  What bounds it: the
// latency of the softmax's chain.  Of a tile's 2950 clocks (first case) the softmax warps wait 300, the dequant warps
// 1050 and the MMA warp 2000: blocks of 12 to 64 rows leave the softmax to one or two of four lane quarters, whose two
// passes and the meeting between them follow one another.  No unit is full (issue slots 57%, tensor pipe 36%, DRAM 39%;
// the first stall is long_scoreboard).  Of 2700 clocks (second case) the three wait 700, 1050 and 1200 on one another, and
// each of the two blocks converts every tile for itself.  What the steps were worth, first case / second: one copy of the dequant code for K and V, one masked pass, eight MMAs per
// elect 183 -> 159 / 218; K and V by warps of their own 157 / 204; the merge by a warp per row and without a clearing
// launch 146 / 201; loads straight into registers instead of a staging ring, conflict-free stores without selects,
// waits' unlikely parts out of line 131 / 178; Q and P in tensor memory 124 / 168.  Measured slower, and not kept:
// sixteen warps each taking K and then V (166), rows repeated in idle lane quarters with the keys divided among them
// (137 / 183), one register set per warp rotated by moves (147); (against 117) scores kept in registers from the
// maximum to P (125), a dequant warp less beside the softmax of short blocks (123), the MMA loop without the branches
// of its first steps (120), no mask words on tiles without masks (117 / 169).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "kvq_device.cuh"
#include "kvq_flash.cuh"
#include "kvq_internal.h"
#include "kvq_plan.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace {

constexpr int kM = 128;  // query rows per block (the MMA M)
constexpr int kSmWarps = 8;  // two per tensor-memory lane quarter, each on half of a tile's keys
constexpr int kDwWarps = 8;  // of K, and of V
constexpr int kVWarp = kSmWarps + kDwWarps;     // warp 16: first of V
// Warps 24 and 25 only fill up: a lane quarter's softmax runs on the SM sub-partition of its number, blocks that are not
// full use the first quarters, and so the two other roles belong on the last sub-partitions (123 -> 117 us at 12..64 rows).
constexpr int kPlanWarp = kVWarp + kDwWarps + 2;  // warp 26: pages of the tiles to come
constexpr int kMmaWarp = kPlanWarp + 1;           // warp 27
constexpr int kThreads = (kMmaWarp + 1) * 32;     // 28 warps
constexpr int kDwThreads = kDwWarps * 32;
constexpr int kTmemCols = 512;
constexpr int kMeta = 8;               // tiles whose pages are looked up ahead
constexpr float kLazyRescale = 8.0f;   // log2 headroom before the running max must move

template <int D>
struct TCfg {
  static constexpr int T = (D == 128) ? 128 : 64;  // keys per tile
  static constexpr int PPT = T / kPage;            // pages per tile
  static constexpr int CHUNK = T * 128;            // bytes of a 64-column chunk of a K or V tile
  static constexpr int KV_TILE = T * D * 2;        // one bf16 K or V tile
  static constexpr int NB = D / 32;                // scale blocks of a row
  // A dequant warp converts 2 KB of codes of K or V per tile: four 16-byte pieces per lane, consecutive lanes
  // consecutive pieces of a row.
  static constexpr int CPR = D / 16;               // pieces of a row
  static constexpr int RPI = 32 / CPR;             // rows per load
  static constexpr int RPW = 4 * RPI;              // rows per warp
  static constexpr int K_OFF = 0;                  // [2] bf16 K tiles; 1024-byte aligned: swizzle atoms
  static constexpr int V_OFF = K_OFF + 2 * KV_TILE;  // [2] bf16 V tiles
  static constexpr int BASE_OFF = V_OFF + 2 * KV_TILE;              // [kMeta][PPT] pool row group of each page, or -1
  static constexpr int NVAL_OFF = BASE_OFF + kMeta * PPT * 8;   // [kMeta][PPT] valid tokens
  static constexpr int RED_OFF = NVAL_OFF + kMeta * PPT * 4;    // [2 parities][2 halves][128 rows] row maxima
  static constexpr int SUM_OFF = RED_OFF + 2 * 2 * kM * 4;      // [2 item parities][2 halves][128 rows] row sums
  static constexpr int TAB_OFF = SUM_OFF + 2 * 2 * kM * 4;      // [batch + 1] units before each sequence
  static constexpr int NBARS = 2 * kMeta + 14 + 12;
  static constexpr int BAR_OFF = (TAB_OFF + (kMaxTreeBatch + 1) * 4 + 15) / 16 * 16;  // mbarriers: 8-byte aligned
  static constexpr int SMEM_BYTES = BAR_OFF + NBARS * 8 + 16 + 1024;  // + slack to align the base
  // tensor-memory columns: O [0, D); Q (bf16, two per column) [D, D + D / 2); S buffer b [S_COL + b T, + T).  P replaces
  // the S it was made from: half hf of the keys takes the first T / 4 columns of its own T / 2.
  static constexpr int Q_COL = D;
  static constexpr int S_COL = D + D / 2;
  static_assert(D == 128 || D == 256, "the tree kernel needs head_dim 128 or 256");
  static_assert(S_COL + 2 * T <= kTmemCols, "tensor-memory columns");
  static_assert(kDwWarps * RPW == T && kPage % RPW == 0, "dequant split");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// Drafted tokens of sequence b after validation; 0 for an inconsistent one (reported in `report`, if given).
__device__ __forceinline__ int32_t drafted(const TreeArgs& a, int32_t b, uint32_t* report) {
  const int32_t q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1), L = __ldg(a.seq_lens + b);
  const int32_t n = q1 - q0;
  if (q0 < 0 || n < 0 || q1 > a.total_q || n > L || n > 64 * a.mask_words ||
      L > static_cast<int64_t>(a.max_pages) * kPage) {
    set_status(report, kStatusBadExtend);
    return 0;
  }
  return n;
}

// The last valid sequence that covers query row i, or -1, when q_start falls and so does not order the sequences: wrong
// entries take nothing from the valid sequences beside them.  (Out of line, and its condition in shared memory: in the
// dequant warps' code and registers it cost 1%, 112.3 -> 113.7 us at 32 sequences of 3..16 drafts.)
__device__ __noinline__ int32_t search_sequence(const int32_t* q_start, const int32_t* seq_lens, int32_t batch,
                                                int32_t total_q, int32_t max_drafts, int64_t max_tokens, int32_t i) {
  int32_t b = batch - 1;
  for (; b >= 0; --b) {
    const int32_t q0 = __ldg(q_start + b), q1 = __ldg(q_start + b + 1), L = __ldg(seq_lens + b);
    if (q0 >= 0 && q0 <= i && i < q1 && q1 <= total_q && q1 - q0 <= L && q1 - q0 <= max_drafts && L <= max_tokens) break;
  }
  return b;
}

__device__ __forceinline__ int32_t row_blocks(int32_t n, int32_t G) { return (n * G + kM - 1) / kM; }

// A segment: the tiles [t0, t1) of row block blk of (sequence b, kv head g); slot: where its partial goes, or -1
// when the segment is the whole block.
struct Seg {
  int32_t b, g, blk, n, L, q0, rows, t0, t1, slot;
};

struct Range {
  int32_t u0, u1;  // units of this CTA
};

// The units of CTA c when C CTAs share U.
__device__ __forceinline__ int32_t range_start(int32_t U, int32_t C, int32_t c) {
  return static_cast<int32_t>(static_cast<int64_t>(U) * c / C);
}

template <int D>
__device__ __forceinline__ Seg locate(const int32_t* tab, const TreeArgs& a, int32_t G, const Range& r, int32_t u) {
  using Cfg = TCfg<D>;
  int lo = 0, hi = a.batch;  // first b with tab[b] > u
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (tab[mid] <= u) lo = mid + 1;
    else hi = mid;
  }
  Seg s;
  s.b = lo - 1;
  s.L = __ldg(a.seq_lens + s.b);
  s.q0 = __ldg(a.q_start + s.b);
  s.n = drafted(a, s.b, nullptr);
  const int32_t nt = (s.L + Cfg::T - 1) / Cfg::T;
  const int32_t local = u - tab[s.b];
  const int32_t item = local / nt;
  s.blk = item / a.num_kv_heads;
  s.g = item - s.blk * a.num_kv_heads;
  s.rows = min(kM, s.n * G - s.blk * kM);
  s.t0 = local - item * nt;
  s.t1 = min(nt, s.t0 + (r.u1 - u));
  const bool whole = s.t0 == 0 && s.t1 == nt;
  s.slot = whole ? -1 : 2 * static_cast<int32_t>(blockIdx.x) + (u == r.u0 ? 0 : 1);
  return s;
}

// The (segment, tile) pairs of this CTA, in order.
template <int D>
struct TreeIter {
  Seg s;
  Range r;
  int32_t u, t;  // first unit of the segment; tile
  bool live;
  __device__ __forceinline__ void first(const int32_t* tab, const TreeArgs& a, int32_t G, const Range& range) {
    r = range;
    u = r.u0;
    live = u < r.u1;
    if (live) {
      s = locate<D>(tab, a, G, r, u);
      t = s.t0;
    }
  }
  __device__ __forceinline__ void next_segment(const int32_t* tab, const TreeArgs& a, int32_t G) {
    u += s.t1 - s.t0;
    live = u < r.u1;
    if (live) {
      s = locate<D>(tab, a, G, r, u);
      t = s.t0;
    }
  }
  __device__ __forceinline__ void next(const int32_t* tab, const TreeArgs& a, int32_t G) {
    if (!live) return;
    if (++t < s.t1) return;
    next_segment(tab, a, G);
  }
};

template <int D>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  if constexpr (D == 128) return warp_wait_far(bar, parity);
  else return warp_wait(bar, parity);
}

// 16 ones for each set bit of a 4-bit page mask.
__device__ __forceinline__ uint64_t spread_pages(uint32_t m) {
  uint64_t v = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) v |= ((m >> i) & 1u) ? (0xFFFFull << (16 * i)) : 0ull;
  return v;
}

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(const TreeArgs a) {
  using Cfg = TCfg<D>;
  constexpr int T = Cfg::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // swizzle atoms are 1024 B
  uint8_t* sK = smem + Cfg::K_OFF;
  uint8_t* sV = smem + Cfg::V_OFF;
  int64_t* sBase = reinterpret_cast<int64_t*>(smem + Cfg::BASE_OFF);
  int32_t* sNval = reinterpret_cast<int32_t*>(smem + Cfg::NVAL_OFF);
  int32_t* sTab = reinterpret_cast<int32_t*>(smem + Cfg::TAB_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFF);
  // Every barrier completes once per use of its buffer, so a waiter names an unambiguous phase.
  uint64_t* bar_meta = bars;                      // [kMeta] a tile's pages written
  uint64_t* bar_meta_free = bars + kMeta;         // [kMeta] ... read by every dequant warp
  uint64_t* bar_k_full = bars + 2 * kMeta;        // [2] K tile b written (K warps)
  uint64_t* bar_v_full = bar_k_full + 2;          // [2] V tile b written (V warps)
  uint64_t* bar_qk_done = bar_k_full + 4;         // [2] QK into S buffer b completed (commit)
  uint64_t* bar_pv_done = bar_k_full + 6;         // [2] PV that read P buffer b completed (commit)
  uint64_t* bar_p_full = bar_k_full + 8;          // [2] P buffer b written, S buffer b read (softmax warps)
  uint64_t* bar_q_full = bar_k_full + 10;         // a segment's Q rows written (softmax warps), once per segment
  uint64_t* bar_o_free = bar_k_full + 11;         // a segment's O read out (softmax warps), once per segment
  uint64_t* bar_pair = bar_k_full + 14;           // [4 quarters][2 parities] both half-tile maxima written
  uint64_t* bar_sum = bar_k_full + 22;            // [4 quarters] both half row sums written, once per segment
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + Cfg::BAR_OFF + Cfg::NBARS * 8);  // address; does q_start fall?

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t G = a.num_q_heads / a.num_kv_heads;

  // Each CTA has a status word of its own, which the merge kernel sums up: no clearing launch before this one.
  uint32_t* my_status = a.cta_status + blockIdx.x;
  if (tid == 0) *my_status = 0;
  __syncthreads();

  // ---- plan: units before every sequence
  bool falls = false;  // q_start falls somewhere
  for (int32_t b = tid; b < a.batch; b += kThreads) {
    falls |= __ldg(a.q_start + b + 1) < __ldg(a.q_start + b);
    const int32_t n = drafted(a, b, blockIdx.x == 0 ? my_status : nullptr);
    sTab[b + 1] = n == 0 ? 0 : row_blocks(n, G) * a.num_kv_heads * ((__ldg(a.seq_lens + b) + T - 1) / T);
  }
  if (tid == 0) {
    sTab[0] = 0;
    for (int s = 0; s < kMeta; ++s) {
      mbar_init(&bar_meta[s], 1);
      mbar_init(&bar_meta_free[s], 2 * kDwWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bar_k_full[b], kDwWarps);
      mbar_init(&bar_v_full[b], kDwWarps);
      mbar_init(&bar_qk_done[b], 1);
      mbar_init(&bar_pv_done[b], 1);
      mbar_init(&bar_p_full[b], kSmWarps);
    }
    mbar_init(bar_q_full, kSmWarps);
    mbar_init(bar_o_free, kSmWarps);
    for (int i = 0; i < 12; ++i) mbar_init(&bar_pair[i], 2);
    fence_mbar_init();
  }
  falls = __syncthreads_or(falls);
  if (tid == 0) sTmem[1] = falls;
  if (warp == 0) {  // inclusive prefix, 32 sequences at a time
    int32_t run = 0;
    for (int32_t b0 = 0; b0 < a.batch; b0 += 32) {
      const int32_t b = b0 + lane;
      int32_t x = b < a.batch ? sTab[b + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < a.batch) sTab[b + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sTmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sTmem;
  // the merge kernel may launch now; it waits for this grid to complete before it reads
  asm volatile("griddepcontrol.launch_dependents;");
  const int32_t U = sTab[a.batch];
  const int32_t C = max(1, min(a.grid, U));  // CTAs that share the units
  Range range;
  range.u0 = static_cast<int32_t>(blockIdx.x) < C ? range_start(U, C, blockIdx.x) : 0;
  range.u1 = static_cast<int32_t>(blockIdx.x) < C ? range_start(U, C, blockIdx.x + 1) : 0;
  if (blockIdx.x == 0) {  // the plan, for the merge
    for (int32_t b = tid; b <= a.batch; b += kThreads) a.tab[b] = sTab[b];
    if (tid == 0) a.tab[a.batch + 1] = C;
  }
  bool ok = true;

  if (warp == kPlanWarp) {
    // ===================================================================== pages of the tiles to come
    // Lane pi (< PPT) owns page pi of a tile: its block-table entry (read one tile ahead) and valid tokens.
    auto page_entry = [&](const TreeIter<D>& ti) -> int32_t {
      if (!ti.live || lane >= Cfg::PPT) return -1;
      const int32_t pg = ti.t * Cfg::PPT + lane;
      if (pg >= a.max_pages || pg * kPage >= ti.s.L) return -1;
      return __ldg(a.block_table + static_cast<int64_t>(ti.s.b) * a.max_pages + pg);
    };
    TreeIter<D> t;
    t.first(sTab, a, G, range);
    int32_t bt = page_entry(t);
    for (uint32_t n = 0; t.live; ++n) {
      int32_t phys = bt;
      if (phys >= a.num_pages) {  // never dereferenced; reported in the status word
        set_status(my_status, kStatusBadPage);
        phys = -1;
      }
      const int32_t nval = phys >= 0 ? min(kPage, t.s.L - (t.t * Cfg::PPT + lane) * kPage) : 0;
      const int32_t g = t.s.g;
      t.next(sTab, a, G);
      bt = page_entry(t);
      const uint32_t sl = n % kMeta;
      if (n >= kMeta && !wait<D>(&bar_meta_free[sl], (n / kMeta - 1) & 1)) { ok = false; break; }
      if (lane < Cfg::PPT) {
        sBase[sl * Cfg::PPT + lane] = phys >= 0 ? static_cast<int64_t>(phys) * 2 * a.num_kv_heads + g : -1;
        sNval[sl * Cfg::PPT + lane] = nval;
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&bar_meta[sl]);
    }
  } else if (warp >= kSmWarps && warp < kVWarp + kDwWarps) {
    // ===================================================================== dequant warps
    // Eight for K and eight for V, one copy of the code for both (with four roles on an SM, instruction-cache
    // misses cost more than the selects).  A warp's codes and scales come straight from the pool into registers, two
    // tiles ahead (a staging ring would cost their bytes twice more in shared-memory bandwidth, which two bf16 tiles of K
    // and V and the MMAs' reads of them already use), and leave as bf16 in 128-byte swizzled rows.
    const int kv = warp >= kVWarp ? 1 : 0;
    const int wi = warp - (kv ? kVWarp : kSmWarps);
    // piece c of a row and first row (token) of the tile: four lanes take neighbouring pieces, the next four the same
    // pieces of the next row, whose swizzle differs in the lowest bit; so eight lanes' stores fall into eight banks
    const int c = (lane & 3) | ((lane >> 3) % (Cfg::CPR / 4)) << 2;
    const int r0 = wi * Cfg::RPW + ((lane >> 2) & 1) + 2 * (lane / (2 * Cfg::CPR));
    const int page = wi * Cfg::RPW / kPage, off0 = r0 % kPage;
    const uint32_t total = range.u1 - range.u0;  // tiles of this CTA
    // While the first tile is on its way, the V warps write down the sequence of each query row for the merge, the
    // CTAs taking rows in turn: the last sequence whose rows begin at or before it, -1 where that one does not reach it.
    auto write_row_seq = [&]() {
      for (int32_t i = blockIdx.x * kDwThreads + wi * 32 + lane; i < a.total_q; i += gridDim.x * kDwThreads) {
        int32_t b;
        if (sTmem[1]) {  // q_start falls somewhere
          b = search_sequence(a.q_start, a.seq_lens, a.batch, a.total_q, 64 * a.mask_words,
                              static_cast<int64_t>(a.max_pages) * kPage, i);
        } else {
          int lo = 0, hi = a.batch;  // first b with q_start[b] > i
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.q_start + mid) <= i) lo = mid + 1;
            else hi = mid;
          }
          b = lo - 1;
          if (b >= 0 && !(i >= __ldg(a.q_start + b) && i < __ldg(a.q_start + b) + drafted(a, b, nullptr))) b = -1;
        }
        a.row_seq[i] = b;
      }
    };
    struct Pieces {
      uint4 codes[4];
      uint16_t sc[4];
    };
    // (what lies in unwritten or masked rows does not matter: zero codes times a zero scale)
    auto fetch = [&](uint32_t i, Pieces& p) -> bool {
      const uint32_t sl = i % kMeta;
      if (!wait<D>(&bar_meta[sl], (i / kMeta) & 1)) return false;
      const int64_t base = sBase[sl * Cfg::PPT + page];
      const int32_t nval = sNval[sl * Cfg::PPT + page];
      __syncwarp();
      if (lane == 0) bar_arrive(&bar_meta_free[sl]);
      const int64_t row = (base + (kv ? a.num_kv_heads : 0)) * kPage + off0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p.codes[j] = make_uint4(0u, 0u, 0u, 0u);
        p.sc[j] = 0;
        if (off0 + j * Cfg::RPI < nval) {
          p.codes[j] = ldg_stream(a.codes + (row + j * Cfg::RPI) * D + c * 16);
          if (KindTraits<KIND>::kScaled) p.sc[j] = __ldg(a.scales + (row + j * Cfg::RPI) * Cfg::NB + c / 2);
        }
      }
      return true;
    };
    uint64_t* done = kv ? bar_pv_done : bar_qk_done;
    uint64_t* full = kv ? bar_v_full : bar_k_full;
    // where this lane's first piece goes in a tile: its 64-column chunk, its row, its two 16-byte halves swizzled
    // by the row; rows 8 apart share the swizzle, so later pieces are a constant xor and sum away
    const uint32_t at = smem_u32(kv ? sV : sK) + (c / 4) * Cfg::CHUNK + r0 * 128 + (((2 * (c % 4)) ^ (r0 & 7)) * 16);
    // tile i out of its registers, which then take tile i + 2
    auto step = [&](uint32_t i, Pieces& p) -> bool {
      // the buffer was last read by the QK (PV) two tiles back
      if (i >= 2 && !wait<D>(&done[i & 1], ((i >> 1) - 1) & 1)) return false;
      const uint32_t dst = at + (i & 1) * Cfg::KV_TILE;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t w[8];
        dequant16<KIND>(p.codes[j], p.sc[j], w);
        const uint32_t d = (dst ^ ((j * Cfg::RPI & 7) * 16)) + j * Cfg::RPI * 128;
        sts16(d, w[0], w[1], w[2], w[3]);
        sts16(d ^ 16, w[4], w[5], w[6], w[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(&full[i & 1]);
      return i + 2 >= total || fetch(i + 2, p);
    };
    Pieces even, odd;
    ok = (total < 1 || fetch(0, even)) && (total < 2 || fetch(1, odd));
    if (kv == 1) write_row_seq();
    for (uint32_t i = 0; ok && i < total; i += 2) {
      ok = step(i, even);
      if (ok && i + 1 < total) ok = step(i + 1, odd);
    }
  } else if (warp == kMmaWarp) {
    // ===================================================================== MMA issue (elected lane)
    const uint32_t idesc_qk = x_idesc(T, false);
    const uint32_t idesc_pv = x_idesc(D, true);
    // K: K-major in 128-byte swizzled rows, a k-step is 32 bytes along a 64-column chunk.  V: MN-major in the same rows, a
    // k-step is 16 of them.  Q and P in tensor memory, a k-step is 8 columns.
    const uint64_t dK = sw128_desc(smem_u32(sK), 16, 1024);
    const uint64_t dV = sw128_desc(smem_u32(sV), Cfg::CHUNK, 1024);
    const uint32_t tQ = tmem + Cfg::Q_COL, tS = tmem + Cfg::S_COL, tO = tmem;
    uint32_t n = 0, items = 0;  // tiles QK'd; items finished
    // PV of tile m; the first tile of an item overwrites O, once the previous item's O has been read out
    auto pv = [&](uint32_t m, bool first) -> bool {
      const int bp = m & 1;
      if (!wait<D>(&bar_v_full[bp], (m >> 1) & 1)) return false;
      if (!wait<D>(&bar_p_full[bp], (m >> 1) & 1)) return false;
      if (first && items >= 1 && !wait<D>(bar_o_free, (items - 1) & 1)) return false;
      tc_fence_after();
      const uint64_t v = dV + bp * static_cast<uint64_t>(Cfg::KV_TILE >> 4);
      const uint32_t p = tS + bp * T;
      constexpr uint64_t step = (16 * 128) >> 4;
      if constexpr (T == 128) {
        mma4_bf16_tmem_a(tO, p, 8u, v, step, idesc_pv, first ? 0u : 1u);
        mma4_bf16_tmem_a(tO, p + T / 2, 8u, v + 4 * step, step, idesc_pv, 1u);
      } else {
        mma2x2_bf16_tmem_a(tO, p, p + T / 2, v, step, idesc_pv, first ? 0u : 1u);
      }
      mma_commit(&bar_pv_done[bp]);
      __syncwarp();
      return true;
    };
    TreeIter<D> t;
    for (t.first(sTab, a, G, range); ok && t.live; t.next_segment(sTab, a, G)) {
      const int32_t ntiles = t.s.t1 - t.s.t0;
      if (!wait<D>(bar_q_full, items & 1)) { ok = false; break; }
      for (int32_t i = 0; i < ntiles; ++i, ++n) {
        const int b = n & 1;
        if (!wait<D>(&bar_k_full[b], (n >> 1) & 1)) { ok = false; break; }
        // S buffer b holds P of tile n - 2: its PV, whose P came after the softmax had read S, must have completed
        if (n >= 2 && !wait<D>(&bar_pv_done[b], ((n >> 1) - 1) & 1)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < D / 64; ++q)
          mma4_bf16_tmem_a(tS + b * T, tQ + q * 32, 8u,
                           dK + b * static_cast<uint64_t>(Cfg::KV_TILE >> 4) + static_cast<uint64_t>((q * Cfg::CHUNK) >> 4),
                           32 >> 4, idesc_qk, q > 0 ? 1u : 0u);
        mma_commit(&bar_qk_done[b]);
        __syncwarp();
        if (i > 0 && !pv(n - 1, i == 1)) { ok = false; break; }
      }
      if (!ok) break;
      if (!pv(n - 1, ntiles == 1)) { ok = false; break; }
      ++items;
    }
    // before tensor memory is freed, every MMA issued must have completed (the last commit implies all)
    if (n > 0) (void)mbar_wait_bounded(&bar_pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
    if (n > 0) (void)mbar_wait_bounded(&bar_qk_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
  } else if (warp < kSmWarps) {
    // ===================================================================== softmax warps
    const int quarter = warp & 3, hf = warp >> 2;  // lane quarter; which half of the keys and of O
    const int r = quarter * 32 + lane;             // query row = tensor-memory lane
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + Cfg::S_COL + lane_base + hf * (T / 2);
    const uint32_t tO = tmem + lane_base + hf * (D / 2);
    float* sRed = reinterpret_cast<float*>(smem + Cfg::RED_OFF);
    float* sSum = reinterpret_cast<float*>(smem + Cfg::SUM_OFF);
    // this warp's half of the segment's Q rows into tensor memory (rows past the block's are zero): as the A operand of
    // every tile's QK they would otherwise cost 2 * 128 * D bytes of shared-memory reads a tile
    auto write_q = [&](const Seg& s) {
      if (quarter * 32 < s.rows) {
        const bool valid = r < s.rows;
        const int32_t row = s.blk * kM + (valid ? r : 0);
        const int32_t tok = row / G;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + (static_cast<int64_t>(s.q0 + tok) * a.num_q_heads + s.g * G + (row - tok * G)) * D + hf * (D / 2));
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 x = valid ? __ldg(src + c * 4 + j) : make_uint4(0, 0, 0, 0);
            w[4 * j] = x.x;
            w[4 * j + 1] = x.y;
            w[4 * j + 2] = x.z;
            w[4 * j + 3] = x.w;
          }
          tmem_st16u(tmem + Cfg::Q_COL + lane_base + hf * (D / 4) + c * 16, w);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) bar_arrive(bar_q_full);
    };
    // the two warps of a lane quarter meet on mbarriers (bounded waits: a warp that gave up cannot strand
    // the other)
    auto pair_meet = [&](uint64_t* bar, uint32_t parity) -> bool {
      __syncwarp();
      if (lane == 0) bar_arrive(bar);
      return wait<D>(bar, parity);
    };
    // tiles processed; segments; row sums exchanged and phases of the maxima's barriers (both only of segments in
    // which this lane quarter holds rows)
    uint32_t n = 0, items = 0, sums = 0, pair_phase = 0;
    TreeIter<D> cur;
    cur.first(sTab, a, G, range);
    if (cur.live) write_q(cur.s);
    while (ok && cur.live) {
      const Seg s = cur.s;
      const bool active = quarter * 32 < s.rows;  // (warp-uniform) this lane quarter holds rows
      const bool row_ok = r < s.rows;
      const int32_t row = s.blk * kM + (row_ok ? r : 0);
      const int32_t tok = row / G;
      const int64_t* mask = a.mask + static_cast<int64_t>(s.q0 + tok) * a.mask_words;
      float m_used = -INFINITY, l = 0.0f;
      // lane pi (< PPT) holds the block-table entry of page pi of a tile, read one tile ahead of its use
      auto fetch = [&](int32_t t) -> int32_t {
        const int32_t pg = t * Cfg::PPT + lane;
        if (lane >= Cfg::PPT || t >= s.t1 || pg >= a.max_pages || pg * kPage >= s.L) return -1;
        return __ldg(a.block_table + static_cast<int64_t>(s.b) * a.max_pages + pg);
      };
      int32_t ent = active ? fetch(s.t0) : -1;
      for (int32_t t = s.t0; t < s.t1; ++t, ++n) {
        const int b = n & 1;
        if (!active) {  // only keep the count of the tile's barrier
          if (!wait<D>(&bar_qk_done[b], (n >> 1) & 1)) { ok = false; break; }
          if (lane == 0) bar_arrive(&bar_p_full[b]);
          continue;
        }
        // mapped pages of the tile (chunk c of 16 keys is page c of the tile)
        const uint32_t pmask = __ballot_sync(0xffffffffu, ent >= 0 && ent < a.num_pages) & ((1u << Cfg::PPT) - 1u);
        ent = fetch(t + 1);
        // keys of this warp's half that this row sees
        const int32_t k0 = t * T + hf * (T / 2);
        uint64_t vis = spread_pages(pmask >> (hf * Cfg::PPT / 2));
        if (k0 + T / 2 > s.L - s.n) {  // (warp-uniform) drafted tokens, or keys behind the end
          vis &= tree_window(mask, a.mask_words, k0 - (s.L - s.n));
          const int32_t left = s.L - k0;
          vis &= left >= 64 ? ~0ull : left > 0 ? (1ull << left) - 1ull : 0ull;
        }
        constexpr uint64_t kAll = T / 2 == 64 ? ~0ull : (1ull << (T / 2)) - 1ull;
        vis = row_ok ? vis & kAll : kAll;  // (rows past the block's are zeros that nobody reads)
        if (!wait<D>(&bar_qk_done[b], (n >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        // Keys that some row of the warp does not see: their scores become -inf in tensor memory first, so that the
        // passes below need one variant only.
        if (!__all_sync(0xffffffffu, vis == kAll)) {
#pragma unroll 1
          for (int h = 0; h < T / 64; ++h) {
            uint32_t v[32];
            tmem_ld32(tS + b * T + h * 32, v);
            const uint32_t vw = static_cast<uint32_t>(vis >> (32 * h));
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = ((vw >> e) & 1u) ? v[e] : 0xFF800000u;
            tmem_st32(tS + b * T + h * 32, v);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        // pass 1: the row's max over this half (sm_scale > 0: scaling commutes with it)
        float mh = -INFINITY;
#pragma unroll 1
        for (int h = 0; h < T / 64; ++h) {
          uint32_t v[32], top;
          tmem_ld32_max_issue(tS + b * T + h * 32, v, top);
          tmem_wait_max(top);
          mh = fmaxf(mh, __uint_as_float(top));
        }
        // the row's max over the whole tile: exchange halves with the other warp of the lane quarter
        // (double-buffered by tile parity, so one barrier per tile suffices)
        sRed[(b * 2 + hf) * kM + r] = mh;
        if (!pair_meet(&bar_pair[quarter * 2 + b], (pair_phase >> b) & 1u)) { ok = false; break; }
        pair_phase ^= 1u << b;
        float mx = fmaxf(sRed[(b * 2) * kM + r], sRed[(b * 2 + 1) * kM + r]);
        if (mx > -INFINITY) mx *= a.score_scale;
        float alpha = 1.0f;
        bool resc = false;
        if (mx > -INFINITY && (m_used == -INFINITY || mx > m_used + kLazyRescale)) {
          if (m_used != -INFINITY) {
            alpha = ex2(m_used - mx);
            resc = true;
          }
          m_used = mx;
        }
        if (__any_sync(0xffffffffu, resc)) {  // (only from the second tile of an item on)
          // O must hold the PV of the previous tile before it is scaled; this warp scales its half of O
          if (!wait<D>(&bar_pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + c * 32, o);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          l *= alpha;
        }
        // pass 2: P = 2^(s * scale - m) of this half as bf16 into tensor memory; the row sum in fp32.  (A row without
        // a visible key so far has only scores of -inf: any finite m gives zeros.)
        const float m_fin = m_used == -INFINITY ? 0.0f : m_used;
        const float2 sc2 = make_float2(a.score_scale, a.score_scale), m2 = make_float2(-m_fin, -m_fin);
        float2 ls[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll 1
        for (int h = 0; h < T / 64; ++h) {
          uint32_t v[32];
          tmem_ld32(tS + b * T + h * 32, v);
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = ffma2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), sc2, m2);
            const float2 p = make_float2(ex2(x.x), ex2(x.y));
            ls[e & 1] = fadd2(ls[e & 1], p);
            w[e] = pack_bf16x2(p.x, p.y);
          }
          tmem_st16u(tS + b * T + h * 16, w);  // (over scores that have been read)
        }
        l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar_p_full[b]);
      }
      if (!ok) break;
      // the next segment's Q rows (every QK of this segment has completed: its last S was read above)
      cur.next_segment(sTab, a, G);
      if (cur.live) write_q(cur.s);
      if (active) {
        // the row sum over both halves (double-buffered by the parity of the quarter's meetings)
        float* sum = sSum + (sums & 1) * 2 * kM;
        sum[hf * kM + r] = l;
        if (!pair_meet(&bar_sum[quarter], sums & 1)) { ok = false; break; }
        ++sums;
        const float lt = sum[r] + sum[kM + r];
        // this warp's half of O, once the segment's last PV has completed: normalised into the output when the
        // segment is the whole block, else as a partial
        if (!wait<D>(&bar_pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const bool whole = s.slot < 0;
        const float scale = whole ? (lt > 0.0f ? 1.0f / lt : 0.0f) : 1.0f;
        const int64_t orow =
            (static_cast<int64_t>(s.q0 + tok) * a.num_q_heads + s.g * G + (row - tok * G)) * D + hf * (D / 2);
        const int64_t prow = static_cast<int64_t>(max(s.slot, 0)) * kM + r;
        if (!whole && row_ok && hf == 0)
          *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(m_used, lt);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t ov[32];
          tmem_ld32(tO + c * 32, ov);
          if (row_ok) {
            float o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(ov[e]) * scale;
            if (!whole || a.out_dtype == KVQ_OUT_F32) {
              float* base = whole ? static_cast<float*>(a.out) + orow : a.part_acc + prow * D + hf * (D / 2);
              float4* dst = reinterpret_cast<float4*>(base + c * 32);
#pragma unroll
              for (int q4 = 0; q4 < 8; ++q4)
                dst[q4] = make_float4(o[4 * q4], o[4 * q4 + 1], o[4 * q4 + 2], o[4 * q4 + 3]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow + c * 32);
#pragma unroll
              for (int h8 = 0; h8 < 4; ++h8)
                dst[h8] = make_uint4(pack_bf16x2(o[8 * h8], o[8 * h8 + 1]), pack_bf16x2(o[8 * h8 + 2], o[8 * h8 + 3]),
                                     pack_bf16x2(o[8 * h8 + 4], o[8 * h8 + 5]),
                                     pack_bf16x2(o[8 * h8 + 6], o[8 * h8 + 7]));
            }
          }
        }
      } else if (!wait<D>(&bar_pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) {
        // (that PV was issued after o_free of the segment before had completed: no arrival below can be
        // counted for that one)
        ok = false;
        break;
      }
      ++items;
      tc_fence_before();  // the reads are ordered before the arrival that lets the next PV overwrite O
      __syncwarp();
      if (lane == 0) bar_arrive(bar_o_free);
    }
  }
  if (!ok) set_status(my_status, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// Joins the partials of the segments that a row's block was cut into, WPR warps per row:
// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s with M = max_s m_s.  Rows of blocks that one segment covered
// whole are final already.  A row without a visible key has l = 0 everywhere and gives zeros.
constexpr int kMergeThreads = 128;
constexpr int kMergeWarps = kMergeThreads / 32;

template <int D, int WPR>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const TreeArgs a) {
  constexpr int DPL = D / 32;  // dims per lane
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
  __shared__ float s_a[WPR > 1 ? kMergeWarps : 1][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0) {  // the call's status: any CTA's
    uint32_t st = 0;
    for (int32_t i = tid; i < a.grid; i += kMergeThreads) st = max(st, a.cta_status[i]);
    st = __reduce_max_sync(0xffffffffu, st);
    if (lane == 0) s_m[warp] = __uint_as_float(st);
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kMergeWarps; ++w) st = max(st, __float_as_uint(s_m[w]));
      *a.status = st;
    }
    __syncthreads();
  }
  const int64_t out_row = (static_cast<int64_t>(blockIdx.x) * kMergeWarps + warp) / WPR;
  const int sub = warp % WPR;
  const bool live = out_row < static_cast<int64_t>(a.total_q) * a.num_q_heads;
  const int32_t G = a.num_q_heads / a.num_kv_heads;
  const int32_t tokrow = live ? static_cast<int32_t>(out_row / a.num_q_heads) : 0;
  const int32_t head = static_cast<int32_t>(out_row - static_cast<int64_t>(tokrow) * a.num_q_heads);
  const int32_t b = live ? a.row_seq[tokrow] : -1;  // -1: no sequence covers the row
  int32_t first = 0, last = 0, u0 = 0, U = 0, C = 1, r = 0;
  if (b >= 0) {
    U = a.tab[a.batch];
    C = a.tab[a.batch + 1];
    const int32_t nt = (__ldg(a.seq_lens + b) + TCfg<D>::T - 1) / TCfg<D>::T;
    const int32_t g = head / G, row = (tokrow - __ldg(a.q_start + b)) * G + (head - g * G);
    const int32_t blk = row / kM;
    r = row - blk * kM;
    u0 = a.tab[b] + (blk * a.num_kv_heads + g) * nt;
    // the CTAs whose ranges hold the block's first and last unit: start(c) = floor(U c / C) <= u < start(c + 1)
    auto owner = [&](int32_t u) -> int32_t {
      int32_t c = min(static_cast<int32_t>((static_cast<int64_t>(u) * C + C - 1) / U), C - 1);
      while (c > 0 && range_start(U, C, c) > u) --c;
      while (c + 1 < C && range_start(U, C, c + 1) <= u) ++c;
      return c;
    };
    first = owner(u0);
    last = owner(u0 + nt - 1);
  }
  if (WPR == 1 && first == last) return;  // (the block was one segment, or there is no row)
  auto prow = [&](int32_t c) -> int64_t {  // this row's partial in CTA c: its first segment, or its last
    return static_cast<int64_t>(2 * c + (range_start(U, C, c) >= u0 ? 0 : 1)) * kM + r;
  };
  const bool split = first != last;
  float M = -INFINITY;
  if (split)
    for (int32_t c = first + lane; c <= last; c += 32) M = fmaxf(M, a.part_ml[prow(c) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[DPL], l = 0.0f;
#pragma unroll
  for (int j = 0; j < DPL; ++j) acc[j] = 0.0f;
  if (split) {
#pragma unroll 4
    for (int32_t c = first + sub; c <= last; c += WPR) {
      const int64_t p = prow(c);
      const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + p * 2);
      const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - M);
      l = fmaf(ml.y, w, l);
#pragma unroll
      for (int j = 0; j < DPL / 4; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(a.part_acc + p * D + j * 128 + lane * 4);
        acc[4 * j] = fmaf(v.x, w, acc[4 * j]);
        acc[4 * j + 1] = fmaf(v.y, w, acc[4 * j + 1]);
        acc[4 * j + 2] = fmaf(v.z, w, acc[4 * j + 2]);
        acc[4 * j + 3] = fmaf(v.w, w, acc[4 * j + 3]);
      }
    }
  }
  if constexpr (WPR > 1) {  // the row's warps are this CTA's
    static_assert(WPR == kMergeWarps, "one row per CTA");
#pragma unroll
    for (int j = 0; j < DPL / 4; ++j)
      *reinterpret_cast<float4*>(&s_a[warp][j * 128 + lane * 4]) =
          make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    if (!split || warp != 0) return;
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) l += s_l[w];
#pragma unroll
    for (int j = 0; j < DPL / 4; ++j) {
      float4 v = *reinterpret_cast<const float4*>(&s_a[0][j * 128 + lane * 4]);
#pragma unroll
      for (int w = 1; w < WPR; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&s_a[w][j * 128 + lane * 4]);
        v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
      }
      acc[4 * j] = v.x;
      acc[4 * j + 1] = v.y;
      acc[4 * j + 2] = v.z;
      acc[4 * j + 3] = v.w;
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int j = 0; j < DPL / 4; ++j) {
    const int64_t at = out_row * D + j * 128 + lane * 4;
    const float4 o = make_float4(acc[4 * j] * inv, acc[4 * j + 1] * inv, acc[4 * j + 2] * inv, acc[4 * j + 3] * inv);
    if (a.out_dtype == KVQ_OUT_F32)
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = o;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
          make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  }
}

template <int D>
kvq_status launch_tree_d(const TreeArgs& a, cudaStream_t stream) {
  using Cfg = TCfg<D>;
  decltype(&tree_tc_kernel<D, KVQ_FP8_E4M3>) kern = nullptr;
  switch (a.kind) {
    case KVQ_FP8_E4M3: kern = tree_tc_kernel<D, KVQ_FP8_E4M3>; break;
    case KVQ_Q8_0: kern = tree_tc_kernel<D, KVQ_Q8_0>; break;
    case KVQ_FP8_E4M3_UNSCALED: kern = tree_tc_kernel<D, KVQ_FP8_E4M3_UNSCALED>; break;
    case KVQ_FP8_E5M2_UNSCALED: kern = tree_tc_kernel<D, KVQ_FP8_E5M2_UNSCALED>; break;
  }
  if (kern == nullptr) return KVQ_EKIND;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) != cudaSuccess)
    return KVQ_ECUDA;
  kern<<<static_cast<unsigned>(a.grid), kThreads, Cfg::SMEM_BYTES, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return KVQ_ECUDA;
  // Few rows: a CTA for each; else a warp for each.  The whole call with a CTA / a warp: 128 rows in many segments (one
  // sequence of 64k) 42.2 / 77.4 us, 1024 86.9 / 97.3, 2048 163.7 / 166.5 (four of 64k) and 52.6 / 53.1 (eight of 8k),
  // 2560 54.0 / 53.5, 4096 302.0 / 298.2; in few segments 2048 53.7 / 53.0, 9216 103.0 / 91.3, 32768 113.3 / 73.5.
  const int64_t rows = static_cast<int64_t>(a.total_q) * a.num_q_heads;
  const bool few = rows <= 2048;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(few ? rows : (rows + kMergeWarps - 1) / kMergeWarps));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = few ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, kMergeWarps>, a)
                            : cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 1>, a);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? KVQ_OK : KVQ_ECUDA;
}

// One CTA per sequence: each of its query rows is a sequence of its own to the decode kernels, with the
// sequence's tokens and pages and the row's mask.
__global__ void tree_expand_kernel(const int32_t* __restrict__ q_start, const int32_t* __restrict__ seq_lens,
                                   int32_t total_q, int32_t mask_words, int64_t max_tokens, int32_t* __restrict__ vlens,
                                   int32_t* __restrict__ vrow, int32_t* __restrict__ vbase, uint32_t* status) {
  const int32_t b = blockIdx.x;
  const int32_t q0 = __ldg(q_start + b), q1 = __ldg(q_start + b + 1), L = __ldg(seq_lens + b);
  const int32_t n = q1 - q0;
  if (q0 < 0 || n < 0 || n > L || q1 > total_q || n > 64 * mask_words || L > max_tokens) {
    if (threadIdx.x == 0) set_status(status, kStatusBadExtend);
    return;
  }
  for (int32_t i = threadIdx.x; i < n; i += blockDim.x) {
    vlens[q0 + i] = L;
    vrow[q0 + i] = b;
    vbase[q0 + i] = L - n;
  }
}

}  // namespace

bool tree_tc_supported(int32_t head_dim, int32_t v_dim, int32_t mla, int32_t batch) {
  return !mla && v_dim == head_dim && (head_dim == 128 || head_dim == 256) && batch <= kMaxTreeBatch;
}

kvq_status launch_tree_expand(const int32_t* q_start, const int32_t* seq_lens, int32_t batch, int32_t total_q,
                              int32_t mask_words, int64_t max_tokens, int32_t* vlens, int32_t* vrow, int32_t* vbase,
                              uint32_t* status, cudaStream_t stream) {
  tree_expand_kernel<<<static_cast<unsigned>(batch), 64, 0, stream>>>(q_start, seq_lens, total_q, mask_words, max_tokens,
                                                                       vlens, vrow, vbase, status);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

kvq_status launch_tree_tc(const TreeArgs& a, cudaStream_t stream) {
  if (a.head_dim == 128) return launch_tree_d<128>(a, stream);
  if (a.head_dim == 256) return launch_tree_d<256>(a, stream);
  return KVQ_EUNSUPPORTED;
}

}  // namespace kvq
