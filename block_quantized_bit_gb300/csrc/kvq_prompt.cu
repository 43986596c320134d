// kvq_prompt.cu -- causal attention over whole prompts, packed one behind the other, grouped heads, bf16, on the
// tcgen05 tensor cores:
//   out[i][h] = sum_{t <= i} softmax_t(sm_scale q[i][h].k[t][g]) v[t][g],  g = h / G, within each sequence.
// 4 D FLOPs per (row, visible key) against 2 D bytes per row: bound by the tensor pipe once prompts pass some
// hundred tokens, and by the softmax's exponentials, one per (row, key), close behind.
//
// A tile is 128 tokens of one query head, the MMA's M.  head_dim 64 and 128: a CTA works on two tiles A and B of the
// same kv head, so that one's softmax runs under the other's MMAs:
//   S[128 rows][128 keys] = Q . K^T   (Q, K in shared memory, K-major)
//   O[128 rows][D]       += P . V     (P as bf16 in tensor memory over the columns of S; V in shared memory, MN-major)
// Tensor memory: S_A, S_B, O_A, O_B of 128 columns each.  P replaces the S it was made from.  MMAs of different
// accumulators are not ordered among themselves, so QK of the next key tile, which overwrites P, waits for the
// PV that reads it.  The MMA warp's order, QK_A(j), PV_B(j-1), QK_B(j), PV_A(j), leaves a softmax the time of two
// MMA groups.  Tiles of a kv head are paired in (token block, head) order: with an even number of heads per kv head
// both tiles see the same keys.
//
// Warps 0-3 and 4-7: softmax of A and of B, one thread per row; the row's 128 scores stay in registers from the
// one tensor-memory load to P.  Lazy rescaling as in the extend kernel (the running max moves only when a score
// passes it by more than 2^8).  P is handed over in two halves of 64 keys.
// Warp 8 issues all MMAs.  Warp 9 takes items off a global counter, the longest first, and loads Q, K and V
// tiles with TMA (128-byte swizzle) through a ring of slots.
// Only a tile's last key tile is masked: token blocks and key tiles both start at the sequence's start, so its
// rule is key <= row.  Keys behind the sequence's end are never visible, but their V rows belong to whatever follows
// and may be anything, so the MMA warp clears those rows in shared memory (0 * NaN would be NaN).
// Every wait is bounded (2 s) and reports a timeout in the status word instead of hanging.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_flash.cuh"
#include "kvq_internal.h"
#include "kvq_tc.cuh"

namespace kvq {
namespace {

constexpr int kM = 128;                // rows of a tile, and keys of a key tile
constexpr int kSmWarps = 8;            // softmax: warps 0-3 of tile A, 4-7 of tile B
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;
constexpr int kThreads = 10 * 32;
constexpr int kTmemCols = 512;
constexpr float kLazyRescale = 8.0f;   // log2 headroom before the running max must move

template <int D>
struct PCfg {
  static constexpr int CH = D / 64;              // 128-byte column chunks of a row
  static constexpr int CHUNK = kM * 128;         // bytes of one chunk of a tile
  static constexpr int TILE = CH * CHUNK;        // bytes of a Q, K or V tile
  static constexpr int SLOTS = D == 128 ? 4 : 6; // K and V tiles in flight
  static constexpr int Q_OFF = 0;                // 1024-byte aligned: swizzle atoms
  static constexpr int KV_OFF = Q_OFF + 2 * TILE;
  static constexpr int TAB_OFF = KV_OFF + SLOTS * TILE;                  // [batch] tile pairs of each sequence
  static constexpr int ITEM_OFF = TAB_OFF + kMaxPromptBatch * 4;         // [2] published items
  static constexpr int NBARS = 2 * SLOTS + 2 + 1 + 2 + 4 + 2 + 2 + 4;
  static constexpr int BAR_OFF = ITEM_OFF + 2 * 32;
  static constexpr int SMEM_BYTES = BAR_OFF + NBARS * 8 + 16 + 1024;     // + slack to align the base
  static constexpr int S_COL = 0, O_COL = 256;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// A published item: tiles A and B of (sequence, kv head); q0: the sequence's first row; len: its tokens; per
// tile its token block and query head; n: key tiles (0: no such tile).
struct Item {
  int32_t q0, len, g, blk[2], head[2], live;
  __device__ __forceinline__ int32_t n(int w) const { return blk[w] + 1; }  // blk = -1: no tile
};
static_assert(sizeof(Item) == 32, "item slots");

__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return smem_desc(addr, lbo, sbo) | (static_cast<uint64_t>(2) << 61);  // 128-byte swizzle
}

// One box: 64 elements (128 bytes) of `head`, rows row .. row + 127.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int head, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(row), "r"(smem_u32(bar))
      : "memory");
}

// Four MMAs (k-steps of one 64-element chunk) from a single elect.sync: A at a + k * a_step, B at b + k * b_step.
__device__ __forceinline__ void mma4_bf16(uint32_t d_tmem, uint64_t a, uint64_t a_step, uint64_t b, uint64_t b_step,
                                          uint32_t idesc, uint32_t acc_first) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "add.u64 a1, %1, %5;\n\tadd.u64 a2, a1, %5;\n\tadd.u64 a3, a2, %5;\n\t"
      "add.u64 b1, %2, %6;\n\tadd.u64 b2, b1, %6;\n\tadd.u64 b3, b2, %6;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc_first), "l"(a_step), "l"(b_step)
      : "memory");
}

// The same with A in tensor memory (a_step in columns).
__device__ __forceinline__ void mma4_bf16_tmem_a(uint32_t d_tmem, uint32_t a, uint32_t a_step, uint64_t b,
                                                 uint64_t b_step, uint32_t idesc, uint32_t acc_first) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "add.u32 a1, %1, %5;\n\tadd.u32 a2, a1, %5;\n\tadd.u32 a3, a2, %5;\n\t"
      "add.u64 b1, %2, %6;\n\tadd.u64 b2, b1, %6;\n\tadd.u64 b3, b2, %6;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d_tmem),
      "r"(a), "l"(b), "r"(idesc), "r"(acc_first), "r"(a_step), "l"(b_step)
      : "memory");
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  uint64_t A, B, C;
  memcpy(&A, &a, 8);
  memcpy(&B, &b, 8);
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(C) : "l"(A), "l"(B));
  float2 c;
  memcpy(&c, &C, 8);
  return c;
}

// Tile pairs of a sequence of len tokens: ceil(len / 128) token blocks of G heads.
__device__ __forceinline__ int32_t tile_pairs(int32_t len, int32_t G) { return ((len + kM - 1) / kM * G + 1) / 2; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap qmap,
                                                             const __grid_constant__ CUtensorMap kmap,
                                                             const __grid_constant__ CUtensorMap vmap) {
  using Cfg = PCfg<D>;
  constexpr int SLOTS = Cfg::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem + Cfg::Q_OFF;    // [2] tiles
  uint8_t* sKV = smem + Cfg::KV_OFF;  // [SLOTS]
  int32_t* sTab = reinterpret_cast<int32_t*>(smem + Cfg::TAB_OFF);
  Item* sItem = reinterpret_cast<Item*>(smem + Cfg::ITEM_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFF);
  // Every barrier completes once per use of its buffer, so a waiter names an unambiguous phase.
  uint64_t* bar_full = bars;                   // [SLOTS] K or V tile landed
  uint64_t* bar_empty = bars + SLOTS;          // [SLOTS] its last MMA completed (commit)
  uint64_t* bar_q_full = bars + 2 * SLOTS;     // [2] Q tile landed
  uint64_t* bar_q_empty = bar_q_full + 2;      // the item's last QK completed (commit)
  uint64_t* bar_s_full = bar_q_full + 3;       // [2] QK into S of tile w completed (commit)
  uint64_t* bar_p_full = bar_q_full + 5;       // [2][2] half of P of tile w written (softmax warps)
  uint64_t* bar_pv_done = bar_q_full + 9;      // [2] PV of tile w completed (commit)
  uint64_t* bar_o_free = bar_q_full + 11;      // [2] O of tile w read out (softmax warps), once per item
  uint64_t* bar_item = bar_q_full + 13;        // [2] item slot published
  uint64_t* bar_item_free = bar_q_full + 15;   // [2] item slot read by the MMA warp and every softmax warp
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + Cfg::BAR_OFF + Cfg::NBARS * 8);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t G = a.num_q_heads / a.num_kv_heads;

  for (int32_t b = tid; b < a.batch; b += kThreads) {
    const int32_t q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1);
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.total;
    if (!ok && blockIdx.x == 0) set_status(a.status, kStatusBadExtend);
    sTab[b] = ok ? tile_pairs(q1 - q0, G) : 0;
  }
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&bar_full[i], 1);
      mbar_init(&bar_empty[i], 1);
    }
    mbar_init(bar_q_empty, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_q_full[w], 1);
      mbar_init(&bar_s_full[w], 1);
      mbar_init(&bar_p_full[2 * w], kSmWarps / 2);
      mbar_init(&bar_p_full[2 * w + 1], kSmWarps / 2);
      mbar_init(&bar_pv_done[w], 1);
      mbar_init(&bar_o_free[w], kSmWarps / 2);
      mbar_init(&bar_item[w], 1);
      mbar_init(&bar_item_free[w], kSmWarps + 1);
    }
    fence_mbar_init();
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
  bool ok = true;

  // the item in slot k & 1 (k-th of this CTA), for a consumer warp
  auto take_item = [&](uint32_t k, Item& it) -> bool {
    if (!warp_wait(&bar_item[k & 1], (k >> 1) & 1)) return false;
    it = sItem[k & 1];
    __syncwarp();
    if (lane == 0) bar_arrive(&bar_item_free[k & 1]);
    return true;
  };

  if (warp == kLoadWarp) {
    // ===================================================================== items and loads
    // Items in order of falling pair number p: level p holds the pairs p of all sequences that have one, times the
    // kv heads.  above(p) = items of levels > p.
    auto above = [&](int32_t p) -> int64_t {
      int32_t s = 0;
      for (int32_t b = lane; b < a.batch; b += 32) s += max(sTab[b] - p - 1, 0);
      return static_cast<int64_t>(__reduce_add_sync(0xffffffffu, s)) * a.num_kv_heads;
    };
    int32_t top = 0;  // pairs of the longest sequence
    for (int32_t b = lane; b < a.batch; b += 32) top = max(top, sTab[b]);
    top = __reduce_max_sync(0xffffffffu, top);
    const int64_t n_items = above(-1);
    uint32_t k = 0, kv = 0;  // items published; K/V tiles loaded
    int64_t idx = blockIdx.x;
    uint32_t nq[2] = {0, 0};
    while (ok) {
      Item it;
      it.live = idx < n_items;
      if (it.live) {
        int32_t lo = 0, hi = top - 1;  // smallest p with above(p) <= idx
        while (lo < hi) {
          const int32_t mid = (lo + hi) >> 1;
          if (above(mid) <= idx) hi = mid;
          else lo = mid + 1;
        }
        const int32_t p = lo, q = static_cast<int32_t>(idx - above(p));
        int32_t rank = q / a.num_kv_heads, b = 0;
        it.g = q - rank * a.num_kv_heads;
        for (int32_t b0 = 0; b0 < a.batch; b0 += 32) {  // the rank-th sequence with more than p pairs
          const uint32_t m = __ballot_sync(0xffffffffu, b0 + lane < a.batch && sTab[b0 + lane] > p);
          const int32_t c = __popc(m);
          if (rank < c) {
            b = b0 + __fns(m, 0, rank + 1);
            break;
          }
          rank -= c;
        }
        it.q0 = __ldg(a.q_start + b);
        it.len = __ldg(a.q_start + b + 1) - it.q0;
        const int32_t tiles = (it.len + kM - 1) / kM * G;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int32_t t = 2 * p + w;
          it.blk[w] = t < tiles ? t / G : -1;
          it.head[w] = it.g * G + t % G;
        }
      }
      if (k >= 2 && !warp_wait(&bar_item_free[k & 1], ((k >> 1) - 1) & 1)) { ok = false; break; }
      if (lane == 0) {
        sItem[k & 1] = it;
        bar_arrive(&bar_item[k & 1]);
      }
      __syncwarp();
      if (!it.live) break;
      uint32_t next = 0;
      if (lane == 0) next = atomicAdd(a.counter, 1u);
      // Q tiles, once the previous item's QKs have read theirs
      if (k >= 1 && !warp_wait(bar_q_empty, (k - 1) & 1)) { ok = false; break; }
      if (lane == 0) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (it.blk[w] >= 0) {
            mbar_arrive_expect_tx(&bar_q_full[w], Cfg::TILE);
#pragma unroll
            for (int c = 0; c < Cfg::CH; ++c)
              tma_rows(smem_u32(sQ + w * Cfg::TILE + c * Cfg::CHUNK), &qmap, c * 64, it.head[w], it.q0 + it.blk[w] * kM,
                       &bar_q_full[w]);
          }
      }
      __syncwarp();
#pragma unroll
      for (int w = 0; w < 2; ++w) nq[w] += it.blk[w] >= 0;
      const int32_t n = max(it.blk[0], it.blk[1]) + 1;
      for (int32_t i = 0; i < 2 * n && ok; ++i, ++kv) {  // K of key tile i / 2, then its V
        const int s = kv % SLOTS;
        if (kv >= SLOTS && !warp_wait(&bar_empty[s], (kv / SLOTS - 1) & 1)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_full[s], Cfg::TILE);
#pragma unroll
          for (int c = 0; c < Cfg::CH; ++c)
            tma_rows(smem_u32(sKV + s * Cfg::TILE + c * Cfg::CHUNK), (i & 1) ? &vmap : &kmap, c * 64, it.g,
                     it.q0 + (i >> 1) * kM, &bar_full[s]);
        }
        __syncwarp();
      }
      ++k;
      idx = static_cast<int64_t>(__shfl_sync(0xffffffffu, next, 0)) + gridDim.x;
    }
    // no copy may still be in flight when the CTA exits
    for (uint32_t j = 1; j <= kv && j <= static_cast<uint32_t>(SLOTS); ++j)
      (void)mbar_wait_bounded(&bar_full[(kv - j) % SLOTS], ((kv - j) / SLOTS) & 1);
    for (int w = 0; w < 2; ++w)
      if (nq[w] > 0) (void)mbar_wait_bounded(&bar_q_full[w], (nq[w] - 1) & 1);
  } else if (warp == kMmaWarp) {
    // ===================================================================== MMA issue (elected lane)
    const uint32_t idesc_qk = x_idesc(kM, false);
    const uint32_t idesc_pv = x_idesc(D, true);
    uint32_t kv = 0;                                    // K/V tiles of finished items
    uint32_t nqt[2] = {0, 0}, nt[2] = {0, 0}, ni[2] = {0, 0};  // per tile w: Q tiles; PVs issued; items
    Item it;
    auto qk = [&](int w, uint32_t slot) -> bool {
      // P of the tile's last PV lies in the columns that this QK writes
      if (nt[w] > 0 && !warp_wait(&bar_pv_done[w], (nt[w] - 1) & 1)) return false;
      tc_fence_after();
      const uint64_t dq = sw128_desc(smem_u32(sQ + w * Cfg::TILE), 16, 1024);
      const uint64_t dk = sw128_desc(smem_u32(sKV + slot * Cfg::TILE), 16, 1024);
#pragma unroll
      for (int c = 0; c < Cfg::CH; ++c)  // a k-step is 32 bytes of the swizzled 128-byte rows
        mma4_bf16(tmem + Cfg::S_COL + w * kM, dq + static_cast<uint64_t>((c * Cfg::CHUNK) >> 4), 2,
                  dk + static_cast<uint64_t>((c * Cfg::CHUNK) >> 4), 2, idesc_qk, c > 0 ? 1u : 0u);
      mma_commit(&bar_s_full[w]);
      __syncwarp();
      return true;
    };
    auto pv = [&](int w, uint32_t slot, bool first) -> bool {
      if (first && ni[w] > 1 && !warp_wait(&bar_o_free[w], (ni[w] - 2) & 1)) return false;
      const uint64_t dv = sw128_desc(smem_u32(sKV + slot * Cfg::TILE), Cfg::CHUNK, 1024);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!warp_wait(&bar_p_full[2 * w + h], nt[w] & 1)) return false;
        tc_fence_after();
        mma4_bf16_tmem_a(tmem + Cfg::O_COL + w * kM, tmem + Cfg::S_COL + w * kM + h * 32, 8u,
                         dv + static_cast<uint64_t>((h * 64 * 128) >> 4), static_cast<uint64_t>((16 * 128) >> 4), idesc_pv,
                         (!first || h > 0) ? 1u : 0u);
      }
      mma_commit(&bar_pv_done[w]);
      __syncwarp();
      ++nt[w];
      return true;
    };
    for (uint32_t k = 0; ok; ++k) {
      if (!take_item(k, it)) { ok = false; break; }
      if (!it.live) break;
      const int32_t nA = it.n(0), nB = it.n(1), n = max(nA, nB);
      ni[0] += nA > 0;
      ni[1] += nB > 0;
      auto slot_of = [&](int32_t j, int v) -> uint32_t { return (kv + 2 * j + v) % SLOTS; };
      auto landed = [&](int32_t j, int v) -> bool {
        const uint32_t u = kv + 2 * j + v;
        return warp_wait(&bar_full[u % SLOTS], (u / SLOTS) & 1);
      };
      // the V rows of keys behind the sequence's end
      auto clear_tail = [&](int32_t j) {
        const int32_t from = it.len - j * kM;
        if (from >= kM) return;
        uint8_t* v = sKV + slot_of(j, 1) * Cfg::TILE;
#pragma unroll
        for (int c = 0; c < Cfg::CH; ++c)
          for (int32_t o = from * 128 + lane * 16; o < Cfg::CHUNK; o += 512)
            *reinterpret_cast<uint4*>(v + c * Cfg::CHUNK + o) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
      };
      int32_t v_ready = 0;  // V tiles that have landed (and whose tail is clear)
      auto need_v = [&](int32_t j) -> bool {
        if (v_ready > j) return true;
        if (!landed(j, 1)) return false;
        clear_tail(j);
        v_ready = j + 1;
        return true;
      };
      for (int32_t j = 0; j <= n; ++j) {
        if (j < n && !landed(j, 0)) { ok = false; break; }
        if (j < nA) {
          if (j == 0 && !warp_wait(&bar_q_full[0], nqt[0]++ & 1)) { ok = false; break; }
          if (!qk(0, slot_of(j, 0))) { ok = false; break; }
        }
        if (j >= 1) {
          if (j - 1 < nB && (!need_v(j - 1) || !pv(1, slot_of(j - 1, 1), j == 1))) { ok = false; break; }
          mma_commit(&bar_empty[slot_of(j - 1, 1)]);
        }
        if (j < nB) {
          if (j == 0 && !warp_wait(&bar_q_full[1], nqt[1]++ & 1)) { ok = false; break; }
          if (!qk(1, slot_of(j, 0))) { ok = false; break; }
        }
        if (j < n) {
          mma_commit(&bar_empty[slot_of(j, 0)]);
          if (j == n - 1) mma_commit(bar_q_empty);
        }
        if (j < nA && (!need_v(j) || !pv(0, slot_of(j, 1), j == 0))) { ok = false; break; }
      }
      kv += 2 * n;
    }
    // before tensor memory is freed, every MMA issued must have completed
    for (int w = 0; w < 2; ++w)
      if (nt[w] > 0) (void)mbar_wait_bounded(&bar_pv_done[w], (nt[w] - 1) & 1);
  } else {
    // ===================================================================== softmax warps
    const int w = warp >> 2;                   // tile
    const int r = tid & (kM - 1);              // row = tensor-memory lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + Cfg::S_COL + w * kM + lane_base;
    const uint32_t tO = tmem + Cfg::O_COL + w * kM + lane_base;
    uint32_t nt = 0;  // key tiles processed
    Item it;
    for (uint32_t k = 0; ok; ++k) {
      if (!take_item(k, it)) { ok = false; break; }
      if (!it.live) break;
      const int32_t n = it.n(w);
      if (n == 0) continue;
      float m = -INFINITY;
      float2 l2 = make_float2(0.0f, 0.0f);
      for (int32_t j = 0; j < n; ++j, ++nt) {
        if (!warp_wait(&bar_s_full[w], nt & 1)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[kM];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_issue(tS + 32 * c, s + 32 * c);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_wait_ld32(s + 32 * c);
        if (j == n - 1) {
#pragma unroll
          for (int e = 0; e < kM; ++e) s[e] = e <= r ? s[e] : 0xFF800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kM; e += 2)
          mx[(e >> 1) & 3] = fmaxf(mx[(e >> 1) & 3], fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 1])));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.score_scale;
        float alpha = 1.0f;
        if (top > m + kLazyRescale) {  // (also from the first tile's -inf)
          alpha = j > 0 ? ex2(m - top) : 1.0f;
          m = top;
        }
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
          // O holds the PV of the tile before: QK of this tile was issued after it had completed
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + c * 32, o);
          }
          l2.x *= alpha;
          l2.y *= alpha;
        }
        const float2 sc2 = make_float2(a.score_scale, a.score_scale), m2 = make_float2(-m, -m);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pw[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int i = h * 64 + 2 * e;
            const float2 x = ffma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), sc2, m2);
            const float2 p = make_float2(ex2(x.x), ex2(x.y));
            l2 = fadd2(l2, p);
            pw[e] = pack_bf16x2(p.x, p.y);
          }
          tmem_st32(tS + h * 32, pw);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&bar_p_full[2 * w + h]);
        }
      }
      if (!ok) break;
      // O / l of this row, once the item's last PV has completed
      if (!warp_wait(&bar_pv_done[w], (nt - 1) & 1)) { ok = false; break; }
      tc_fence_after();
      const float inv = 1.0f / (l2.x + l2.y);
      const int32_t tok = it.blk[w] * kM + r;
      const int64_t orow = static_cast<int64_t>(it.q0 + tok) * a.out_token + static_cast<int64_t>(it.head[w]) * a.out_head;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(tO + c * 32, ov);
        if (tok < it.len) {
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(ov[e]) * inv;
          if (a.out_dtype == KVQ_OUT_F32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow + c * 32);
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4) dst[q4] = make_float4(o[4 * q4], o[4 * q4 + 1], o[4 * q4 + 2], o[4 * q4 + 3]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow + c * 32);
#pragma unroll
            for (int h8 = 0; h8 < 4; ++h8)
              dst[h8] = make_uint4(pack_bf16x2(o[8 * h8], o[8 * h8 + 1]), pack_bf16x2(o[8 * h8 + 2], o[8 * h8 + 3]),
                                   pack_bf16x2(o[8 * h8 + 4], o[8 * h8 + 5]), pack_bf16x2(o[8 * h8 + 6], o[8 * h8 + 7]));
          }
        }
      }
      tc_fence_before();  // the reads are ordered before the arrival that lets the next PV overwrite O
      __syncwarp();
      if (lane == 0) bar_arrive(&bar_o_free[w]);
    }
  }
  if (!ok) set_status(a.status, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// (element, head, token) view of a bf16 tensor [total][heads][D] with the given strides in elements; a box is 64
// elements of 128 tokens of one head.
bool encode_rows(CUtensorMap* map, const void* x, int64_t total, int32_t heads, int D, int64_t token, int64_t head) {
  const EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(total)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(token) * 2};
  const cuuint32_t box[3] = {64, 1, kM};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
kvq_status launch_prompt_d(const PromptArgs& a, cudaStream_t stream) {
  using Cfg = PCfg<D>;
  auto kern = prompt_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) != cudaSuccess)
    return KVQ_ECUDA;
  CUtensorMap qm, km, vm;
  if (!encode_rows(&qm, a.q, a.total, a.num_q_heads, D, a.q_token, a.q_head) ||
      !encode_rows(&km, a.k, a.total, a.num_kv_heads, D, a.k_token, a.k_head) ||
      !encode_rows(&vm, a.v, a.total, a.num_kv_heads, D, a.v_token, a.v_head))
    return KVQ_ECUDA;
  const int64_t G = a.num_q_heads / a.num_kv_heads;
  const int64_t blocks = static_cast<int64_t>(a.total) / kM + std::min<int64_t>(a.batch, a.total);  // at most
  const int64_t bound = (blocks * G / 2 + a.batch) * a.num_kv_heads;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(bound, a.sms));
  kern<<<static_cast<unsigned>(grid), kThreads, Cfg::SMEM_BYTES, stream>>>(a, qm, km, vm);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

}  // namespace

bool prompt_supported(int32_t head_dim, int32_t batch) {
  return (head_dim == 64 || head_dim == 128) && batch <= kMaxPromptBatch;
}

kvq_status launch_prompt(const PromptArgs& a, cudaStream_t stream) {
  if (a.head_dim == 64) return launch_prompt_d<64>(a, stream);
  if (a.head_dim == 128) return launch_prompt_d<128>(a, stream);
  return KVQ_EUNSUPPORTED;
}

}  // namespace kvq
