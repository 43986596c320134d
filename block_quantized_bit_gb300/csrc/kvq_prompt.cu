// kvq_prompt.cu -- causal attention over whole prompts, packed one behind the other, grouped heads, bf16, on the tcgen05
// tensor cores (head_dim 64 and 128; 256: kvq_prompt_wide.cu):
//   out[i][h] = sum_{t <= i} softmax_t(sm_scale q[i][h].k[t][g]) v[t][g],  g = h / G, within each sequence.
// 4 D FLOPs per (row, visible key) against 2 D bytes per row: bound by the tensor pipe once prompts pass some
// hundred tokens, and by the softmax's exponentials, one per (row, key), close behind.
//
// A tile is 128 tokens of one query head, the MMA's M.  A CTA works on two tiles A and B of the same kv head, so
// that one's softmax runs under the other's MMAs:
//   S[128 rows][128 keys] = Q . K^T   (Q, K in shared memory, K-major)
//   O[128 rows][D]       += P . V     (P as bf16 in tensor memory over the columns of S; V in shared memory, MN-major)
// Tensor memory: S_A, S_B, O_A, O_B of 128 columns each.  P replaces the S it was made from.  MMAs of different
// accumulators are not ordered among themselves, so QK of the next key tile, which overwrites P, waits for the
// PV that reads it.  The MMA warp's order, QK_A(j), PV_B(j-1), QK_B(j), PV_A(j), leaves a softmax the time of two
// MMA groups.  Tiles of a kv head are paired in (token block, head) order: with an even number of heads per kv head
// both tiles see the same keys.
//
// Warps 0-3 and 4-7: softmax of A and of B, one thread per row; the row's 128 scores stay in registers from the
// one tensor-memory load, which also returns their maxima, to P.  Lazy rescaling as in the extend kernel (the running max
// moves only when a score passes it by more than 2^8).  O is read into registers at once, so that the next item's first PV
// may overwrite it, and leaves through shared memory.
// Warp 8 issues all MMAs.  Warp 9 takes items off a global counter, the longest first, and loads Q, K and V
// tiles with TMA (128-byte swizzle), K and V of a key tile as one stage.
// Only a tile's last key tile is masked: token blocks and key tiles both start at the sequence's start, so its
// rule is key <= row, and a warp's 32 rows meet the diagonal in one 32-key chunk.  Keys behind the sequence's end are never
// visible, but their V rows belong to whatever follows and may be anything, so the MMA warp clears those rows in
// shared memory (0 * NaN would be NaN).
// Every wait is bounded (2 s) and reports a timeout in the status word instead of hanging.
//
// Measured, 32 heads of 128 over 8, one prompt of 16384 tokens: 1280 us = 1718 TFLOP/s, 91% of the measured GEMM burst
// rate (long runs back to back, under the board's power cap: 1390 us); 8192 tokens 336 us; 16 heads over 8, eight
// prompts of 150 to 2048 tokens: 40.5 us in a graph, of which the longest item's chain of key tiles is 25.  32 heads of 64
// over 8, 8192 tokens: 263 us = 1045 TFLOP/s, eight prompts of 150 to 2048 tokens 54.5 us: half the products for the
// same softmax, so a tile's own chain (2340 clocks a key tile, see the trace) paces it.  What bounds head_dim 128: the MMA
// warp's path (four MMA groups and five waits per pair of key tiles), then the board's power.  A trace of one CTA's
// key tile: QK to S visible 500 clocks, softmax 1400, P to PV issued 350. What the steps were worth, 16384 tokens: one
// stage and one wait for K and V, eight MMAs per elect 1720 -> 1430; maxima with the tensor-memory load, waits'
// unlikely parts out of line 1400; output through shared memory, the diagonal's masks on 32 keys 1366; the MMA loop
// without the branches of its first and last step 1280. Measured slower, and not kept: P handed over in halves, P
// formed against the old maximum with the row's maximum beside it, two threads per row, polling waits, the scores read
// twice from tensor memory in rolled loops; (against 1370) the next item's first QK before this item's last PV 1410, a
// warp of its own for Q 1395; (against 1280) a softmax loop of its own for the diagonal 1293, commits of the key stage
// behind the second QK 1557.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_flash.cuh"
#include "kvq_internal.h"
#include "kvq_prompt.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace {

constexpr int kSmWarps = 8;            // softmax: warps 0-3 of tile A, 4-7 of tile B
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;
constexpr int kThreads = 10 * 32;

template <int D>
struct PCfg {
  static constexpr int CH = D / 64;              // 128-byte column chunks of a row
  static constexpr int CHUNK = kM * 128;         // bytes of one chunk of a tile
  static constexpr int TILE = CH * CHUNK;        // bytes of a Q, K or V tile
  static constexpr int STAGES = D == 128 ? 2 : 4; // key tiles (K and V) in flight
  static constexpr int Q_OFF = 0;                // 1024-byte aligned: swizzle atoms
  static constexpr int KV_OFF = Q_OFF + 2 * TILE;
  static constexpr int TAB_OFF = KV_OFF + STAGES * 2 * TILE;             // [batch] tile pairs of each sequence
  static constexpr int ITEM_OFF = TAB_OFF + kMaxPromptBatch * 4;         // [2] published items
  static constexpr int NBARS = 2 * STAGES + 15;
  static constexpr int BAR_OFF = ITEM_OFF + 2 * 32;
  static constexpr int STG_OFF = BAR_OFF + (NBARS * 8 + 16 + 15) / 16 * 16;  // [8 softmax warps] 2 KB of output
  static constexpr int SMEM_BYTES = STG_OFF + kSmWarps * 2048 + 1024;    // + slack to align the base
  static constexpr int S_COL = 0, O_COL = 256;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// S = Q . K^T over CH chunks of 64 elements, both operands K-major with the 128-byte swizzle, from one elect.sync: a
// k-step is 32 bytes (2 descriptor units) along a chunk's rows, and chunks are 16 KB (1024 units) apart.
template <int CH>
__device__ __forceinline__ void mma_chunks(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
  if constexpr (CH == 1) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc)
        : "memory");
  } else {
    static_assert(CH == 2, "one or two chunks");
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\tadd.u64 a4, %1, 1024;\n\t"
        "add.u64 a5, %1, 1026;\n\tadd.u64 a6, %1, 1028;\n\tadd.u64 a7, %1, 1030;\n\t"
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\tadd.u64 b4, %2, 1024;\n\t"
        "add.u64 b5, %2, 1026;\n\tadd.u64 b6, %2, 1028;\n\tadd.u64 b7, %2, 1030;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, 1;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc)
        : "memory");
  }
}

// A value that the compiler takes for a new one at each use: branches on it stay apart (merged, they would index the row's
// scores by it, in local memory).
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap qmap,
                                                             const __grid_constant__ CUtensorMap kmap,
                                                             const __grid_constant__ CUtensorMap vmap) {
  using Cfg = PCfg<D>;
  constexpr int STAGES = Cfg::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem + Cfg::Q_OFF;    // [2] tiles
  uint8_t* sKV = smem + Cfg::KV_OFF;  // [STAGES][K, V]
  int32_t* sTab = reinterpret_cast<int32_t*>(smem + Cfg::TAB_OFF);
  Item* sItem = reinterpret_cast<Item*>(smem + Cfg::ITEM_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFF);
  // Every barrier completes once per use of its buffer, so a waiter names an unambiguous phase.
  uint64_t* bar_full = bars;                   // [STAGES] K and V tile landed
  uint64_t* bar_empty = bars + STAGES;         // [STAGES] their last MMA completed (commit)
  uint64_t* bar_q_full = bars + 2 * STAGES;    // [2] Q tile landed
  uint64_t* bar_q_empty = bar_q_full + 2;      // the item's last QK completed (commit)
  uint64_t* bar_s_full = bar_q_full + 3;       // [2] QK into S of tile w completed (commit)
  uint64_t* bar_p_full = bar_q_full + 5;       // [2] P of tile w written (softmax warps)
  uint64_t* bar_pv_done = bar_q_full + 7;      // [2] PV of tile w completed (commit)
  uint64_t* bar_o_free = bar_q_full + 9;       // [2] O of tile w read out (softmax warps), once per item
  uint64_t* bar_item = bar_q_full + 11;        // [2] item slot published
  uint64_t* bar_item_free = bar_q_full + 13;   // [2] item slot read by the MMA warp and every softmax warp
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + Cfg::BAR_OFF + Cfg::NBARS * 8);

  uint8_t* sStage = smem + Cfg::STG_OFF;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == kLoadWarp * 32) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  prompt_table<2>(a, sTab);
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&bar_full[i], 1);
      mbar_init(&bar_empty[i], 1);
    }
    mbar_init(bar_q_empty, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_q_full[w], 1);
      mbar_init(&bar_s_full[w], 1);
      mbar_init(&bar_p_full[w], kSmWarps / 2);
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
    if (!warp_wait_far(&bar_item[k & 1], (k >> 1) & 1)) return false;
    it = sItem[k & 1];
    __syncwarp();
    if (lane == 0) bar_arrive(&bar_item_free[k & 1]);
    return true;
  };

  if (warp == kLoadWarp) {
    // ===================================================================== items and loads
    const ItemSource<2> source(a, sTab);
    uint32_t k = 0, kv = 0;  // items published; key tiles loaded
    int64_t idx = blockIdx.x;
    uint32_t nq[2] = {0, 0};
    while (ok) {
      const Item it = source.get(idx);
      if (k >= 2 && !warp_wait_far(&bar_item_free[k & 1], ((k >> 1) - 1) & 1)) { ok = false; break; }
      if (lane == 0) {
        sItem[k & 1] = it;
        bar_arrive(&bar_item[k & 1]);
      }
      __syncwarp();
      if (k == 0) wait_cleared();
      if (!it.live) break;
      // Q tiles, once the previous item's QKs have read theirs
      if (k >= 1 && !warp_wait_far(bar_q_empty, (k - 1) & 1)) { ok = false; break; }
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
      uint32_t next = 0;
      if (lane == 0) next = atomicAdd(a.counter, 1u);
#pragma unroll
      for (int w = 0; w < 2; ++w) nq[w] += it.blk[w] >= 0;
      const int32_t n = max(it.blk[0], it.blk[1]) + 1;
      for (int32_t j = 0; j < n; ++j, ++kv) {
        const int s = kv % STAGES;
        if (kv >= STAGES && !warp_wait_far(&bar_empty[s], (kv / STAGES - 1) & 1)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_full[s], 2 * Cfg::TILE);
          uint8_t* dst = sKV + s * 2 * Cfg::TILE;
#pragma unroll
          for (int c = 0; c < Cfg::CH; ++c)
            tma_rows(smem_u32(dst + c * Cfg::CHUNK), &kmap, c * 64, it.g, it.q0 + j * kM, &bar_full[s]);
#pragma unroll
          for (int c = 0; c < Cfg::CH; ++c)
            tma_rows(smem_u32(dst + Cfg::TILE + c * Cfg::CHUNK), &vmap, c * 64, it.g, it.q0 + j * kM, &bar_full[s]);
        }
        __syncwarp();
      }
      ++k;
      idx = static_cast<int64_t>(__shfl_sync(0xffffffffu, next, 0)) + gridDim.x;
    }
    // no copy may still be in flight when the CTA exits
    for (uint32_t j = 1; j <= kv && j <= static_cast<uint32_t>(STAGES); ++j)
      (void)mbar_wait_bounded(&bar_full[(kv - j) % STAGES], ((kv - j) / STAGES) & 1);
    for (int w = 0; w < 2; ++w)
      if (nq[w] > 0) (void)mbar_wait_bounded(&bar_q_full[w], (nq[w] - 1) & 1);
  } else if (warp == kMmaWarp) {
    // ===================================================================== MMA issue (elected lane)
    const uint32_t idesc_qk = x_idesc(kM, false);
    const uint32_t idesc_pv = x_idesc(D, true);
    const uint64_t dq = sw128_desc(smem_u32(sQ), 16, 1024);
    const uint64_t dk0 = sw128_desc(smem_u32(sKV), 16, 1024);
    const uint64_t dv0 = sw128_desc(smem_u32(sKV + Cfg::TILE), Cfg::CHUNK, 1024);
    constexpr uint64_t kStageStep = (2 * Cfg::TILE) >> 4;
    uint32_t kv = 0;                           // key tiles of finished items
    uint32_t nt[2] = {0, 0}, ni[2] = {0, 0};   // per tile w: PVs issued; items
    Item it;
    auto qk = [&](int w, uint32_t stage) -> bool {
      // P of the tile's last PV lies in the columns that this QK writes
      if (nt[w] > 0 && !warp_wait_far(&bar_pv_done[w], (nt[w] - 1) & 1)) return false;
      tc_fence_after();
      mma_chunks<Cfg::CH>(tmem + Cfg::S_COL + w * kM, dq + ((w * Cfg::TILE) >> 4), dk0 + stage * kStageStep, idesc_qk);
      mma_commit(&bar_s_full[w]);
      return true;
    };
    auto pv = [&](int w, uint32_t stage, bool first) -> bool {
      if (first && ni[w] > 1 && !warp_wait_far(&bar_o_free[w], (ni[w] - 2) & 1)) return false;
      if (!warp_wait_far(&bar_p_full[w], nt[w] & 1)) return false;
      tc_fence_after();
      // a k-step is 16 keys: 8 columns of P, 16 rows of V
      mma8_bf16_tmem_a(tmem + Cfg::O_COL + w * kM, tmem + Cfg::S_COL + w * kM, 8u, dv0 + stage * kStageStep,
                       static_cast<uint64_t>((16 * 128) >> 4), idesc_pv, first ? 0u : 1u);
      mma_commit(&bar_pv_done[w]);
      ++nt[w];
      return true;
    };
    for (uint32_t k = 0; ok; ++k) {
      if (!take_item(k, it)) { ok = false; break; }
      if (!it.live) break;
      const int32_t nA = it.blk[0] + 1, nB = it.blk[1] + 1, n = max(nA, nB);
      if (nA > 0 && !warp_wait_far(&bar_q_full[0], ni[0]++ & 1)) { ok = false; break; }
      if (nB > 0 && !warp_wait_far(&bar_q_full[1], ni[1]++ & 1)) { ok = false; break; }
      auto clear = [&](int32_t j, uint32_t stage) {  // before the first PV that reads the tile
        if (it.len - j * kM < kM)
          clear_rows<Cfg::CH, kM>(sKV + stage * 2 * Cfg::TILE + Cfg::TILE, it.len - j * kM);
      };
      if (nA == nB) {  // (the usual item: its loop has no more branches than it needs)
        uint32_t stage = kv % STAGES;
        if (!warp_wait_far(&bar_full[stage], (kv / STAGES) & 1) || !qk(0, stage) || !qk(1, stage)) { ok = false; break; }
        if (n == 1) mma_commit(bar_q_empty);
        clear(0, stage);
        if (!pv(0, stage, true)) { ok = false; break; }
        for (int32_t j = 1; j < n; ++j) {
          const uint32_t before = stage;
          stage = ++kv % STAGES;
          if (!warp_wait_far(&bar_full[stage], (kv / STAGES) & 1) || !qk(0, stage) || !pv(1, before, j == 1)) {
            ok = false;
            break;
          }
          mma_commit(&bar_empty[before]);
          if (!qk(1, stage)) { ok = false; break; }
          if (j == n - 1) {
            mma_commit(bar_q_empty);
            clear(j, stage);
          }
          if (!pv(0, stage, false)) { ok = false; break; }
        }
        if (!ok || !pv(1, stage, n == 1)) { ok = false; break; }
        mma_commit(&bar_empty[stage]);
        ++kv;
        continue;
      }
      uint32_t stage = 0, before = 0;
      for (int32_t j = 0; j <= n; ++j) {
        before = stage;
        if (j < n) {
          stage = kv % STAGES;
          if (!warp_wait_far(&bar_full[stage], (kv / STAGES) & 1)) { ok = false; break; }
          ++kv;
          if (j < nA && !qk(0, stage)) { ok = false; break; }
        }
        if (j >= 1) {
          if (j - 1 < nB && !pv(1, before, j == 1)) { ok = false; break; }
          mma_commit(&bar_empty[before]);
        }
        if (j < n) {
          if (j < nB && !qk(1, stage)) { ok = false; break; }
          if (j == n - 1) mma_commit(bar_q_empty);
          if (it.len - j * kM < kM)  // (before the first PV that reads the tile)
            clear_rows<Cfg::CH, kM>(sKV + stage * 2 * Cfg::TILE + Cfg::TILE, it.len - j * kM);
          if (j < nA && !pv(0, stage, j == 0)) { ok = false; break; }
        }
      }
    }
    // before tensor memory is freed, every MMA issued must have completed
    for (int w = 0; w < 2; ++w)
      if (nt[w] > 0) (void)mbar_wait_bounded(&bar_pv_done[w], (nt[w] - 1) & 1);
  } else {
    // ===================================================================== softmax warps
    const int w = warp >> 2;                   // tile
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + Cfg::S_COL + w * kM + lane_base;
    const uint32_t tO = tmem + Cfg::O_COL + w * kM + lane_base;
    uint32_t nt = 0;  // key tiles processed
    Item it, next;
    ok = take_item(0, it);
    for (uint32_t k = 0; ok && it.live; ++k, it = next) {
      const int32_t blk = w == 0 ? it.blk[0] : it.blk[1], head = w == 0 ? it.head[0] : it.head[1];
      const int32_t n = blk + 1;  // key tiles; 0: no such tile
      if (n == 0) {
        ok = take_item(k + 1, next);
        continue;
      }
      float m = -INFINITY;
      float2 l2 = make_float2(0.0f, 0.0f);
      // the running max moves only when some row's passes it by more than 2^8; O and l are then rescaled (O holds
      // the PV of the tile before: QK of this tile was issued after it had completed)
      auto update_max = [&](float top, int32_t j) {
        if (j == 0) {
          m = top;
          return;
        }
        const bool moved = top > m + kLazyRescale;
        if (!__any_sync(0xffffffffu, moved)) return;
        const float alpha = moved ? ex2(m - top) : 1.0f;
        m = moved ? top : m;
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {  // (8 columns at a time: the row's scores stay in registers)
          float o[8];
          tmem_ld8(tO + c * 8, o);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] *= alpha;
          tmem_st8(tO + c * 8, o);
        }
        l2.x *= alpha;
        l2.y *= alpha;
      };
      for (int32_t j = 0; j < n; ++j, ++nt) {
        if (!warp_wait_far(&bar_s_full[w], nt & 1)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[kM];
        uint32_t mx[4];
        if (j < n - 1) {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_max_issue(tS + 32 * c, s + 32 * c, mx[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_wait_ld32(s + 32 * c);
            tmem_wait_max(mx[c]);
          }
        } else {
          // on the diagonal the warp's rows see the 32-key chunks before their own whole, their own up to the row,
          // and none behind it
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx[c] = 0xFF800000u;
            const int own = opaque(warp & 3);
            if (c < own) {
              tmem_ld32_max_issue(tS + 32 * c, s + 32 * c, mx[c]);
            } else if (c == own) {
              tmem_ld32_issue(tS + 32 * c, s + 32 * c);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) s[32 * c + e] = 0xFF800000u;
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_wait_ld32(s + 32 * c);
            tmem_wait_max(mx[c]);
            if (c == opaque(warp & 3)) {
              float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                s[32 * c + e] = e <= lane ? s[32 * c + e] : 0xFF800000u;
                x[e & 3] = fmaxf(x[e & 3], __uint_as_float(s[32 * c + e]));
              }
              mx[c] = __float_as_uint(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
            }
          }
        }
        const float top = a.score_scale * fmaxf(fmaxf(__uint_as_float(mx[0]), __uint_as_float(mx[1])),
                                                fmaxf(__uint_as_float(mx[2]), __uint_as_float(mx[3])));
        update_max(top, j);
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
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar_p_full[w]);
      }
      if (!ok || !take_item(k + 1, next)) { ok = false; break; }
      // O / l of this row, once the item's last PV has completed
      if (!warp_wait_far(&bar_pv_done[w], (nt - 1) & 1)) { ok = false; break; }
      tc_fence_after();
      const float inv = 1.0f / (l2.x + l2.y);
      const int32_t tok = blk * kM + (warp & 3) * 32;  // the warp's first row
      const int64_t orow = static_cast<int64_t>(it.q0 + tok) * a.out_token + head * a.out_head;
      auto read_out = [&] {  // the reads are ordered before the arrival that lets the next PV overwrite O
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar_o_free[w]);
      };
      if (a.out_dtype == KVQ_OUT_F32) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(tO + c * 32, ov);
          store_rows32<true>(a, sStage + warp * 2048, orow + c * 32, it.len - tok, ov, inv);
        }
        read_out();
      } else {
        uint32_t ov[D / 32][32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld32_issue(tO + c * 32, ov[c]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_wait_ld32(ov[c]);
        read_out();
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          store_rows32<false>(a, sStage + warp * 2048, orow + c * 32, it.len - tok, ov[c], inv);
      }
    }
  }
  if (!ok) prompt_report(a, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

template <int D>
kvq_status launch_prompt_d(const PromptArgs& a, cudaStream_t stream) {
  using Cfg = PCfg<D>;
  auto kern = prompt_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) != cudaSuccess)
    return KVQ_ECUDA;
  CUtensorMap qm, km, vm;
  if (!encode_rows(&qm, a.q, a.total, a.num_q_heads, D, a.q_token, a.q_head, kM) ||
      !encode_rows(&km, a.k, a.total, a.num_kv_heads, D, a.k_token, a.k_head, kM) ||
      !encode_rows(&vm, a.v, a.total, a.num_kv_heads, D, a.v_token, a.v_head, kM))
    return KVQ_ECUDA;
  const int64_t G = a.num_q_heads / a.num_kv_heads;
  const int64_t blocks = static_cast<int64_t>(a.total) / kM + std::min<int64_t>(a.batch, a.total);  // at most
  const int64_t bound = (blocks * G / 2 + a.batch) * a.num_kv_heads;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(bound, a.sms));
  return launch_cleared(kern, a, grid, kThreads, Cfg::SMEM_BYTES, qm, km, vm, stream);
}

}  // namespace

bool prompt_supported(int32_t head_dim, int32_t batch) {
  return (head_dim == 64 || head_dim == 128 || head_dim == 256) && batch <= kMaxPromptBatch;
}

kvq_status launch_prompt(const PromptArgs& a, cudaStream_t stream) {
  if (a.head_dim == 64) return launch_prompt_d<64>(a, stream);
  if (a.head_dim == 128) return launch_prompt_d<128>(a, stream);
  if (a.head_dim == 256) return launch_prompt_wide(a, stream);
  return KVQ_EUNSUPPORTED;
}

}  // namespace kvq
