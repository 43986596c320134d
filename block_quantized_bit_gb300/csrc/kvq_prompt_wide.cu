// kvq_prompt_wide.cu -- causal attention over packed prompts for head_dim 256 (the mathematics, the items and their
// order as in kvq_prompt.cu).
//
// Two tiles' outputs of 256 columns would fill tensor memory, so a CTA works on one tile of 128 rows and its overlap
// comes from two S buffers of 64 keys: QK of key tile j + 1 is issued before the softmax of tile j is waited for.
//   S[128 rows][64 keys] = Q . K^T,   O[128 rows][256] += P . V
// Tensor memory: O 256 columns, S 2 x 64, P 2 x 32 (bf16), so that no MMA overwrites what another still reads.
// Q 64 KB and four slots of 32 KB (K and V tiles in turn) of shared memory.
// Warps 0-3: softmax, one thread per row.  Warp 4 issues the MMAs, warp 5 takes items and loads tiles.
// A K/V tile pair (64 KB) serves 128 x 64 scores only, so L2 feeds each SM about 50 B per clock at the tensor pipe's
// pace; that and the N = 64 QK (whose operands' shared-memory reads take 1.5 times its MMAs) bound it.
// Measured, 8192 tokens, 16 heads of 256 over 2: 383 us = 1437 TFLOP/s, 76% of the measured GEMM burst rate (440 before
// the waits' unlikely parts moved out of line and the rows left through shared memory, 404 before the MMA loop lost its
// branches); 4 prompts of 900 to 2048 tokens 65.5 us, 8 of 150 to 2048 77.  Not kept: Q in tensor memory and P over S, which spares the QKs' reads
// of Q (371 us) but puts a copy of Q between items (69 us).
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

constexpr int kD = 256;
constexpr int kKeys = 64;              // keys of a key tile
constexpr int kSmWarps = 4;
constexpr int kMmaWarp = 4;
constexpr int kLoadWarp = 5;
constexpr int kThreads = 6 * 32;
constexpr int kChunks = kD / 64;       // 128-byte column chunks of a row
constexpr int kQChunk = kM * 128;      // bytes of one chunk of the Q tile
constexpr int kKvChunk = kKeys * 128;  // ... and of a K or V tile
constexpr int kQTile = kChunks * kQChunk;
constexpr int kKvTile = kChunks * kKvChunk;
constexpr int kSlots = 4;
constexpr int kKvOff = kQTile;                                // 1024-byte aligned: swizzle atoms
constexpr int kTabOff = kKvOff + kSlots * kKvTile;            // [batch] items per kv head of each sequence
constexpr int kItemOff = kTabOff + kMaxPromptBatch * 4;       // [2] published items
constexpr int kBarOff = kItemOff + 2 * 32;
constexpr int kBars = 2 * kSlots + 13;
constexpr int kStgOff = kBarOff + (kBars * 8 + 16 + 15) / 16 * 16;  // [4 softmax warps] 2 KB of output
constexpr int kSmem = kStgOff + kSmWarps * 2048 + 1024;       // + slack to align the base
constexpr int kOCol = 0, kSCol = 256, kPCol = 384;
static_assert(kSmem <= 227 * 1024, "shared memory");

// Four k-steps of one 64-element chunk of QK, both operands K-major with the 128-byte swizzle.
__device__ __forceinline__ void mma_chunk(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc_first) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc_first)
      : "memory");
}

// PV of one key tile: four k-steps of 16 keys, P in tensor memory (8 columns each), V MN-major (2 KB each).
__device__ __forceinline__ void mma_pv(uint32_t d_tmem, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc_first) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.u64 b1, %2, 128;\n\tadd.u64 b2, %2, 256;\n\tadd.u64 b3, %2, 384;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d_tmem),
      "r"(a), "l"(b), "r"(idesc), "r"(acc_first)
      : "memory");
}

// Key tiles that a tile sees.
__device__ __forceinline__ int32_t key_tiles(const Item& it) {
  return (min(it.len, (it.blk[0] + 1) * kM) + kKeys - 1) / kKeys;
}

__global__ void __launch_bounds__(kThreads, 1) prompt_wide_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap qmap,
                                                                  const __grid_constant__ CUtensorMap kmap,
                                                                  const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + kKvOff;  // [kSlots]
  int32_t* sTab = reinterpret_cast<int32_t*>(smem + kTabOff);
  Item* sItem = reinterpret_cast<Item*>(smem + kItemOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
  // Every barrier completes once per use of its buffer, so a waiter names an unambiguous phase.
  uint64_t* bar_full = bars;                   // [kSlots] K or V tile landed
  uint64_t* bar_empty = bars + kSlots;         // [kSlots] its MMAs completed (commit)
  uint64_t* bar_q_full = bars + 2 * kSlots;    // Q tile landed
  uint64_t* bar_q_empty = bar_q_full + 1;      // the item's last QK completed (commit)
  uint64_t* bar_s_full = bar_q_full + 2;       // [2] QK into S buffer b completed (commit)
  uint64_t* bar_p_full = bar_q_full + 4;       // [2] P buffer b written, S buffer b read (softmax warps)
  uint64_t* bar_pv_done = bar_q_full + 6;      // [2] PV that read P buffer b completed (commit)
  uint64_t* bar_o_free = bar_q_full + 8;       // O read out (softmax warps), once per item
  uint64_t* bar_item = bar_q_full + 9;         // [2] item slot published
  uint64_t* bar_item_free = bar_q_full + 11;   // [2] item slot read by the MMA warp and every softmax warp
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + kBarOff + kBars * 8);

  uint8_t* sStage = smem + kStgOff;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == kLoadWarp * 32) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  prompt_table<1>(a, sTab);
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bar_full[i], 1);
      mbar_init(&bar_empty[i], 1);
    }
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_empty, 1);
    mbar_init(bar_o_free, kSmWarps);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bar_s_full[b], 1);
      mbar_init(&bar_p_full[b], kSmWarps);
      mbar_init(&bar_pv_done[b], 1);
      mbar_init(&bar_item[b], 1);
      mbar_init(&bar_item_free[b], kSmWarps + 1);
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
    const ItemSource<1> source(a, sTab);
    uint32_t k = 0, kv = 0;  // items published; K and V tiles loaded
    int64_t idx = blockIdx.x;
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
      // the Q tile, once the previous item's QKs have read theirs
      if (k >= 1 && !warp_wait_far(bar_q_empty, (k - 1) & 1)) { ok = false; break; }
      if (lane == 0) {
        mbar_arrive_expect_tx(bar_q_full, kQTile);
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          tma_rows(smem_u32(sQ + c * kQChunk), &qmap, c * 64, it.head[0], it.q0 + it.blk[0] * kM, bar_q_full);
      }
      __syncwarp();
      uint32_t next = 0;
      if (lane == 0) next = atomicAdd(a.counter, 1u);
      ++k;
      const int32_t n = key_tiles(it);
      for (int32_t i = 0; i < 2 * n; ++i, ++kv) {  // K of key tile i / 2, then its V
        const int s = kv % kSlots;
        if (kv >= kSlots && !warp_wait_far(&bar_empty[s], (kv / kSlots - 1) & 1)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_full[s], kKvTile);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            tma_rows(smem_u32(sKV + s * kKvTile + c * kKvChunk), (i & 1) ? &vmap : &kmap, c * 64, it.g,
                     it.q0 + (i >> 1) * kKeys, &bar_full[s]);
        }
        __syncwarp();
      }
      idx = static_cast<int64_t>(__shfl_sync(0xffffffffu, next, 0)) + gridDim.x;
    }
    // no copy may still be in flight when the CTA exits
    for (uint32_t j = 1; j <= kv && j <= static_cast<uint32_t>(kSlots); ++j)
      (void)mbar_wait_bounded(&bar_full[(kv - j) % kSlots], ((kv - j) / kSlots) & 1);
    if (k > 0) (void)mbar_wait_bounded(bar_q_full, (k - 1) & 1);
  } else if (warp == kMmaWarp) {
    // ===================================================================== MMA issue (elected lane)
    const uint32_t idesc_qk = x_idesc(kKeys, false);
    const uint32_t idesc_pv = x_idesc(kD, true);
    const uint64_t dq = sw128_desc(smem_u32(sQ), 16, 1024);
    const uint64_t dk0 = sw128_desc(smem_u32(sKV), 16, 1024);
    const uint64_t dv0 = sw128_desc(smem_u32(sKV), kKvChunk, 1024);
    uint32_t kv = 0, nqk = 0, npv = 0;  // K and V tiles of finished items; QKs and PVs issued
    Item it;
    for (uint32_t k = 0; ok; ++k) {
      if (!take_item(k, it)) { ok = false; break; }
      if (!it.live) break;
      const int32_t n = key_tiles(it);
      if (!warp_wait_far(bar_q_full, k & 1)) { ok = false; break; }
      auto landed = [&](uint32_t u) -> bool { return warp_wait_far(&bar_full[u % kSlots], (u / kSlots) & 1); };
      // QK of key tile j.  Its S buffer was read by the softmax two tiles back, whose P the PV issued last has waited for.
      auto qk = [&](int32_t j) -> bool {
        const uint32_t u = kv + 2 * j;
        if (!landed(u)) return false;
        tc_fence_after();
        const uint64_t dk = dk0 + static_cast<uint64_t>((u % kSlots) * (kKvTile >> 4));
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          mma_chunk(tmem + kSCol + (nqk & 1) * kKeys, dq + c * (kQChunk >> 4), dk + c * (kKvChunk >> 4), idesc_qk,
                    c > 0 ? 1u : 0u);
        mma_commit(&bar_s_full[nqk & 1]);
        mma_commit(&bar_empty[u % kSlots]);
        ++nqk;
        return true;
      };
      auto pv = [&](int32_t j) -> bool {
        const uint32_t u = kv + 2 * j + 1;
        if (!warp_wait_far(&bar_p_full[npv & 1], (npv >> 1) & 1)) return false;
        tc_fence_after();
        mma_pv(tmem + kOCol, tmem + kPCol + (npv & 1) * (kKeys / 2),
               dv0 + static_cast<uint64_t>((u % kSlots) * (kKvTile >> 4)), idesc_pv, j > 0 ? 1u : 0u);
        mma_commit(&bar_pv_done[npv & 1]);
        mma_commit(&bar_empty[u % kSlots]);
        ++npv;
        return true;
      };
      // (the first output and the last tile are taken out of the loop: its path is what the softmax waits for)
      if (!qk(0)) { ok = false; break; }
      for (int32_t j = 0; j < n - 1; ++j) {
        if (!qk(j + 1)) { ok = false; break; }
        if (j == 0 && k > 0 && !warp_wait_far(bar_o_free, (k - 1) & 1)) { ok = false; break; }
        if (!landed(kv + 2 * j + 1) || !pv(j)) { ok = false; break; }
      }
      if (!ok) break;
      mma_commit(bar_q_empty);
      const uint32_t u = kv + 2 * n - 1;
      if (!landed(u)) { ok = false; break; }
      if (it.len - (n - 1) * kKeys < kKeys)
        clear_rows<kChunks, kKeys>(sKV + (u % kSlots) * kKvTile, it.len - (n - 1) * kKeys);
      if (n == 1 && k > 0 && !warp_wait_far(bar_o_free, (k - 1) & 1)) { ok = false; break; }
      if (!pv(n - 1)) { ok = false; break; }
      kv += 2 * n;
    }
    // before tensor memory is freed, every MMA issued must have completed
    if (npv > 0) (void)mbar_wait_bounded(&bar_pv_done[(npv - 1) & 1], ((npv - 1) >> 1) & 1);
    if (nqk > 0) (void)mbar_wait_bounded(&bar_s_full[(nqk - 1) & 1], ((nqk - 1) >> 1) & 1);
  } else {
    // ===================================================================== softmax warps
    const int r = tid;  // row = tensor-memory lane
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tO = tmem + kOCol + lane_base;
    uint32_t nt = 0;  // key tiles processed
    Item it;
    for (uint32_t k = 0; ok; ++k) {
      if (!take_item(k, it)) { ok = false; break; }
      if (!it.live) break;
      const int32_t n = key_tiles(it);
      const int32_t tok = it.blk[0] * kM + r;
      float m = -INFINITY;
      float2 l2 = make_float2(0.0f, 0.0f);
      for (int32_t j = 0; j < n; ++j, ++nt) {
        const uint32_t b = nt & 1;
        const uint32_t tS = tmem + kSCol + b * kKeys + lane_base, tP = tmem + kPCol + b * (kKeys / 2) + lane_base;
        if (!warp_wait_far(&bar_s_full[b], (nt >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[kKeys];
        float top;
        if ((j + 1) * kKeys <= it.blk[0] * kM) {
          uint32_t mx[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_ld32_max_issue(tS + 32 * c, s + 32 * c, mx[c]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_wait_ld32(s + 32 * c);
            tmem_wait_max(mx[c]);
          }
          top = fmaxf(__uint_as_float(mx[0]), __uint_as_float(mx[1]));
        } else {  // the tile reaches past the block's first row
          tmem_ld32_issue(tS, s);
          tmem_ld32_issue(tS + 32, s + 32);
          tmem_wait_ld32(s);
          tmem_wait_ld32(s + 32);
          const int32_t last = tok - j * kKeys;  // this row sees keys <= last of the tile
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kKeys; ++e) {
            s[e] = e <= last ? s[e] : 0xFF800000u;
            mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
          }
          top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        }
        top *= a.score_scale;
        if (j == 0) {
          m = top;
        } else {
          const bool moved = top > m + kLazyRescale;
          if (__any_sync(0xffffffffu, moved)) {
            const float alpha = moved ? ex2(m - top) : 1.0f;
            m = moved ? top : m;
            // O must hold the PV of the tile before
            if (!warp_wait_far(&bar_pv_done[(nt - 1) & 1], ((nt - 1) >> 1) & 1)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kD / 16; ++c) {
              float o[16];
              tmem_ld16(tO + c * 16, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= alpha;
              tmem_st16(tO + c * 16, o);
            }
            l2.x *= alpha;
            l2.y *= alpha;
          }
        }
        const float2 sc2 = make_float2(a.score_scale, a.score_scale), m2 = make_float2(-m, -m);
        uint32_t pw[kKeys / 2];
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e) {
          const float2 x = ffma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), sc2, m2);
          const float2 p = make_float2(ex2(x.x), ex2(x.y));
          l2 = fadd2(l2, p);
          pw[e] = pack_bf16x2(p.x, p.y);
        }
        // the P buffer was last read by the PV two tiles back
        if (nt >= 2 && !warp_wait_far(&bar_pv_done[b], ((nt >> 1) - 1) & 1)) { ok = false; break; }
        tc_fence_after();
        tmem_st32(tP, pw);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar_p_full[b]);
      }
      if (!ok) break;
      // O / l of this row, once the item's last PV has completed
      if (!warp_wait_far(&bar_pv_done[(nt - 1) & 1], ((nt - 1) >> 1) & 1)) { ok = false; break; }
      tc_fence_after();
      const float inv = 1.0f / (l2.x + l2.y);
      const int32_t tok0 = it.blk[0] * kM + warp * 32;  // the warp's first row
      const int64_t orow = static_cast<int64_t>(it.q0 + tok0) * a.out_token + static_cast<int64_t>(it.head[0]) * a.out_head;
#pragma unroll 1
      for (int c = 0; c < kD / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(tO + c * 32, ov);
        if (a.out_dtype == KVQ_OUT_F32) store_rows32<true>(a, sStage + warp * 2048, orow + c * 32, it.len - tok0, ov, inv);
        else store_rows32<false>(a, sStage + warp * 2048, orow + c * 32, it.len - tok0, ov, inv);
      }
      tc_fence_before();  // the reads are ordered before the arrival that lets the next PV overwrite O
      __syncwarp();
      if (lane == 0) bar_arrive(bar_o_free);
    }
  }
  if (!ok) prompt_report(a, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

}  // namespace

kvq_status launch_prompt_wide(const PromptArgs& a, cudaStream_t stream) {
  if (cudaFuncSetAttribute(prompt_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
    return KVQ_ECUDA;
  CUtensorMap qm, km, vm;
  if (!encode_rows(&qm, a.q, a.total, a.num_q_heads, kD, a.q_token, a.q_head, kM) ||
      !encode_rows(&km, a.k, a.total, a.num_kv_heads, kD, a.k_token, a.k_head, kKeys) ||
      !encode_rows(&vm, a.v, a.total, a.num_kv_heads, kD, a.v_token, a.v_head, kKeys))
    return KVQ_ECUDA;
  const int64_t blocks = static_cast<int64_t>(a.total) / kM + std::min<int64_t>(a.batch, a.total);  // at most
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(blocks * a.num_q_heads, a.sms));
  return launch_cleared(prompt_wide_kernel, a, grid, kThreads, kSmem, qm, km, vm, stream);
}

}  // namespace kvq
