// kvq_page_flash.cu -- causal attention of many query rows over a KVQ_FP8_E4M3_PAGE cache (kvq_extend), on the tcgen05 tensor
// cores, head_dim 64, 128 and 256, any number of query heads per kv head.  With K = 2^ek[page] code, V = 2^ev[page] code:
//   y_t = log2(e) sm_scale 2^ek q.code_t + ev,   p_t = 2^(y_t - m),   out = sum p_t code_t / sum 2^-ev p_t.
// 4 D FLOPs per (row, key) against 2 D bytes per key for up to 256 rows: the tensor pipe's floor.
//
// K's scales never meet a code, so its codes go to the tensor cores as they lie in the pool: S = Q . K^T in 8 bits,
// with each row of q, scaled by a power of two, as the sum of an E5M2 and an E4M3 term: bf16 has 8 significant bits;
// the first takes 3 of them, and what is left of an element in [2^e, 2^(e + 1)) is a multiple of 2^(e - 7) up to
// 2^(e - 3), which 4 bits hold.  With the row's largest element in [2^11, 2^12) (what is left of it then ends below 448),
// elements of 2^-13 of it and more enter exactly, smaller ones are off by at most 2^-21 of it (half of E4M3's least
// step, 2^-10, to 2^11).  Two E4M3 terms with the largest in [2^7, 2^8) were exact down to 2^-9 of it and off by up
// to 2^-17.  Two 8-bit products take the time of one 16-bit one and need no conversion of K.  For the output P has to
// keep more bits than 8-bit terms give cheaply (two terms would cost five instructions a probability), so V's codes
// become f16 instead, exactly and once for up to 256 rows, and P is rounded to f16: 2^-11, or 2^-28 of the row's
// largest p where V's scales are within 2^18 (codes_down).
//
// A tile is 128 query rows of one kv head: tokens times heads of its group (at most 128 heads; larger groups are cut).
// Tensor memory at head_dim 64 and 128: S_A, S_B, O_A, O_B, two tiles A and B of a CTA whose softmax and MMAs alternate; at
// 256 one tile, with two S buffers of 64 keys.  P (f16) replaces the S it was made from.
// Warps: softmax (one per lane quarter and tile, one thread per row), one that issues all MMAs, one that finds the work,
// reads block table and scales and loads K and V codes with TMA (a page's 16 rows as one box), two that turn V's codes
// into f16 (and clear rows behind the sequence's end and of masked pages, which may hold anything: 0 * NaN would be NaN).
// Work: a unit is a key tile of an item (one or two tiles of a kv head).  All units lie in one order, and every CTA takes an
// equal run of them, so that a few long contexts fill the GPU as well as many short ones.  A run that is all of an item
// gives its output, other runs leave partial sums for a second kernel, its programmatic dependent.
// Measured: 2048 tokens after 30000 with 32 heads of 128 over 8: 719 us, 1.45 PFLOP/s, 75% of the bf16 GEMM rate;
// eight turns of 100 to 1024 tokens after 700 to 8192, 16 heads over 8: 228 us, 1.0 PFLOP/s; four turns of 600 to
// 2048 tokens with 32 heads of 64 over 8: 123 us, 0.43 PFLOP/s.  No pipe is busy in these two (tensor 51 and 24%,
// exponentials 25 and 24%): what is left is the way from scores to P, one key tile after the other, and the items'
// starts, six key tiles' time each, in which the softmax warps fetch q.  head_dim 256, one tile a CTA: 2048 tokens
// after 30000, 16 heads over 2: 1200 us, 0.87 PFLOP/s.  The rows' scores stay in registers (128 of a row at head_dim
// 64 and 128): read twice from tensor memory the first case took 960 us.
// Every wait is bounded (2 s) and reports a timeout in the status word instead of hanging.
#include <cuda.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_flash.cuh"
#include "kvq_internal.h"
#include "kvq_page.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace {

constexpr int kM = 128;           // rows of a tile
constexpr int kConvWarps = 2;     // that turn V's codes into f16
constexpr int kTmemCols = 512;

// What a row's factor from codes to scores is kept within, so that it is neither 0 nor infinite once a page's scale (2^-32 ..
// 2^32) has joined it: 0 times the -inf of an unseen key would be NaN.  It changes no result: under 2^-94 every score is
// below 2^-30 (|S| < 2^29), and from 2^65 on scores that differ at all do so by more than 2^7, which leaves the largest alone.
constexpr float kMultLeast = 0x1p-94f, kMultMost = 0x1p65f;
// A row whose reference would pass this is given up: NaN, and a report.  Its reference is then above every score.
// One fused multiply-add makes a key's exponent of its product and keeps bits of that which the reference has rounded
// away: half a unit at most here, and from 2^24 on more than f16 has room for.  To round the scores first where they
// are large cost 2 to 7% of the calls where none are (a branch in the softmax).
constexpr float kFarScore = 0x1p22f, kGivenUp = 0x1.fffffep127f;

// What the softmax and the converting warps know of the pages of a key tile.
template <int PAGES>
struct alignas(16) PageInfo {
  float ks[PAGES];                // K's scale (1 for a masked page)
  float ev[PAGES], unv[PAGES];    // V's exponent but for what the codes take of it, and 2^-ev
  uint8_t rows[PAGES];            // rows that hold tokens; 0: masked
  uint8_t down[PAGES];            // V's codes take 2^-down of the scale
  int32_t full;                   // every page of the tile has all its rows
  int32_t any_down;
};

template <int D>
struct FCfg {
  static constexpr int TILES = D == 256 ? 1 : 2;
  static constexpr int KT = D == 256 ? 64 : 128;        // keys of a key tile
  static constexpr int PAGES = KT / kPage;
  static constexpr int SLICES = D == 256 ? 2 : 1;       // 128-byte (D = 64: 64-byte) slices of a row of codes
  static constexpr int SLICE = D == 64 ? 64 : 128;
  static constexpr int Q_TERM = kM * D;                 // bytes of one term of a tile's q
  static constexpr int K_TILE = KT * D, V_TILE = 2 * KT * D;
  static constexpr int KST = 3, VST = 2;                // stages of K codes; of V codes and of V in f16
  // Key tiles whose pages are described in shared memory.  A slot is written once QK of the tile KST before has completed; by
  // then all have read that of the tile before that one (one tile per CTA: two before).
  static constexpr int INFO = TILES == 2 ? 4 : 8;
  static_assert(INFO >= KST + (TILES == 2 ? 1 : 2), "info slots");
  static constexpr int ITEMS = 4;                       // item slots
  static constexpr int SM_WARPS = 4 * TILES;
  static constexpr int MMA_WARP = SM_WARPS, LOAD_WARP = SM_WARPS + 1, CONV_WARP = SM_WARPS + 2;
  static constexpr int THREADS = (SM_WARPS + 2 + kConvWarps) * 32;
  static constexpr int Q_OFF = 0;                       // 1024-byte aligned: swizzle atoms
  static constexpr int K_OFF = Q_OFF + TILES * 2 * Q_TERM;
  static constexpr int C_OFF = K_OFF + KST * K_TILE;    // V codes
  static constexpr int V_OFF = C_OFF + VST * K_TILE;
  static constexpr int STG_OFF = V_OFF + VST * V_TILE;  // [softmax warps] 2 KB of output
  static constexpr int INFO_OFF = STG_OFF + SM_WARPS * 2048;
  static constexpr int ITEM_OFF = INFO_OFF + INFO * static_cast<int>(sizeof(PageInfo<PAGES>));
  static constexpr int BAR_OFF = ITEM_OFF + ITEMS * 64;
  static constexpr int NBARS = 2 * KST + 4 * VST + INFO + 10 + 2 * ITEMS;
  static constexpr int SMEM = BAR_OFF + NBARS * 8 + 16 + 1024;  // + slack to align the base
  static constexpr int O_COL = D == 256 ? 128 : 256;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(O_COL + TILES * D <= kTmemCols, "tensor memory");
};

// A run of an item's key tiles.  A CTA leaves its first one in the workspace where that begins inside an item, for the
// joining kernel.
struct Item {
  __device__ __forceinline__ int32_t token_of(int32_t r) const { return static_cast<int32_t>(r * per_head >> 16); }
  int64_t first;                  // the item's first unit
  int32_t live, q0, n, len;
  int32_t head0, heads;           // first query head of the group, heads of it
  int32_t tok0;                   // first token of the item
  uint32_t per_head;              // 2^16 / heads, rounded up: r * per_head >> 16 = r / heads for r < 128
  int32_t kt0, kt1, all;          // key tiles of the run; of the item
  __device__ __forceinline__ bool whole() const { return kt0 == 0 && kt1 == all; }
};
static_assert(sizeof(Item) <= kPageRunMost && sizeof(Item) <= 64, "item slots");

// Sum over i < n of floor((a i + b) / m), a, b >= 0 (the lattice points under a line, by the Euclidean algorithm).
__device__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t s = 0;
  while (n > 0) {
    s += (n - 1) * n / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t top = a * n + b;
    n = top / m;
    b = top % m;
    const int64_t t = m;
    m = a;
    a = t;
    if (m == 0) break;
  }
  return s;
}

// How a call's rows fall into items: groups of at most 128 heads, tokens of a tile and of an item.
template <int D>
struct Shape {
  using Cfg = FCfg<D>;
  int32_t G, groups, heads, tile_tok, item_tok;  // groups: per kv head; heads: of a group (the last may have fewer)
  __device__ __forceinline__ explicit Shape(const PageArgs& a) {
    G = a.num_q_heads / a.num_kv_heads;
    groups = (G + kM - 1) / kM;
    heads = (G + groups - 1) / groups;
    groups = (G + heads - 1) / heads;
    tile_tok = kM / heads;
    item_tok = tile_tok * Cfg::TILES;
  }
  __device__ __forceinline__ int32_t items(const PageSeq& s) const { return (s.n + item_tok - 1) / item_tok; }
  // key tiles that item p of a sequence sees
  __device__ __forceinline__ int32_t key_tiles(const PageSeq& s, int32_t p) const {
    const int64_t last = s.len - s.n + min(static_cast<int64_t>(s.n), static_cast<int64_t>(p + 1) * item_tok);
    return static_cast<int32_t>((last + Cfg::KT - 1) / Cfg::KT);
  }
  // units of the items before p (p < items: all of these have item_tok tokens): their key tiles, and a start for each
  __device__ __forceinline__ int64_t before(const PageSeq& s, int32_t p) const {
    return floor_sum(p, Cfg::KT, item_tok, static_cast<int64_t>(s.len - s.n) + item_tok + Cfg::KT - 1) +
           static_cast<int64_t>(p) * kPageItemUnits;
  }
  __device__ __forceinline__ int64_t per_group(const PageSeq& s) const {
    if (s.n == 0) return 0;
    const int32_t p = items(s) - 1;
    return before(s, p) + kPageItemUnits + key_tiles(s, p);
  }
  __device__ __forceinline__ int64_t units(const PageArgs& a, const PageSeq& s) const {
    return per_group(s) * groups * a.num_kv_heads;
  }
  // the item in which unit `local` of a sequence lies; returns the units from the item's start to it
  __device__ __forceinline__ int64_t locate(const PageSeq& s, int64_t local, int32_t& group, int32_t& p) const {
    const int64_t per = per_group(s);
    group = static_cast<int32_t>(local / per);
    const int64_t rest = local - group * per;
    int32_t lo = 0, hi = items(s) - 1;  // the last item that begins at or before `rest`
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) / 2;
      if (before(s, mid) <= rest) lo = mid;
      else hi = mid - 1;
    }
    p = lo;
    return rest - before(s, p);
  }
};

// S = Q . K^T in 8 bits over a slice of STEPS k-steps of 32 bytes, both terms of q (`term` descriptor units apart, the second
// with an instruction descriptor of its own) into the same sums, from one elect.sync.
template <int STEPS>
__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint64_t term, uint32_t idesc, uint32_t idesc2,
                                        uint32_t acc) {
  if constexpr (STEPS == 4) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 a1, a2, a3, c0, c1, c2, c3, b1, b2, b3;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
        "add.u64 c0, %1, %5;\n\tadd.u64 c1, c0, 2;\n\tadd.u64 c2, c0, 4;\n\tadd.u64 c3, c0, 6;\n\t"
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], c0, %2, %6, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], c1, b1, %6, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], c2, b2, %6, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], c3, b3, %6, 1;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "l"(term), "r"(idesc2)
        : "memory");
  } else {
    static_assert(STEPS == 2, "2 or 4 steps");
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 a1, c0, c1, b1;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 c0, %1, %5;\n\tadd.u64 c1, c0, 2;\n\tadd.u64 b1, %2, 2;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], c0, %2, %6, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], c1, b1, %6, 1;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "l"(term), "r"(idesc2)
        : "memory");
  }
}

// Instruction descriptor: M = 128, N columns, fp32 sums; E4M3 x E4M3 and f16 x f16 both have code 0, E5M2 for A adds kE5M2A.
constexpr uint32_t kE5M2A = 1u << 7;
__device__ __forceinline__ uint32_t page_idesc(int n, bool b_mn_major) {
  return 1u << 4 | static_cast<uint32_t>(b_mn_major) << 16 | static_cast<uint32_t>(n >> 3) << 17 |
         static_cast<uint32_t>(kM >> 4) << 24;
}

// 16 columns of this lane's row and their maximum.
__device__ __forceinline__ void tmem_ld16_max_issue(uint32_t taddr, uint32_t* r, uint32_t& top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(top)
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait16_max(uint32_t* r, uint32_t& top) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(top)
               :
               : "memory");
}

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void cp_async16(uint8_t* to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}

// Two values as the sum of an E5M2 and an E4M3 term each: codes of the nearest and of what is left.
__device__ __forceinline__ void fp8_terms(uint32_t f16x2, uint32_t& hi, uint32_t& lo) {
  asm("{\n\t.reg .b16 h, l;\n\t.reg .b32 b, d;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 h, %2;\n\tcvt.rn.f16x2.e5m2x2 b, h;\n\tsub.f16x2 d, %2, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 l, d;\n\tcvt.u32.u16 %0, h;\n\tcvt.u32.u16 %1, l;\n\t}"
      : "=r"(hi), "=r"(lo)
      : "r"(f16x2));
}

// Multiplies the f16 that a lane of a converting warp has written by what their pages' codes take of the scales; out of line, as
// hardly any key tile needs it.
template <int D>
__device__ __noinline__ void take_down(uint8_t* v, const uint8_t* down, int cw, int r8, int c4) {
  constexpr int KT = FCfg<D>::KT, PER_ROW = D / 64;
  for (int i = cw; i < KT / 8 * PER_ROW; i += kConvWarps) {
    const int row = i / PER_ROW * 8 + r8;
    const uint32_t f = f16x2_power(down[row / kPage]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint4* x = reinterpret_cast<uint4*>(v + i % PER_ROW * KT * 128 + row * 128 + (((2 * c4 + k) ^ (row & 7)) << 4));
      *x = make_uint4(mul_f16x2(x->x, f), mul_f16x2(x->y, f), mul_f16x2(x->z, f), mul_f16x2(x->w, f));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(FCfg<D>::THREADS, 1)
    page_flash_kernel(const PageArgs a, const __grid_constant__ CUtensorMap map) {
  using Cfg = FCfg<D>;
  constexpr int TILES = Cfg::TILES, KT = Cfg::KT, PAGES = Cfg::PAGES, SLICES = Cfg::SLICES;
  constexpr int KST = Cfg::KST, VST = Cfg::VST, INFO = Cfg::INFO, ITEMS = Cfg::ITEMS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem + Cfg::Q_OFF;  // [tile][term]
  uint8_t* sK = smem + Cfg::K_OFF;  // [KST]
  uint8_t* sC = smem + Cfg::C_OFF;  // [VST] codes of V
  uint8_t* sV = smem + Cfg::V_OFF;  // [VST] V in f16
  using Info = PageInfo<PAGES>;
  Info* sInfo = reinterpret_cast<Info*>(smem + Cfg::INFO_OFF);  // [INFO]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFF);
  uint64_t* bar_k_full = bars;                    // [KST] K codes landed
  uint64_t* bar_k_empty = bar_k_full + KST;       // [KST] their last QK completed (commit)
  uint64_t* bar_c_full = bar_k_empty + KST;       // [VST] V codes landed
  uint64_t* bar_c_empty = bar_c_full + VST;       // [VST] turned into f16
  uint64_t* bar_v_full = bar_c_empty + VST;       // [VST] V in f16 written
  uint64_t* bar_v_empty = bar_v_full + VST;       // [VST] its last PV completed (commit)
  uint64_t* bar_info = bar_v_empty + VST;         // [INFO] the key tile's pages are described
  uint64_t* bar_s_full = bar_info + INFO;        // [2] QK into S buffer w completed (commit)
  uint64_t* bar_p_full = bar_s_full + 2;          // [2] P of buffer w written
  uint64_t* bar_pv_done = bar_p_full + 2;         // [2] PV of buffer w completed (commit)
  uint64_t* bar_q_full = bar_pv_done + 2;         // [TILES] q of the item written
  uint64_t* bar_o_free = bar_q_full + 2;          // [TILES] O read out
  uint64_t* bar_item = bar_o_free + 2;            // [ITEMS] item slot published
  uint64_t* bar_item_free = bar_item + ITEMS;     // [ITEMS] every consuming warp is done with the item
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + Cfg::BAR_OFF + Cfg::NBARS * 8);
  auto sItem = [&](uint32_t k) { return reinterpret_cast<Item*>(smem + Cfg::ITEM_OFF + k % ITEMS * 64); };

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t cta = blockIdx.x;
  const Shape<D> shape(a);
  bool ok = true, bad = false;
  asm volatile("griddepcontrol.launch_dependents;");  // (the joining kernel waits for this one's end)

  page_clear(a);
  if (tid == 0) {
    for (int i = 0; i < KST; ++i) {
      mbar_init(&bar_k_full[i], 1);
      mbar_init(&bar_k_empty[i], 1);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(&bar_c_full[i], 1);
      mbar_init(&bar_c_empty[i], kConvWarps);
      mbar_init(&bar_v_full[i], kConvWarps);
      mbar_init(&bar_v_empty[i], 1);
    }
    for (int i = 0; i < INFO; ++i) mbar_init(&bar_info[i], 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_s_full[w], 1);
      mbar_init(&bar_p_full[w], 4);
      mbar_init(&bar_pv_done[w], 1);
      mbar_init(&bar_q_full[w], 4);
      mbar_init(&bar_o_free[w], 4);
    }
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(&bar_item[i], 1);
      mbar_init(&bar_item_free[i], Cfg::SM_WARPS + 1 + kConvWarps);
    }
    fence_mbar_init();
  }
  if (warp == Cfg::MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sTmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  const Place place = page_place<Cfg::THREADS / 32>(
      a.batch, cta == 0 ? a.total : nullptr, [&](int32_t i) { return shape.units(a, page_sequence(a, i, bad)); },
      [&](int64_t U) {  // this CTA's first unit
        const int32_t C = sharers(U, a.grid, kPageFlashUnits);
        return cta < C && U > 0 ? first_unit(U, C, cta) : U;
      });
  if (cta == 0 && bad) page_report(a, kStatusBadExtend);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sTmem;

  // The k-th item of this CTA, for a consuming warp, stays in its slot until the warp is done with it: as registers its
  // fields would be spilled, and be read back from L2 when they are needed.
  auto take_item = [&](uint32_t k) { return warp_wait_far(&bar_item[k % ITEMS], (k / ITEMS) & 1); };
  auto end_item = [&](uint32_t k) {
    __syncwarp();
    if (lane == 0) bar_arrive(&bar_item_free[k % ITEMS]);
  };

  if (warp == Cfg::LOAD_WARP) {
    // ===================================================================== items, pages, loads
    // The first item is searched for; from there on they are taken in order.
    const int32_t C = sharers(place.total, a.grid, kPageFlashUnits);
    int64_t u = place.b < 0 ? 0 : first_unit(place.total, C, cta);
    const int64_t u_end = place.b < 0 ? 0 : first_unit(place.total, C, cta + 1);
    int32_t b = place.b, group = 0, p = 0, at = 0;  // the next item, and its units before the run
    PageSeq s = {0, 0, 0};
    if (u < u_end) {
      s = page_sequence(a, b, bad);
      at = static_cast<int32_t>(shape.locate(s, u - place.before, group, p));
    }
    uint32_t kv = 0, kc = 0, vc = 0;  // key tiles; K and V stages that hold copies
    for (uint32_t k = 0; ok; ++k) {
      Item it;
      it.live = u < u_end && at + (u_end - u) > kPageItemUnits;  // (a run that ends in an item's start leaves it to the next)
      int32_t g = 0;
      if (it.live) {
        it.first = u - at + kPageItemUnits;
        it.q0 = s.q0;
        it.n = s.n;
        it.len = s.len;
        g = group / shape.groups;
        const int32_t part = group - g * shape.groups;
        it.head0 = g * shape.G + part * shape.heads;
        it.heads = min(shape.heads, shape.G - part * shape.heads);
        it.tok0 = p * shape.item_tok;
        it.per_head = (65536u + it.heads - 1) / it.heads;
        it.kt0 = max(at - kPageItemUnits, 0);
        it.all = shape.key_tiles(s, p);
        it.kt1 = static_cast<int32_t>(min(static_cast<int64_t>(it.all), at + (u_end - u) - kPageItemUnits));
      }
      if (k == 0 && lane == 0) {
        Item x = it;
        x.live = it.live && it.kt0 > 0;
        static_cast<Item*>(a.runs)[cta] = x;
      }
      if (k >= ITEMS && !warp_wait_far(&bar_item_free[k % ITEMS], (k / ITEMS - 1) & 1)) { ok = false; break; }
      if (lane == 0) {
        *sItem(k) = it;
        bar_arrive(&bar_item[k % ITEMS]);
      }
      __syncwarp();
      if (!it.live) break;
      // pages of the run, 32 at a time, one per lane, the next 32 fetched meanwhile
      const int32_t pg0 = it.kt0 * PAGES, np = min(it.kt1 * PAGES, (it.len + kPage - 1) / kPage) - pg0;
      const int32_t* table = a.block_table + static_cast<int64_t>(b) * a.max_pages + pg0;
      auto fetch = [&](int32_t batch) -> int32_t {
        const int32_t i = batch * 32 + lane;
        if (i >= np) return -1;
        const int32_t x = __ldg(table + i);
        if (x < a.num_pages) return x;
        page_report(a, kStatusBadPage);
        return -1;
      };
      auto scales = [&](int32_t x, float& ks, float& vs) {
        ks = vs = 1.0f;
        if (x < 0) return;
        const float* at = a.scales + static_cast<int64_t>(x) * 2 * a.num_kv_heads + g;
        ks = __ldg(at);
        vs = __ldg(at + a.num_kv_heads);
      };
      constexpr int BATCH = 32 / PAGES;  // key tiles whose pages the lanes hold
      int32_t phys = fetch(0), phys_next = fetch(1);
      float ks, vs, ks_next = 1.0f, vs_next = 1.0f;
      scales(phys, ks, vs);
      int32_t ref = -127, e = 0, down = 0;  // V's largest exponent so far; the lane's page's, and what its codes take
      uint32_t downs = 0;                   // lanes whose page's codes take some
      auto shares = [&] {                   // (of the 32 pages that the lanes hold)
        e = phys >= 0 ? scale_exponent(vs) : -127;
        ref = max(ref, __reduce_max_sync(0xffffffffu, e));
        down = phys >= 0 ? codes_down(e, ref) : 0;
        downs = __ballot_sync(0xffffffffu, down > 0);
      };
      shares();
      for (int32_t j = 0; j < it.kt1 - it.kt0; ++j, ++kv) {
        if (j > 0 && j % BATCH == 0) {
          phys = phys_next;
          ks = ks_next;
          vs = vs_next;
          phys_next = fetch(j / BATCH + 1);
          shares();
        }
        if (j % BATCH == 1) scales(phys_next, ks_next, vs_next);
        const int32_t first = j % BATCH * PAGES;            // the lane of the tile's first page
        const bool mine = lane >= first && lane < first + PAGES;
        const int32_t x = lane - first;                     // page of the tile
        const uint32_t count = __popc(__ballot_sync(0xffffffffu, mine && phys >= 0));
        const int sk = kv % KST, sv = kv % VST;
        if (kv >= KST && !warp_wait_far(&bar_k_empty[sk], (kv / KST - 1) & 1)) { ok = false; break; }
        Info& info = sInfo[kv % INFO];
        const int32_t rows = mine && phys >= 0 ? min(kPage, it.len - (pg0 + j * PAGES + x) * kPage) : 0;
        const uint32_t fulls = __popc(__ballot_sync(0xffffffffu, rows == kPage));
        if (mine) {
          info.ks[x] = phys >= 0 ? ks : 1.0f;
          info.ev[x] = phys >= 0 ? static_cast<float>(e + down) : 0.0f;
          info.unv[x] = phys >= 0 ? power_inverse(e + down) : 1.0f;
          info.rows[x] = static_cast<uint8_t>(rows);
          info.down[x] = static_cast<uint8_t>(down);
          if (x == 0) {
            info.full = fulls == PAGES;
            info.any_down = downs >> first & ((1u << PAGES) - 1);
          }
        }
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&bar_info[kv % INFO]);
          mbar_arrive_expect_tx(&bar_k_full[sk], count * kPage * D);
        }
        __syncwarp();
        if (mine && phys >= 0) {
#pragma unroll
          for (int s = 0; s < SLICES; ++s)
            tma_load_codes(smem_u32(sK + sk * Cfg::K_TILE + s * KT * Cfg::SLICE + x * kPage * Cfg::SLICE), &map, s, g * kPage,
                           0, phys, &bar_k_full[sk]);
        }
        kc = kv + 1;
        __syncwarp();
        if (kv >= VST && !warp_wait_far(&bar_c_empty[sv], (kv / VST - 1) & 1)) { ok = false; break; }
        if (lane == 0) mbar_arrive_expect_tx(&bar_c_full[sv], count * kPage * D);
        __syncwarp();
        if (mine && phys >= 0) {
#pragma unroll
          for (int s = 0; s < SLICES; ++s)
            tma_load_codes(smem_u32(sC + sv * Cfg::K_TILE + s * KT * Cfg::SLICE + x * kPage * Cfg::SLICE), &map, s, g * kPage,
                           1, phys, &bar_c_full[sv]);
        }
        vc = kv + 1;
        __syncwarp();
      }
      if (!ok) break;
      u += kPageItemUnits + it.kt1 - at;
      at = 0;
      if (u < u_end && ++p == shape.items(s)) {  // (a run that ends inside an item is the CTA's last)
        p = 0;
        if (++group == shape.groups * a.num_kv_heads) {
          group = 0;
          do s = page_sequence(a, ++b, bad);
          while (s.n == 0);
        }
      }
    }
    // no copy may still be in flight when the CTA exits
    for (uint32_t j = 1; j <= kc && j <= static_cast<uint32_t>(KST); ++j)
      (void)mbar_wait_bounded(&bar_k_full[(kc - j) % KST], ((kc - j) / KST) & 1);
    for (uint32_t j = 1; j <= vc && j <= static_cast<uint32_t>(VST); ++j)
      (void)mbar_wait_bounded(&bar_c_full[(vc - j) % VST], ((vc - j) / VST) & 1);
  } else if (warp >= Cfg::CONV_WARP) {
    // ===================================================================== V's codes to f16
    // A warp takes 8 rows x 64 codes at a time: lanes 4 h .. 4 h + 3 the four 16-byte pieces of a row, rows r and r ^ 5
    // side by side, so that neither the reads of 16 bytes nor the writes of 2 x 16 meet in a bank.
    const int32_t cw = warp - Cfg::CONV_WARP;
    const int r8 = (lane >> 3) ^ (lane & 4 ? 5 : 0), c4 = lane & 3;
    uint32_t kv = 0;
    for (uint32_t k = 0; ok; ++k) {
      if (!take_item(k)) { ok = false; break; }
      const Item& it = *sItem(k);
      if (!it.live) break;
      const int32_t n = it.kt1 - it.kt0;
      end_item(k);
      for (int32_t j = 0; j < n; ++j, ++kv) {
        const int s = kv % VST;
        if (!warp_wait_far(&bar_info[kv % INFO], (kv / INFO) & 1) || !warp_wait_far(&bar_c_full[s], (kv / VST) & 1) ||
            (kv >= VST && !warp_wait_far(&bar_v_empty[s], (kv / VST - 1) & 1))) {
          ok = false;
          break;
        }
        const uint8_t* src = sC + s * Cfg::K_TILE;
        uint8_t* dst = sV + s * Cfg::V_TILE;
        const Info& info = sInfo[kv % INFO];
        const int32_t some_down = *const_cast<const volatile int32_t*>(&info.any_down);  // (here, not behind the codes' loop)
        constexpr int PER_ROW = D / 64;  // steps of 64 codes in a row
#pragma unroll 2
        for (int i = cw; i < KT / 8 * PER_ROW; i += kConvWarps) {
          const int row = i / PER_ROW * 8 + r8, step = i % PER_ROW;
          const int c = step * 4 + c4;   // 16-byte piece of the row of codes
          uint4 w;
          if constexpr (D == 64)
            w = *reinterpret_cast<const uint4*>(src + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
          else
            w = *reinterpret_cast<const uint4*>(src + c / 8 * KT * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
          const bool live = row % kPage < info.rows[row / kPage];
          const uint32_t in[4] = {live ? w.x : 0u, live ? w.y : 0u, live ? w.z : 0u, live ? w.w : 0u};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) codes_to_f16x2<KVQ_FP8_E4M3>(in[e], h[2 * e], h[2 * e + 1]);
          uint8_t* to = dst + step * KT * 128 + row * 128;  // 64 f16: 128-byte rows
          *reinterpret_cast<uint4*>(to + (((2 * c4) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(to + (((2 * c4 + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        if (some_down) take_down<D>(dst, info.down, cw, r8, c4);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&bar_v_full[s]);
          bar_arrive(&bar_c_empty[s]);
        }
      }
    }
  } else if (warp == Cfg::MMA_WARP) {
    // ===================================================================== MMA issue (elected lane)
    const uint32_t idesc_qk = page_idesc(KT, false), idesc_pv = page_idesc(D, true);
    auto k_major = [&](const uint8_t* p) {
      return D == 64 ? smem_desc(smem_u32(p), 16, 512) | static_cast<uint64_t>(4) << 61 : sw128_desc(smem_u32(p), 16, 1024);
    };
    const uint64_t dq0 = k_major(sQ), dk0 = k_major(sK), dv0 = sw128_desc(smem_u32(sV), KT * 128, 1024);
    uint32_t ks = 0, kp = 0, vs = 0, vp = 0;   // stage and parity of the K and the V ring
    uint32_t nt[2] = {0, 0}, ni[2] = {0, 0};   // PVs issued from S buffer w; items of tile w
    auto qk = [&](int w, uint32_t buf) -> bool {
      // P of the buffer's last PV lies in the columns that this QK writes
      if (nt[buf] > 0 && !warp_wait_far(&bar_pv_done[buf], (nt[buf] - 1) & 1)) return false;
      tc_fence_after();
      const uint64_t q = dq0 + ((w * 2 * Cfg::Q_TERM) >> 4), kk = dk0 + ks * (Cfg::K_TILE >> 4);
#pragma unroll
      for (int s = 0; s < SLICES; ++s)
        mma_fp8<Cfg::SLICE / 32>(tmem + buf * KT, q + ((s * kM * 128) >> 4), kk + ((s * KT * 128) >> 4), Cfg::Q_TERM >> 4,
                                 idesc_qk | kE5M2A, idesc_qk, s > 0 ? 1u : 0u);
      mma_commit(&bar_s_full[buf]);
      return true;
    };
    auto pv = [&](int w, uint32_t buf, bool first) -> bool {
      if (first && ni[w] > 1 && !warp_wait_far(&bar_o_free[w], (ni[w] - 2) & 1)) return false;
      if (!warp_wait_far(&bar_p_full[buf], nt[buf] & 1)) return false;
      tc_fence_after();
      // a k-step is 16 keys: 8 columns of P, 16 rows of V
      const uint32_t o = tmem + Cfg::O_COL + w * D, acc = first ? 0u : 1u;
      const uint64_t v = dv0 + vs * (Cfg::V_TILE >> 4), step = (16 * 128) >> 4;
      if constexpr (KT == 128) mma8_bf16_tmem_a(o, tmem + buf * KT, 8u, v, step, idesc_pv, acc);
      else mma4_bf16_tmem_a(o, tmem + buf * KT, 8u, v, step, idesc_pv, acc);
      mma_commit(&bar_pv_done[buf]);
      ++nt[buf];
      return true;
    };
    auto k_there = [&] { return warp_wait_far(&bar_k_full[ks], kp); };
    auto v_there = [&] { return warp_wait_far(&bar_v_full[vs], vp); };
    auto k_done = [&] {
      mma_commit(&bar_k_empty[ks]);
      if (++ks == KST) {
        ks = 0;
        kp ^= 1;
      }
    };
    auto v_done = [&] {
      mma_commit(&bar_v_empty[vs]);
      if (++vs == VST) {
        vs = 0;
        vp ^= 1;
      }
    };
    for (uint32_t k = 0; ok; ++k) {
      if (!take_item(k)) { ok = false; break; }
      const Item& it = *sItem(k);
      if (!it.live) break;
      const int32_t n = it.kt1 - it.kt0;
      const bool two = TILES == 2 && it.tok0 + shape.tile_tok < it.n;
      end_item(k);
      if (!warp_wait_far(&bar_q_full[0], ni[0]++ & 1)) { ok = false; break; }
      if (two && !warp_wait_far(&bar_q_full[1], ni[1]++ & 1)) { ok = false; break; }
      if (two) {
        // QK_A(j), PV_B(j - 1), QK_B(j), PV_A(j): a softmax has the time of two MMA groups
        ok = k_there() && qk(0, 0) && qk(1, 1);
        if (ok) {
          k_done();
          ok = v_there() && pv(0, 0, true);
        }
        for (int32_t j = 1; ok && j < n; ++j) {
          ok = k_there() && qk(0, 0) && pv(1, 1, j == 1);
          if (!ok) break;
          v_done();
          ok = qk(1, 1);
          if (!ok) break;
          k_done();
          ok = v_there() && pv(0, 0, false);
        }
        ok = ok && pv(1, 1, n == 1);
        if (ok) v_done();
      } else {
        // one tile: QK(j), PV(j - 1), through two S buffers where there is but one tile anyway
        const uint32_t alt = TILES == 1 ? 1u : 0u;
        uint32_t buf = TILES == 1 ? (nt[0] + nt[1]) & 1 : 0u;
        for (int32_t j = 0; ok && j < n; ++j) {
          if (alt || j == 0) ok = k_there() && qk(0, buf);
          if (ok && (alt || j == 0)) k_done();
          if (alt) {
            if (ok && j > 0) ok = v_there() && pv(0, buf ^ 1, j == 1);
            if (ok && j > 0) v_done();
            buf ^= 1;
          } else {
            if (ok) ok = v_there() && pv(0, 0, j == 0);
            if (ok) v_done();
            if (ok && j + 1 < n) {
              ok = k_there() && qk(0, 0);
              if (ok) k_done();
            }
          }
        }
        if (alt && ok) ok = v_there() && pv(0, buf ^ 1, n == 1);
        if (alt && ok) v_done();
      }
    }
    // before tensor memory is freed, every MMA issued must have completed
    for (int w = 0; w < 2; ++w)
      if (nt[w] > 0) (void)mbar_wait_bounded(&bar_pv_done[w], (nt[w] - 1) & 1);
  } else {
    // ===================================================================== softmax warps
    const int w = warp >> 2;                   // tile
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + Cfg::O_COL + w * D + lane_base;
    const int32_t r = (warp & 3) * 32 + lane;  // this thread's row of the tile
    uint8_t* const stage = smem + Cfg::STG_OFF + warp * 2048;
    uint32_t kv = 0;  // key tiles of finished items
    uint32_t nt = 0;  // key tiles processed
    float m = kNoMax, l = 0.0f, mult = 0.0f;
    int32_t lim = 0, lim_least = 0;  // tokens that the row sees; the least of the warp's
    constexpr int PER_LINE = D / 8, ROWS = 32 / PER_LINE;  // lanes of a row of q, rows of a step
    const int c16 = lane % PER_LINE, sub = lane / PER_LINE;
    uint8_t* const q_own = sQ + w * 2 * Cfg::Q_TERM;
    auto q_raw = [&](int rr) {  // this lane's 16 bytes of row rr of the tile
      const int at = c16 * 16 % D;
      return q_own + c16 * 16 / D * Cfg::Q_TERM + at / 128 * kM * 128 + rr * Cfg::SLICE + at % 128;
    };
    bool open = false;  // an item's output is still to be written: k - 1
    for (uint32_t k = 0;; ++k) {
      if (!take_item(k)) { ok = false; break; }
      const Item& it = *sItem(k);
      const bool mine = it.live && it.tok0 + w * shape.tile_tok < it.n;  // it has this tile
      const bool was_live = lim != 0x7fffffff;
      // ---- its q, before the output of the item before, so that its first QK runs meanwhile.  The QKs of the item before
      // have completed.  The warp's 32 rows are fetched into their own place, 16 bytes a lane, the first half of a row where
      // its first terms will be, the second where its second ones will be.
      if (mine) {
        const uint16_t* q = a.q + (static_cast<int64_t>(it.q0) * a.num_q_heads + it.head0) * D + c16 * 8;
#pragma unroll 2
        for (int i = 0; i < 32 / ROWS; ++i) {
          const int rr = (warp & 3) * 32 + i * ROWS + sub, t = it.token_of(rr), tok = it.tok0 + w * shape.tile_tok + t;
          const bool there = t < shape.tile_tok && tok < it.n;
          cp_async16(q_raw(rr), q + (static_cast<int64_t>(there ? tok : 0) * a.num_q_heads + (there ? rr - t * it.heads : 0)) * D,
                     there);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        const int32_t rt = it.token_of(r), tok = it.tok0 + w * shape.tile_tok + rt;
        lim = rt < shape.tile_tok && tok < it.n ? it.len - it.n + tok + 1 : 0x7fffffff;
        lim_least = __reduce_min_sync(0xffffffffu, lim);
        // as two terms of 8 bits, in place: the lanes of a row find its largest element together, all read before any writes
        constexpr int STEPS = 32 / ROWS, AT_ONCE = 4;
#pragma unroll 1
        for (int i0 = 0; i0 < STEPS; i0 += AT_ONCE) {
          uint4 v[AT_ONCE];
#pragma unroll
          for (int i = 0; i < AT_ONCE; ++i) v[i] = *reinterpret_cast<const uint4*>(q_raw((warp & 3) * 32 + (i0 + i) * ROWS + sub));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < AT_ONCE; ++i) {
            const int rr = (warp & 3) * 32 + (i0 + i) * ROWS + sub;
            uint32_t big = __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                    __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));  // bf16 magnitudes sort as integers
#pragma unroll
            for (int o = PER_LINE / 2; o > 0; o >>= 1) big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, o));
            // (-115: 2^(11 - e2) ends at 2^126; rows that lie below keep fewer bits)
            const int e2 = max(static_cast<int>(max(big >> 16, big & 0xFFFFu) >> 7) - 127, -115);
            // the largest comes to [2^11, 2^12); a row with an infinity becomes NaN throughout, as one with a NaN does: the conversion
            // would make a number of it
            const float up = __int_as_float(e2 == 128 ? 0x7FFFFFFF : (11 - e2 + 127) << 23);
            const int of_mine = __shfl_sync(0xffffffffu, e2, lane % ROWS * PER_LINE);  // (row lane % ROWS of this step)
            if (lane / ROWS == i0 + i)
              mult = fminf(fmaxf(a.score_scale * __int_as_float((of_mine - 11 + 127) << 23), kMultLeast), kMultMost);
            const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack_bf16x2(x[e]);
              fp8_terms(pack_f16x2(f.x * up, f.y * up), hi[e], lo[e]);  // (f16 holds a scaled bf16 exactly, down to 2^-24)
            }
            uint8_t* to = q_own + c16 % 2 * 8 +
                          (D == 64 ? rr * 64 + (((c16 / 2) ^ ((rr >> 1) & 3)) << 4)
                                   : c16 / 16 * kM * 128 + rr * 128 + (((c16 / 2 & 7) ^ (rr & 7)) << 4));
            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2*>(to + Cfg::Q_TERM) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar_q_full[w]);
      }
      // ---- the output of the item before, once its last PV has completed
      if (open) {
        open = false;
        const int last_buf = TILES == 2 ? w : (kv - 1) & 1;
        const uint32_t last_use = TILES == 2 ? nt - 1 : (kv - 1) >> 1;
        if (!warp_wait_far(&bar_pv_done[last_buf], last_use & 1)) { ok = false; break; }
        tc_fence_after();
        const Item& was = *sItem(k - 1);
        if (m == kGivenUp && was_live) {
          l = __int_as_float(0x7FFFFFFF);
          page_report(a, kStatusBadExtend);
        }
        const float inv = was.whole() ? (l > 0.0f ? 1.0f / l : l) : 1.0f;  // (l: 0, or NaN)
        const int64_t slot = part_slot(place.total, sharers(place.total, a.grid, kPageFlashUnits), cta, was.first);
        const int32_t tok_w = was.tok0 + w * shape.tile_tok;
        // rows pass through the warp's 2 KB, 32 columns at a time, so that four lanes write 64 or 128 bytes of one row
        const int r0 = lane >> 2, c4 = lane & 3;
        int64_t at[4];  // where rows r0 + 8 i begin, -1: no such row
        const int64_t base = was.whole() ? (static_cast<int64_t>(was.q0 + tok_w) * a.num_q_heads + was.head0) * D
                                      : (slot * TILES + w) * kM * D;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t x = (warp & 3) * 32 + r0 + 8 * i, t = was.token_of(x);
          at[i] = t >= shape.tile_tok || tok_w + t >= was.n ? -1
                  : was.whole()                               ? base + (static_cast<int64_t>(t) * a.num_q_heads + (x - t * was.heads)) * D
                                                           : base + x * D;
        }
        if (!was.whole() && was_live)
          *reinterpret_cast<float2*>(a.part_ml + ((slot * TILES + w) * kM + r) * 2) = make_float2(m, l);
        auto put = [&](int h, uint4 x) {
          *reinterpret_cast<uint4*>(stage + lane * 64 + ((h ^ ((lane >> 1) & 3)) << 4)) = x;
        };
        auto get = [&](int i) {
          const int row = r0 + 8 * i;
          return *reinterpret_cast<const uint4*>(stage + row * 64 + ((c4 ^ ((row >> 1) & 3)) << 4));
        };
        const bool f32 = !was.whole() || a.out_dtype == KVQ_OUT_F32;
        float* const out32 = was.whole() ? static_cast<float*>(a.out) : a.part_acc;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(tO + c * 32, ov);
          if (c == D / 32 - 1) {  // the reads are ordered before the arrival that lets the next PV overwrite O
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&bar_o_free[w]);
          }
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(ov[e]) * inv;
          if (f32) {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              __syncwarp();
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const float* y = o + 16 * f + 4 * h;
                put(h, make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])));
              }
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (at[i] >= 0) *reinterpret_cast<uint4*>(out32 + at[i] + c * 32 + 16 * f + 4 * c4) = get(i);
            }
          } else {
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 4; ++h)
              put(h, make_uint4(pack_bf16x2(o[8 * h], o[8 * h + 1]), pack_bf16x2(o[8 * h + 2], o[8 * h + 3]),
                                pack_bf16x2(o[8 * h + 4], o[8 * h + 5]), pack_bf16x2(o[8 * h + 6], o[8 * h + 7])));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (at[i] >= 0) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at[i] + c * 32 + 8 * c4) = get(i);
          }
        }
        end_item(k - 1);
      }
      if (!it.live) break;
      const int32_t n = it.kt1 - it.kt0, first_key = it.kt0 * KT;
      if (!mine) {
        kv += n;
        end_item(k);
        continue;
      }
      m = kNoMax;
      l = 0.0f;
      for (int32_t j = 0; j < n; ++j, ++nt) {
        const int buf = TILES == 2 ? w : (kv + j) & 1;
        const uint32_t uses = TILES == 2 ? nt : (kv + j) >> 1;
        const uint32_t tS = tmem + buf * KT + lane_base;
        const uint32_t slot = (kv + j) % INFO;
        if (!warp_wait_far(&bar_info[slot], ((kv + j) / INFO) & 1)) { ok = false; break; }
        const Info& info = sInfo[slot];
        const int32_t t0 = first_key + j * KT;
        const bool plain = t0 + KT <= lim_least && info.full;
        float ks[PAGES], ev[PAGES];
#pragma unroll
        for (int p = 0; p < PAGES; ++p) {
          ks[p] = mult * info.ks[p];
          ev[p] = info.ev[p];
        }
        if (!warp_wait_far(&bar_s_full[buf], uses & 1)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[KT], mx[PAGES];
#pragma unroll
        for (int p = 0; p < PAGES; ++p) tmem_ld16_max_issue(tS + 16 * p, s + 16 * p, mx[p]);
#pragma unroll
        for (int p = 0; p < PAGES; ++p) tmem_wait16_max(s + 16 * p, mx[p]);
        if (!plain) {
#pragma unroll
          for (int p = 0; p < PAGES; ++p) {
            if (info.rows[p] == kPage && t0 + (p + 1) * kPage <= lim_least) continue;  // all of the page is seen
            const int32_t see = info.rows[p] > 0 ? lim - t0 - p * kPage : 0;
            float x = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              s[16 * p + e] = e < see ? s[16 * p + e] : 0xFF800000u;
              x = fmaxf(x, __uint_as_float(s[16 * p + e]));
            }
            mx[p] = __float_as_uint(x);
          }
        }
        float top = fmaf(__uint_as_float(mx[0]), ks[0], ev[0]);
#pragma unroll
        for (int p = 1; p < PAGES; ++p) top = fmaxf(top, fmaf(__uint_as_float(mx[p]), ks[p], ev[p]));
        // the reference moves when some row's largest passes it by more than 2^15; O and l are then rescaled
        const bool moved = top - m > kLimit;
        if (__any_sync(0xffffffffu, moved)) {
          const float now = moved ? (fabsf(top) > kFarScore ? kGivenUp : top - kHead) : m;
          const float alpha = moved ? ex2(m - now) : 1.0f;
          m = now;
          l *= alpha;
          if (j > 0) {
            // (one tile: the PV before may still run; two: this QK was issued after it had completed)
            if (TILES == 1 && !warp_wait_far(&bar_pv_done[(kv + j - 1) & 1], ((kv + j - 1) >> 1) & 1)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 8; ++c) {  // (8 columns at a time: the row's scores stay in registers)
              float o[8];
              tmem_ld8(tO + c * 8, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] *= alpha;
              tmem_st8(tO + c * 8, o);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < KT / 64; ++h) {
          uint32_t pw[32];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int pg = 4 * h + q;
            const float2 sc2 = make_float2(ks[pg], ks[pg]), m2 = make_float2(ev[pg] - m, ev[pg] - m);
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int i = pg * 16 + 2 * e;
              const float2 x = ffma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), sc2, m2);
              const float2 p = make_float2(ex2(x.x), ex2(x.y));
              sum = fadd2(sum, p);
              pw[q * 8 + e] = pack_f16x2(p.x, p.y);
            }
            l = fmaf(sum.x + sum.y, info.unv[pg], l);
          }
          tmem_st32(tS + h * 32, pw);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar_p_full[buf]);
      }
      if (!ok) break;
      kv += n;
      open = true;
    }
  }
  if (!ok) page_report(a, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == Cfg::MMA_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// Joins the runs of the items that several CTAs worked on.  CTA (c - 1, y): the item that CTA c went on with first, if that
// is the item's first joint; rows 8 y ... + 7, a warp for each.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) page_flash_join_kernel(const PageArgs a) {
  using Cfg = FCfg<D>;
  const Shape<D> shape(a);
  const int32_t c = blockIdx.x + 1, lane = threadIdx.x & 31;
  const int32_t row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), w = row / kM, r = row - w * kM;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  page_collect(a);
  const int64_t U = *a.total;
  const int32_t C = sharers(U, a.grid, kPageFlashUnits);
  if (c >= C || U == 0) return;
  const Item& it = static_cast<const Item*>(a.runs)[c];
  if (!it.live || first_unit(U, C, c - 1) > it.first) return;
  const int32_t rt = it.token_of(r), tok = it.tok0 + w * shape.tile_tok + rt;
  if (rt >= shape.tile_tok || tok >= it.n) return;
  const int32_t c1 = owner_of(U, C, it.first + it.all - 1);
  constexpr int V2 = D / 64;  // float2 of a lane
  float m = kNoMax, l = 0.0f;
  float2 x[V2];
#pragma unroll
  for (int k = 0; k < V2; ++k) x[k] = make_float2(0.0f, 0.0f);
#pragma unroll 4
  for (int32_t i = c - 1; i <= c1; ++i) {
    const int64_t at = (part_slot(U, C, i, it.first) * Cfg::TILES + w) * kM + r;
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
    const float now = fmaxf(m, ml.x), f = ex2(ml.x - now), keep = ex2(m - now);
    m = now;
    l = fmaf(ml.y, f, l * keep);
#pragma unroll
    for (int k = 0; k < V2; ++k) {
      const float2 y = *reinterpret_cast<const float2*>(a.part_acc + at * D + k * 64 + lane * 2);
      x[k].x = fmaf(y.x, f, x[k].x * keep);
      x[k].y = fmaf(y.y, f, x[k].y * keep);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : l;  // (0, or NaN)
  const int64_t out = (static_cast<int64_t>(it.q0 + tok) * a.num_q_heads + it.head0 + (r - rt * it.heads)) * D;
#pragma unroll
  for (int k = 0; k < V2; ++k) {
    const int64_t at = out + k * 64 + lane * 2;
    if (a.out_dtype == KVQ_OUT_F32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(x[k].x * inv, x[k].y * inv);
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) = pack_bf16x2(x[k].x * inv, x[k].y * inv);
  }
}

template <int D>
kvq_status launch_d(const PageArgs& a, cudaStream_t stream) {
  using Cfg = FCfg<D>;
  CUtensorMap map;
  if (!encode_code_map(&map, a.codes, a.num_pages, a.num_kv_heads, D)) return KVQ_ECUDA;
  auto kern = page_flash_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM) != cudaSuccess) return KVQ_ECUDA;
  kern<<<a.grid, Cfg::THREADS, Cfg::SMEM, stream>>>(a, map);
  if (cudaGetLastError() != cudaSuccess) return KVQ_ECUDA;
  if (a.grid == 1) return KVQ_OK;
  const dim3 joins(a.grid - 1, Cfg::TILES * kM / kJoinWarps);
  return launch_dependent(page_flash_join_kernel<D>, joins, kJoinWarps * 32, 0, stream, a) ? KVQ_OK : KVQ_ECUDA;
}

}  // namespace

int32_t page_flash_rows(int32_t head_dim) { return head_dim == 256 ? kM : 2 * kM; }

kvq_status launch_page_flash(const PageArgs& a, cudaStream_t stream) {
  if (a.head_dim == 64) return launch_d<64>(a, stream);
  if (a.head_dim == 128) return launch_d<128>(a, stream);
  return launch_d<256>(a, stream);
}

}  // namespace kvq
