// kvq_page_rows.cu -- attention of few query rows over a KVQ_FP8_E4M3_PAGE cache (kvq_decode, and kvq_extend's short
// turns): K = 2^ek[page] code, V = 2^ev[page] code, one exponent per page of 16 tokens and head, so that
//   y_t = log2(e) sm_scale 2^ek q.code_t + ev,   p_t = 2^(y_t - m),   out = sum p_t code_t / sum 2^-ev p_t:
// the scales meet no code (but for V's on pages far below others, codes_down).  Codes become f16 exactly, two per
// conversion; the products run on the warp-level tensor-core instructions with f16 inputs and fp32 sums.  q enters as
// f16 as well, each row scaled by a power of two (exact: bf16 has 8 significant bits; only elements 2^31 times
// smaller than the row's largest lose some).  P is rounded to f16: by 2^-11 of each, or 2^-28 of the row's largest p
// where V's scales are within 2^18 of one another (codes_down), since the reference m is 2^7 to 2^15 below the
// largest.  2 D bytes per token and kv head are read once for up to 16 query rows: bound by HBM.
//
// A tile is 8 or 16 query rows of one kv head (heads of its group, and for kvq_extend tokens times heads).  In every warp-level
// product m16n8k16 codes are A, straight from shared memory: 16 tokens of a page (scores) or 16 dims (output) are its M, and 8 of
// the tile's rows its N.  So a decode of a few heads leaves few columns empty, and the order of the dims within a product,
// which does not matter, lets a lane read 16 bytes of a token's K row at a time, and of V 16 bytes of four tokens, whose codes pair
// up by byte permutes.  Scores come out with tokens as rows; the output's products want them as columns, one movmatrix each.
// Work: a unit is a (tile, page).  All units of the call lie in one order, sequence by sequence, and every CTA takes an
// equal run of them, whatever the lengths.  The 8 warps of a CTA (4 at head_dim 256) take its pages in turn, each with its own
// ring of TMA boxes (swizzled: no bank conflicts), and join at the end of each tile's run.  A run that is all of a tile's pages
// gives the output, other runs leave partial sums, which a second kernel, its programmatic dependent, joins.
// Measured: one token each of 64 sequences over 256 to 16384 tokens, 32 heads of 128 over 8: 213 us, 5.4 of the 6.8 TB/s that a
// copy reaches (with tiles of 16 rows, half of them empty, 256 us); of 4 over 131072 tokens, 16 heads of 256 over 2: 101 us, 5.3 TB/s.
#include <cuda.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_flash.cuh"
#include "kvq_internal.h"
#include "kvq_page.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace {

// NT: the tile's query rows in groups of 8.
template <int D, int NT>
struct RCfg {
  static constexpr int ROWS = 8 * NT;                  // query rows of a tile
  static constexpr int WARPS = D == 256 ? 4 : 8;
  static constexpr int THREADS = WARPS * 32;
  // Resident per SM.  At head_dim 64 and 128 the kernels spill 16 to 124 bytes a thread for that: their caps are 64, 80
  // and 128 registers.
  static constexpr int CTAS = D == 64 ? (NT == 1 ? 4 : 3) : NT == 1 ? 3 : 2;
  static constexpr int PAGE_BYTES = kPage * D;         // codes of K or V of a page
  static constexpr int STAGE = 2 * PAGE_BYTES;
  static constexpr int STAGES = D == 64 ? (NT == 1 ? 3 : 4) : NT == 1 ? 2 : 3;
  static constexpr int SLICES = D == 256 ? 2 : 1;      // 128-byte (D = 64: 64-byte) slices of a row
  static constexpr int KSTEPS = D / 16;
  static constexpr int MT = D / 16;                    // products of 16 dims each
  static constexpr bool Q_SHARED = D == 256 && NT == 2;  // q fragments in shared memory (registers hold O)
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int JOIN = WARPS * ROWS * (D + 2) * 4;  // the warps' sums, over the ring
  static constexpr int DATA = RING > JOIN ? RING : JOIN;
  static constexpr int Q_OFF = (DATA + 127) / 128 * 128;
  static constexpr int BAR_OFF = Q_OFF + (Q_SHARED ? KSTEPS * NT * 256 : 0);
  static constexpr int SMEM = BAR_OFF + WARPS * STAGES * 8 + 1024;  // + slack to align the base
};

// A tile that a CTA went on with first, for the joining kernel.
struct Run {
  int64_t first;                         // the tile's first unit
  int32_t live, pages, q0, g, row0, rows; // its pages; sequence's first row; kv head; first row of the group's, and how many
};
static_assert(sizeof(Run) <= kPageRunMost, "run slots");

// One sequence's rows, pages and tiles.
struct Seq : PageSeq {
  int32_t pages, tiles;
  int64_t units;
};

template <int ROWS>
__device__ __forceinline__ Seq rows_sequence(const PageArgs& a, int32_t b, bool& bad) {
  Seq s;
  static_cast<PageSeq&>(s) = page_sequence(a, b, bad);
  s.pages = s.n > 0 ? (s.len + kPage - 1) / kPage : 0;
  s.tiles = (s.n * (a.num_q_heads / a.num_kv_heads) + ROWS - 1) / ROWS;
  s.units = static_cast<int64_t>(s.pages) * s.tiles * a.num_kv_heads;
  return s;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Lane (g8, t4) = (i / 4, i % 4) holds row g8 and columns 2 t4, 2 t4 + 1 of an 8 x 8 matrix of f16; of its transpose:
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D, int NT>
__global__ void __launch_bounds__(RCfg<D, NT>::THREADS, RCfg<D, NT>::CTAS)
    page_rows_kernel(const PageArgs a, const __grid_constant__ CUtensorMap map) {
  using Cfg = RCfg<D, NT>;
  constexpr int STAGES = Cfg::STAGES, SLICES = Cfg::SLICES, KSTEPS = Cfg::KSTEPS, MT = Cfg::MT;
  constexpr int kWarps = Cfg::WARPS, kThreads = Cfg::THREADS, kRows = Cfg::ROWS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint2* sQ = reinterpret_cast<uint2*>(smem + Cfg::Q_OFF);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;  // of a product: row or column g8, columns 2 t4 and 2 t4 + 1
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFF) + warp * STAGES;
  uint8_t* ring = smem + warp * STAGES * Cfg::STAGE;

  page_clear(a);
  if (lane < STAGES) mbar_init(&bars[lane], 1);
  fence_mbar_init();
  __syncwarp();
  const int32_t cta = blockIdx.x;
  bool bad = false;
  asm volatile("griddepcontrol.launch_dependents;");  // (the joining kernel waits for this one's end)
  if (a.q_start == nullptr) {  // the rows of sequences without tokens
    for (int32_t b = cta; b < a.batch; b += a.grid)
      if (__ldg(a.seq_lens + b) <= 0)
        for (int32_t i = tid; i < a.num_q_heads * (D / 4); i += kThreads)
          page_store_out(a, static_cast<int64_t>(b) * a.num_q_heads * D + i * 4, make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f);
  }
  const Place place = page_place<kWarps>(
      a.batch, cta == 0 ? a.total : nullptr, [&](int32_t i) { return rows_sequence<kRows>(a, i, bad).units; },
      [&](int64_t U) {  // this CTA's first unit
        const int32_t C = sharers(U, a.grid, kPageMinUnits);
        return cta < C && U > 0 ? first_unit(U, C, cta) : U;
      });
  if (cta == 0 && bad) page_report(a, kStatusBadExtend);
  if (place.b < 0) return;
  const int32_t C = sharers(place.total, a.grid, kPageMinUnits);
  int64_t u = first_unit(place.total, C, cta);
  const int64_t u_first = u, u_end = first_unit(place.total, C, cta + 1);
  const int32_t G = a.num_q_heads / a.num_kv_heads;
  int32_t b = place.b;
  int64_t before = place.before;
  uint32_t done = 0;  // pages that went through this warp's ring
  bool ok = true;

  while (u < u_end) {
    Seq s = rows_sequence<kRows>(a, b, bad);
    if (u >= before + s.units) {
      before += s.units;
      ++b;
      continue;
    }
    // the run: pages [pg0, pg1) of a tile
    const int64_t local = u - before;
    const int32_t tile_at = static_cast<int32_t>(local / s.pages);
    const int32_t pg0 = static_cast<int32_t>(local - static_cast<int64_t>(tile_at) * s.pages);
    const int32_t pg1 = static_cast<int32_t>(min(static_cast<int64_t>(s.pages), pg0 + (u_end - u)));
    const int32_t g = tile_at / s.tiles, tile = tile_at - g * s.tiles;
    const int32_t rows = min(kRows, s.n * G - tile * kRows);
    const int64_t tile_first = u - pg0;  // the tile's first unit
    if (tid == 0 && u == u_first)
      static_cast<Run*>(a.runs)[cta] = {tile_first, pg0 > 0, s.pages, s.q0, g, tile * kRows, rows};

    // ---- where the q of this lane's rows g8 lies, how many tokens its rows 2 t4 and 2 t4 + 1 see
    const uint16_t* qrow[NT];
    int32_t sees[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int32_t r = min(g8 + 8 * n, rows - 1) + tile * kRows, tok = r / G;
      qrow[n] = a.q + (static_cast<int64_t>(s.q0 + tok) * a.num_q_heads + g * G + (r - tok * G)) * D;
#pragma unroll
      for (int e = 0; e < 2; ++e) sees[n][e] = s.len - s.n + (min(2 * t4 + e + 8 * n, rows - 1) + tile * kRows) / G + 1;
    }
    const int32_t sees_least = s.len - s.n + tile * kRows / G + 1;

    // ---- pages: 32 at a time, one per lane, the next 32 fetched meanwhile
    const int32_t np = pg1 - pg0, nw = np > warp ? (np - warp + kWarps - 1) / kWarps : 0;
    const int32_t* table = a.block_table + static_cast<int64_t>(b) * a.max_pages + pg0 + warp;
    auto fetch = [&](int32_t batch) -> int32_t {
      const int32_t i = batch * 32 + lane;
      if (i >= nw) return -1;
      const int32_t p = __ldg(table + i * kWarps);
      if (p < a.num_pages) return p;
      page_report(a, kStatusBadPage);
      return -1;
    };
    auto scales = [&](int32_t p, float& ks, float& vs) {
      ks = vs = 1.0f;
      if (p < 0) return;
      const float* x = a.scales + static_cast<int64_t>(p) * 2 * a.num_kv_heads + g;
      ks = __ldg(x);
      vs = __ldg(x + a.num_kv_heads);
    };
    int32_t phys = fetch(0), phys_next = fetch(1);
    float ks, vs, ks_next = 1.0f, vs_next = 1.0f;
    scales(phys, ks, vs);
    auto issue = [&](int32_t i, int32_t p) {  // page i of this warp's, in slot (done + i) % STAGES
      if (lane != 0) return;
      const uint32_t slot = (done + i) % STAGES;
      if (p < 0) {
        bar_arrive(&bars[slot]);
        return;
      }
      mbar_arrive_expect_tx(&bars[slot], Cfg::STAGE);
      uint8_t* dst = ring + slot * Cfg::STAGE;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int x = 0; x < SLICES; ++x)
          tma_load_codes(smem_u32(dst + kv * Cfg::PAGE_BYTES + x * 2048), &map, x, g * kPage, kv, p, &bars[slot]);
    };
    fence_proxy_async_smem();  // (the ring held the warps' sums)
    __syncwarp();
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
      const int32_t p = __shfl_sync(0xffffffffu, phys, i);
      if (i < nw) issue(i, p);
    }

    // ---- q as f16 fragments, the row's largest element brought to [2^14, 2^15)
    float rowscale[NT][2];  // of rows 2 t4 and 2 t4 + 1
    uint32_t qf[Cfg::Q_SHARED ? 1 : KSTEPS][NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top = 0.0f;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(qrow[n] + (x * 4 + t4) * 8));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = unpack_bf16x2(w[k]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max((__float_as_int(top) >> 23) - 127, -100);  // (2^114 still brings the least bf16 to an f16)
      // (a row with an infinity becomes NaN throughout: scores of -inf alone would look like a row that sees nothing)
      const float up = __int_as_float(e == 128 ? 0x7FFFFFFF : (14 - e + 127) << 23);
      // (within 2^95, so that no page's scale makes it infinite: 0 times that would be NaN.  Scores that differ there do so by
      // 2^-33 2^95 2^-32 at least, which leaves the largest alone)
      const float back = fminf(fmaxf(a.score_scale * __int_as_float((e - 14 + 127) << 23), -0x1p95f), 0x1p95f);
#pragma unroll
      for (int c = 0; c < 2; ++c) rowscale[n][c] = __shfl_sync(0xffffffffu, back, (2 * t4 + c) * 4);
      // k-step (x, c, i): lane t4 holds dims 128 x + 32 t4 + 16 c + 4 i ... + 3 of its row (D = 64: 16 t4 + 4 i)
#pragma unroll
      for (int k = 0; k < KSTEPS; ++k) {
        const int x = k / 8, c = (k / 4) % 2, i = k % 4;
        const int d = D == 64 ? 16 * t4 + 4 * i : 128 * x + 32 * t4 + 16 * c + 4 * i;
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(qrow[n] + d));
        const float2 lo = unpack_bf16x2(v.x), hi = unpack_bf16x2(v.y);
        const uint32_t f0 = pack_f16x2(lo.x * up, lo.y * up), f1 = pack_f16x2(hi.x * up, hi.y * up);
        if constexpr (Cfg::Q_SHARED) {
          if (warp == k % kWarps) sQ[(k * NT + n) * 32 + lane] = make_uint2(f0, f1);
        } else {
          qf[k][n][0] = f0;
          qf[k][n][1] = f1;
        }
      }
    }
    if constexpr (Cfg::Q_SHARED) __syncthreads();

    float o[NT][MT][4];  // of 16 dims: dims of rows g8 and g8 + 8 of the product, query rows 2 t4 and 2 t4 + 1
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] = 0.0f;
      m[n][0] = m[n][1] = kNoMax;
      l[n][0] = l[n][1] = 0.0f;
    }
    int32_t landed = 0, ref = -127;  // ref: V's largest exponent so far

    for (int32_t i = 0; i < nw; ++i) {
      if (i > 0 && i % 32 == 0) {
        phys = phys_next;
        ks = ks_next;
        vs = vs_next;
        phys_next = fetch(i / 32 + 1);
      }
      if (i % 32 == 8) scales(phys_next, ks_next, vs_next);
      const uint32_t slot = (done + i) % STAGES;
      if (!warp_wait(&bars[slot], ((done + i) / STAGES) & 1)) { ok = false; break; }
      landed = i + 1;
      const int32_t p = __shfl_sync(0xffffffffu, phys, i & 31);
      const float kscale = __shfl_sync(0xffffffffu, ks, i & 31), vscale = __shfl_sync(0xffffffffu, vs, i & 31);
      if (p >= 0) {
        const uint8_t* kc = ring + slot * Cfg::STAGE;
        const uint8_t* vc = kc + Cfg::PAGE_BYTES;
        const int32_t t0 = (pg0 + warp + i * kWarps) * kPage;  // the page's first token
        // ---- scores of tokens g8 and g8 + 8 with rows 2 t4, 2 t4 + 1
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
        for (int q = 0; q < KSTEPS / 4; ++q) {
          uint32_t w[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = g8 + 8 * h;
            uint4 v;
            if constexpr (D == 64) {
              v = *reinterpret_cast<const uint4*>(kc + row * 64 + ((t4 ^ ((row >> 1) & 3)) << 4));
            } else {
              v = *reinterpret_cast<const uint4*>(kc + (q / 2) * 2048 + row * 128 + (((2 * t4 + q % 2) ^ (row & 7)) << 4));
            }
            w[h][0] = v.x; w[h][1] = v.y; w[h][2] = v.z; w[h][3] = v.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t f[4];
            codes_to_f16x2<KVQ_FP8_E4M3>(w[0][e], f[0], f[2]);
            codes_to_f16x2<KVQ_FP8_E4M3>(w[1][e], f[1], f[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if constexpr (Cfg::Q_SHARED) {
                const uint2 x = sQ[((q * 4 + e) * NT + n) * 32 + lane];
                mma_f16(sc[n], f, x.x, x.y);
              } else {
                mma_f16(sc[n], f, qf[q * 4 + e][n][0], qf[q * 4 + e][n][1]);
              }
            }
          }
        }
        // ---- y = score + ev in the exponent; what a row does not see is -inf
        const int32_t e2 = scale_exponent(vscale);
        ref = max(ref, e2);
        const int32_t down = codes_down(e2, ref);
        const float ev = static_cast<float>(e2 + down), unv = power_inverse(e2 + down);
        const bool whole = t0 + kPage <= sees_least;
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mult = rowscale[n][e] * kscale;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& x = sc[n][2 * h + e];
              x = fmaf(x, mult, ev);
              if (!whole && t0 + 8 * h + g8 >= sees[n][e]) x = -INFINITY;
            }
            over |= fmaxf(sc[n][e], sc[n][2 + e]) - m[n][e] > kLimit;  // (m + kLimit would be rounded where m is large)
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(sc[n][e], sc[n][2 + e]);
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              const float now = fmaxf(m[n][e], x - kHead);
              const float alpha = ex2(m[n][e] - now);
              m[n][e] = now;
              l[n][e] *= alpha;
#pragma unroll
              for (int j = 0; j < MT; ++j) {
                o[n][j][e] *= alpha;
                o[n][j][2 + e] *= alpha;
              }
            }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = ex2(sc[n][2 * h] - m[n][0]), p1 = ex2(sc[n][2 * h + 1] - m[n][1]);
            l[n][0] = fmaf(p0, unv, l[n][0]);
            l[n][1] = fmaf(p1, unv, l[n][1]);
            pf[n][h] = transposed(pack_f16x2(p0, p1));
          }
        // ---- output: dims 128 x + 16 g8 + byte (D = 64: 8 g8 + byte) of tokens 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9
        constexpr int WORDS = D == 64 ? 2 : 4;
#pragma unroll
        for (int x = 0; x < SLICES; ++x) {
          uint32_t v[4][WORDS];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 2 * t4 + (r & 1) + 8 * (r >> 1);
            if constexpr (D == 64) {
              const uint2 w = *reinterpret_cast<const uint2*>(vc + row * 64 + (((g8 >> 1) ^ ((row >> 1) & 3)) << 4) + 8 * (g8 & 1));
              v[r][0] = w.x; v[r][1] = w.y;
            } else {
              const uint4 w = *reinterpret_cast<const uint4*>(vc + x * 2048 + row * 128 + ((g8 ^ (row & 7)) << 4));
              v[r][0] = w.x; v[r][1] = w.y; v[r][2] = w.z; v[r][3] = w.w;
            }
            if (!whole && t0 + row >= s.len) {  // rows behind the last token may hold anything, NaN codes too
#pragma unroll
              for (int k = 0; k < WORDS; ++k) v[r][k] = 0u;
            }
          }
#pragma unroll
          for (int k = 0; k < WORDS; ++k)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t pick = half == 0 ? 0x5140u : 0x7362u;
              uint32_t f[4];
              codes_to_f16x2<KVQ_FP8_E4M3>(__byte_perm(v[0][k], v[1][k], pick), f[0], f[1]);
              codes_to_f16x2<KVQ_FP8_E4M3>(__byte_perm(v[2][k], v[3][k], pick), f[2], f[3]);
              if (down > 0) {
#pragma unroll
                for (int y = 0; y < 4; ++y) f[y] = mul_f16x2(f[y], f16x2_power(down));
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(o[n][(x * WORDS + k) * 2 + half], f, pf[n][0], pf[n][1]);
            }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      const int32_t j = i + STAGES;
      const int32_t pj = __shfl_sync(0xffffffffu, (j ^ i) & 32 ? phys_next : phys, j & 31);
      if (j < nw) issue(j, pj);
    }
    if (!ok) {
      page_report(a, kStatusTimeout);
      for (int32_t i = landed; i < min(nw, landed + STAGES); ++i)  // no copy may still be in flight at the end
        (void)mbar_wait_bounded(&bars[(done + i) % STAGES], ((done + i) / STAGES) & 1);
    }
    done += nw;

    // ---- the warps' sums, joined in shared memory over the ring
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
    __syncthreads();
    float2* sml = reinterpret_cast<float2*>(smem);                        // [warps][rows]
    float* sacc = reinterpret_cast<float*>(smem + kWarps * kRows * 8);    // [warps][rows][D]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * t4 + e + 8 * n;
        if (r < rows) {
          if (g8 == 0) sml[warp * kRows + r] = make_float2(m[n][e], l[n][e]);
          // the lane's dims: 128 x + 16 g8 ... + 15 (D = 64: 8 g8 ... + 7)
          constexpr int RUN = D == 64 ? 4 : 8;  // products of them
          float* dst = sacc + (warp * kRows + r) * D + g8 * 2 * RUN;
#pragma unroll
          for (int x = 0; x < SLICES; ++x)
#pragma unroll
            for (int k = 0; k < RUN; k += 2) {
              const int j = x * RUN + k;
              *reinterpret_cast<float4*>(dst + x * 128 + 2 * k) =
                  make_float4(o[n][j][e], o[n][j][2 + e], o[n][j + 1][e], o[n][j + 1][2 + e]);
            }
        }
      }
    ok = __syncthreads_and(ok);
    const bool whole_tile = pg0 == 0 && pg1 == s.pages;
    const int64_t slot = part_slot(place.total, C, cta, tile_first);
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float M = kNoMax;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w * kRows + r].x);
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = sml[w * kRows + r];
        const float f = ex2(ml.x - M);
        const float4 y = *reinterpret_cast<const float4*>(sacc + (w * kRows + r) * D + d);
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
        sum = fmaf(ml.y, f, sum);
      }
      if (whole_tile) {
        const int32_t R = tile * kRows + r, tok = R / G;
        page_store_out(a, (static_cast<int64_t>(s.q0 + tok) * a.num_q_heads + g * G + (R - tok * G)) * D + d, x,
                       sum > 0.0f ? 1.0f / sum : 0.0f);
      } else {
        *reinterpret_cast<float4*>(a.part_acc + (slot * kRows + r) * D + d) = x;
        if (d == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * kRows + r) * 2) = make_float2(M, sum);
      }
    }
    __syncthreads();
    if (!ok) break;
    u += np;
  }
}

// Joins the runs of the tiles that several CTAs worked on.  CTA (c - 1, r): row r of the tile that CTA c went on with
// first, if that is the tile's first joint; its warps share the runs.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) page_join_kernel(const PageArgs a) {
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  __shared__ __align__(16) float s_a[kJoinWarps][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t c = blockIdx.x + 1, r = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  page_collect(a);
  const int64_t U = *a.total;
  const int32_t C = sharers(U, a.grid, kPageMinUnits);
  if (c >= C || U == 0) return;
  const Run run = static_cast<const Run*>(a.runs)[c];
  if (!run.live || r >= run.rows || first_unit(U, C, c - 1) > run.first) return;
  const int32_t c1 = owner_of(U, C, run.first + run.pages - 1);
  constexpr int V4 = D / 128 > 0 ? D / 128 : 1;  // float4 of a lane (D = 64: of half the lanes)
  float m = kNoMax, l = 0.0f;
  float4 x[V4];
#pragma unroll
  for (int k = 0; k < V4; ++k) x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int32_t i = c - 1 + warp; i <= c1; i += kJoinWarps) {
    const int64_t at = part_slot(U, C, i, run.first) * a.tile + r;
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
    const float now = fmaxf(m, ml.x), f = ex2(ml.x - now), keep = ex2(m - now);
    m = now;
    l = fmaf(ml.y, f, l * keep);
#pragma unroll
    for (int k = 0; k < V4; ++k) {
      if (D == 64 && lane >= 16) continue;
      const float4 y = *reinterpret_cast<const float4*>(a.part_acc + at * D + k * 128 + lane * 4);
      x[k].x = fmaf(y.x, f, x[k].x * keep);
      x[k].y = fmaf(y.y, f, x[k].y * keep);
      x[k].z = fmaf(y.z, f, x[k].z * keep);
      x[k].w = fmaf(y.w, f, x[k].w * keep);
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int k = 0; k < V4; ++k)
    if (D != 64 || lane < 16) *reinterpret_cast<float4*>(&s_a[warp][k * 128 + lane * 4]) = x[k];
  __syncthreads();
  const int32_t G = a.num_q_heads / a.num_kv_heads, R = run.row0 + r, tok = R / G;
  const int64_t out = (static_cast<int64_t>(run.q0 + tok) * a.num_q_heads + run.g * G + (R - tok * G)) * D;
  if (tid < D / 4) {
    const int d = tid * 4;
    float M = kNoMax, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_m[w]);
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = ex2(s_m[w] - M);
      const float4 v = *reinterpret_cast<const float4*>(&s_a[w][d]);
      sum = fmaf(s_l[w], f, sum);
      y.x = fmaf(v.x, f, y.x);
      y.y = fmaf(v.y, f, y.y);
      y.z = fmaf(v.z, f, y.z);
      y.w = fmaf(v.w, f, y.w);
    }
    page_store_out(a, out + d, y, sum > 0.0f ? 1.0f / sum : 0.0f);
  }
}

template <int D, int NT>
kvq_status launch_d(const PageArgs& a, cudaStream_t stream) {
  using Cfg = RCfg<D, NT>;
  CUtensorMap map;
  if (!encode_code_map(&map, a.codes, a.num_pages, a.num_kv_heads, D)) return KVQ_ECUDA;
  auto kern = page_rows_kernel<D, NT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM) != cudaSuccess) return KVQ_ECUDA;
  kern<<<a.grid, Cfg::THREADS, Cfg::SMEM, stream>>>(a, map);
  if (cudaGetLastError() != cudaSuccess) return KVQ_ECUDA;
  if (a.grid == 1) return KVQ_OK;
  const int64_t rows = static_cast<int64_t>(a.total_q) * (a.num_q_heads / a.num_kv_heads);
  const dim3 joins(a.grid - 1, std::min<int64_t>(a.tile, rows));
  return launch_dependent(page_join_kernel<D>, joins, kJoinWarps * 32, 0, stream, a) ? KVQ_OK : KVQ_ECUDA;
}

}  // namespace

bool page_supported(int32_t head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }

int32_t page_rows_grid(int32_t head_dim, int32_t tile, int32_t sms) {
  const bool one = tile == 8;
  return sms * (head_dim == 64    ? (one ? RCfg<64, 1>::CTAS : RCfg<64, 2>::CTAS)
                : head_dim == 128 ? (one ? RCfg<128, 1>::CTAS : RCfg<128, 2>::CTAS)
                                  : (one ? RCfg<256, 1>::CTAS : RCfg<256, 2>::CTAS));
}

kvq_status launch_page_rows(const PageArgs& a, cudaStream_t stream) {
  const bool one = a.tile == 8;
  if (a.head_dim == 64) return one ? launch_d<64, 1>(a, stream) : launch_d<64, 2>(a, stream);
  if (a.head_dim == 128) return one ? launch_d<128, 1>(a, stream) : launch_d<128, 2>(a, stream);
  return one ? launch_d<256, 1>(a, stream) : launch_d<256, 2>(a, stream);
}

}  // namespace kvq
