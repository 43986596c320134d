// kvq_append.cu -- appends a step's keys and values to the paged cache, rotated to their positions on the way, and
// rotates its queries.
//
// Of token t of sequence b at place p = seq_lens[b] - n_b + (t - q_start[b]), with the angles of its position P:
//   x'[i] = x[i] cos_P,i - x[j] sin_P,i,  x'[j] = x[j] cos_P,i + x[i] sin_P,i,   (i, j) the rotation's pairs,
// in fp32 with each product and sum rounded by itself; queries leave as bf16, keys (and values, as they came) are
// quantized from fp32: no bf16 in between, whose rounding would be one more.  Bound by HBM: 2 B per element in, 2 B per
// query element or 1 B per key or value element (and its scales) out.
//
// append_rows_kernel: queries, and the keys and values of the kinds whose scale belongs to one row.  A thread owns 8
// elements of a row (16 bytes), four lanes a block of 32, and its partners' elements come from their lane where a row lies in
// one warp (head_dim 64, 128, 256; otherwise from a second load).  A CTA takes up to 8 tokens, and finds their places, pages
// and angles once, into shared memory, while its first rows are on their way; 3 or 4 rows a thread are in flight.  With
// one row in flight and one token a CTA, four prompts of 400 to 2048 tokens with 128 heads of 576 (64 of them rotated) and
// their latent rows took 666 us, eight turns of 500 to 4096 tokens with 32 + 2 x 8 heads of 128 197 us; now 374 us (5.1 of
// the 6.8 TB/s that a copy reaches) and 114 us (4.0 TB/s, with the pages below).  The arithmetic between loads bounds it:
// with one value at a time in place of two (mul2, add2) these took 381 and 117 us.  Rows of 576 leave 40 of a CTA's 256 threads idle.
// Further from the floor where a token has few rows: 18400 tokens with 32 + 2 x 8 heads of 128 take 119 us in KVQ_FP8_E4M3 and
// 100 us in KVQ_FP8_E4M3_UNSCALED against 61 us, their keys and values alone 62 and 41 us against 17 us (kvq_store: 0.87 of the
// rate).  A token is then one pass, and at most 8 of them stand behind a CTA's search for sequences, pages and angles.
// append_pages_kernel: KVQ_FP8_E4M3_PAGE.  A warp owns one (page, K or V, head): its scale is a power of two that only
// grows, s = 2^e with the least e that lets every row stored since the page was opened fit (|x| <= 448 s), so a page that outgrows
// its scale has its older codes multiplied by 2^(e_old - e_new): exact but for values that fall below E4M3's normal
// range.  The page's new rows are read once, all loads in flight together, and stay in registers as they came; they are
// turned twice, for the maximum and for the codes (kept turned they would take twice the registers).  18400 tokens x 2 x 8
// heads of 128: 47 us, read twice from memory 58 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 8;  // tokens of a CTA at most

// Whether sequence b's numbers agree; q0, n and len are its first row, new tokens and stored tokens.
__device__ __forceinline__ bool append_sequence(const AppendArgs& a, int32_t b, int32_t& q0, int32_t& n, int32_t& len) {
  q0 = __ldg(a.q_start + b);
  const int64_t q1 = __ldg(a.q_start + b + 1);
  len = __ldg(a.seq_lens + b);
  n = static_cast<int32_t>(q1 - q0);
  return q0 >= 0 && q1 >= q0 && q1 <= a.total && n <= len && len <= static_cast<int64_t>(a.max_pages) * a.page_size;
}

// The call's first CTA reads all that the call's numbers can get wrong and writes the status word; the others only skip or
// clamp what it finds.  With reports from all CTAs the word would have to be cleared by a launch of its own, 2 us of a small call.
__device__ __forceinline__ void append_check(const AppendArgs& a) {
  __shared__ uint32_t s_code;
  if (threadIdx.x == 0) s_code = 0;
  __syncthreads();
  constexpr int kAlone = 32;  // tokens that a thread looks through by itself; a warp shares those of longer sequences
  const int lane = threadIdx.x & 31;
  uint32_t code = 0;
  auto look = [&](int32_t b, int32_t q0, int32_t n, int32_t len, int32_t from, int32_t step) {
    const int32_t first = (len - n) / a.page_size, last = (len - 1) / a.page_size;
    for (int32_t i = first + from; i <= last; i += step)
      if (__ldg(a.block_table + static_cast<int64_t>(b) * a.max_pages + i) >= a.num_pages) code = max(code, kStatusBadPage);
    if (a.rot_dim > 0 && a.positions != nullptr)
      for (int32_t i = from; i < n; i += step)
        if (static_cast<uint32_t>(__ldg(a.positions + q0 + i)) >= static_cast<uint32_t>(a.max_position))
          code = max(code, kStatusBadExtend);
    if (a.rot_dim > 0 && a.positions == nullptr && len > a.max_position) code = max(code, kStatusBadExtend);
  };
  for (int32_t b0 = threadIdx.x - lane; b0 < a.batch; b0 += kThreads) {
    int32_t q0 = 0, n = 0, len = 0;
    if (b0 + lane < a.batch && !append_sequence(a, b0 + lane, q0, n, len)) {
      code = max(code, kStatusBadExtend);
      n = 0;
    }
    if (n > 0 && n <= kAlone) look(b0 + lane, q0, n, len, 0, 1);
    for (uint32_t more = __ballot_sync(0xffffffffu, n > kAlone); more != 0; more &= more - 1) {
      const int from = __ffs(more) - 1;
      look(b0 + from, __shfl_sync(0xffffffffu, q0, from), __shfl_sync(0xffffffffu, n, from),
           __shfl_sync(0xffffffffu, len, from), lane, 32);
    }
  }
  if (code != 0) atomicMax(&s_code, code);
  __syncthreads();
  if (threadIdx.x == 0) *a.status = s_code;
}

// The first consistent sequence for which `mine` holds, or batch: by the whole CTA.
template <typename F>
__device__ __forceinline__ int32_t append_find(const AppendArgs& a, F mine) {
  __shared__ int32_t s_found;
  if (threadIdx.x == 0) s_found = a.batch;
  __syncthreads();
  for (int32_t b = threadIdx.x; b < a.batch; b += kThreads) {
    int32_t q0, n, len;
    if (append_sequence(a, b, q0, n, len) && mine(b, q0, n, len)) atomicMin(&s_found, b);
  }
  __syncthreads();
  return s_found;
}

// The page of block-table entry (b, i), or -1.
__device__ __forceinline__ int32_t append_page(const AppendArgs& a, int32_t b, int32_t i) {
  const int32_t page = __ldg(a.block_table + static_cast<int64_t>(b) * a.max_pages + i);
  return page < a.num_pages ? page : -1;
}

// The position to which row t, at place p of its sequence, is rotated.
__device__ __forceinline__ int32_t append_position(const AppendArgs& a, int32_t t, int32_t p) {
  if (a.rot_dim == 0) return 0;
  const int32_t at = a.positions ? __ldg(a.positions + t) : p;
  return min(max(at, 0), a.max_position - 1);
}

__device__ __forceinline__ void bf16x8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Products of two values, each rounded by itself, and their sums.  A packed product and sum would be contracted into one
// rounding, also with .rn: the product is a fused one with -0, which the compiler does not know to be that (minus_zero).
__device__ __forceinline__ float2 mul2(float2 a, float2 b, float minus_zero) {
  return ffma2(a, b, make_float2(minus_zero, minus_zero));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Angles of a token in shared memory, rot_dim floats in quads.  Halves that pair: a thread takes two neighbouring quads of
// the cosines and of the sines, so the even ones come first, which lets eight neighbouring threads read 128 bytes in a row.
__device__ __forceinline__ int32_t quad_place(const AppendArgs& a, int32_t quad) {
  return a.interleaved ? quad : (quad & 1) * (a.rot_dim / 8) + (quad >> 1);
}

// Where a thread's 8 elements from `e` on lie in the rotation, and their cos and sin (of 4 pairs when neighbours pair).
struct Turn {
  int32_t partner;  // elements from here to the partners'; 0: neighbours pair, or no rotation
  bool on, low;     // low: the first of each pair
  float c[8], s[8];
  __device__ __forceinline__ void place(const AppendArgs& a, int32_t e) {
    const int32_t j = e - a.rot_offset, half = a.rot_dim / 2;
    on = j >= 0 && j < a.rot_dim;
    low = j < half;
    partner = !on || a.interleaved ? 0 : low ? half : -half;
  }
  __device__ __forceinline__ void angles(const AppendArgs& a, const float* row, int32_t e) {
    if (!on) return;
    const float4* p = reinterpret_cast<const float4*>(row);
    const int32_t half = a.rot_dim / 2, j = e - a.rot_offset;
    if (a.interleaved) {
      four(p[j / 8], c);
      four(p[j / 8 + half / 4], s);
    } else {
      const int32_t q = (low ? j : j - half) / 8, odd = a.rot_dim / 8;  // quads 2 q and 2 q + 1, then half / 4 further
      four(p[q], c);
      four(p[q + odd], c + 4);
      four(p[q + half / 8], s);
      four(p[q + half / 8 + odd], s + 4);
    }
  }
  __device__ __forceinline__ static void four(float4 v, float* x) {
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  // x: the thread's elements, y: their partners
  __device__ __forceinline__ void apply(float (&x)[8], const float (&y)[8], float minus_zero) const {
    if (!on) return;
    // two at a time; a difference as the sum with the negative product
    if (partner == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 z = add2(mul2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(c[i], c[i]), minus_zero),
                              mul2(make_float2(x[2 * i + 1], x[2 * i]), make_float2(-s[i], s[i]), minus_zero));
        x[2 * i] = z.x;
        x[2 * i + 1] = z.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 q = mul2(make_float2(y[i], y[i + 1]), make_float2(s[i], s[i + 1]), minus_zero);
        const float2 z = add2(mul2(make_float2(x[i], x[i + 1]), make_float2(c[i], c[i + 1]), minus_zero),
                              low ? make_float2(-q.x, -q.y) : q);
        x[i] = z.x;
        x[i + 1] = z.y;
      }
    }
  }
};

__device__ __forceinline__ float amax8(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  return m;
}

// E4M3 or E5M2 codes of 8 values: one rounding to nearest-even that saturates.
template <__nv_fp8_interpretation_t T>
__device__ __forceinline__ uint2 fp8x8(const float (&y)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]), __NV_SATFINITE, T);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]), __NV_SATFINITE, T);
    w[i] = lo | hi << 16;
  }
  return make_uint2(w[0], w[1]);
}

// Codes of 8 elements of a block of 32 that four neighbouring lanes hold; scale: its fp16 scale.
template <int KIND>
__device__ __forceinline__ uint2 block_codes(float (&x)[8], __half& scale) {
  if constexpr (KIND == KVQ_FP8_E4M3_UNSCALED) return fp8x8<__NV_E4M3>(x);
  if constexpr (KIND == KVQ_FP8_E5M2_UNSCALED) return fp8x8<__NV_E5M2>(x);
  float m = amax8(x);
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  scale = block_scale<KIND>(m);
  const float s = __half2float(scale);
  if (s == 0.0f) return make_uint2(0u, 0u);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], s);
  if constexpr (KIND == KVQ_Q8_0) {
    int32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = q8_trunc_code(x[i]);
    return make_uint2(pack_q8x4(q[0], q[1], q[2], q[3]), pack_q8x4(q[4], q[5], q[6], q[7]));
  } else {
    return fp8x8<__NV_E4M3>(x);
  }
}

// What a CTA finds out about its tokens before it turns their rows.
struct Tokens {
  int32_t seq[kTokens], page[kTokens], off[kTokens], angle[kTokens];
};

// The rows of tokens t0 ... (nt of them): the CTA takes as many rows at once as its threads hold, passes of queries' heads
// first, then (KIND != KVQ_FP8_E4M3_PAGE) of the keys' and the values', every row_chunks-th pass of a token from `chunk`
// on.  All threads of the CTA call it; thread i of a row's D / 8 takes its elements 8 i ...  SHFL: a row's threads lie in one
// warp, and a thread gets its partners' elements from there.  `turns`: shared memory for the tokens' angles.
template <int KIND, bool SHFL>
__device__ __forceinline__ void append_rows(const AppendArgs& a, int32_t t0, int32_t nt, int32_t chunk, Tokens& tok,
                                            float* turns) {
  constexpr bool kQuant = KIND != KVQ_FP8_E4M3_PAGE;
  constexpr int U = SHFL ? 4 : 3;  // passes whose loads are in flight together
  const int32_t per_row = a.head_dim / 8, lanes = kThreads / per_row;
  const int32_t i = threadIdx.x % per_row, slot = threadIdx.x / per_row, e = i * 8;
  const int32_t kv_rows = kQuant ? a.n_kv * a.num_kv_heads : 0;
  const int32_t q_passes = (a.num_q_heads + lanes - 1) / lanes, passes = q_passes + (kv_rows + lanes - 1) / lanes;
  Turn turn;
  turn.place(a, e);
  uint4 raw[U], other[SHFL ? 1 : U];
  struct Cursor {
    int32_t k, p;  // token, pass
    __device__ __forceinline__ void next(int32_t chunk, int32_t by, int32_t passes) {
      p += by;
      if (p >= passes) {
        p = chunk;
        ++k;
      }
    }
  };
  auto load = [&](Cursor c) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (!SHFL) other[u] = raw[u];
      if (c.k < nt) {
        const int64_t t = t0 + c.k;
        const uint16_t* row = nullptr;
        bool turns_too = true;
        if (c.p < q_passes) {
          const int32_t h = c.p * lanes + slot;
          if (h < a.num_q_heads) row = a.q + t * a.q_token + h * a.q_head;
        } else if (kQuant) {
          const int32_t r = (c.p - q_passes) * lanes + slot;
          turns_too = r < a.num_kv_heads;
          if (r < kv_rows)
            row = turns_too ? a.k + t * a.k_token + r * a.k_head : a.v + t * a.v_token + (r - a.num_kv_heads) * a.v_head;
        }
        if (row != nullptr && slot < lanes) {
          // (plain loads: the queries may be turned where they lie, and these stay before the barrier below)
          raw[u] = *reinterpret_cast<const uint4*>(row + e);
          if constexpr (!SHFL)
            if (turns_too && turn.partner != 0) other[u] = *reinterpret_cast<const uint4*>(row + e + turn.partner);
        }
      }
      c.next(chunk, a.row_chunks, passes);
    }
  };
  Cursor at = {0, chunk};
  load(at);
  // ---- meanwhile: the tokens' sequences, pages and angles
  if (threadIdx.x < kTokens) tok.seq[threadIdx.x] = a.batch;
  __syncthreads();
  for (int32_t b = threadIdx.x; b < a.batch; b += kThreads) {
    int32_t q0, n, len;
    if (!append_sequence(a, b, q0, n, len)) continue;
    for (int32_t k = max(q0 - t0, 0); k < min(q0 + n - t0, nt); ++k) atomicMin(&tok.seq[k], b);
  }
  __syncthreads();
  if (threadIdx.x < nt) {
    const int32_t k = threadIdx.x, b = tok.seq[k];
    if (b < a.batch) {
      int32_t q0, n, len;
      append_sequence(a, b, q0, n, len);
      const int32_t place = len - n + (t0 + k - q0);
      tok.angle[k] = append_position(a, t0 + k, place);
      if (kQuant) {
        tok.page[k] = append_page(a, b, place / a.page_size);
        tok.off[k] = place % a.page_size;
      }
    }
  }
  __syncthreads();
  const int32_t quads = a.rot_dim / 4;
  for (int32_t x = threadIdx.x; x < nt * quads; x += kThreads) {
    const int32_t k = x / quads;
    if (tok.seq[k] < a.batch)
      reinterpret_cast<float4*>(turns)[k * quads + quad_place(a, x - k * quads)] =
          __ldg(reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(tok.angle[k]) * a.rot_dim) + (x - k * quads));
  }
  __syncthreads();
  // ---- the rows
  auto turned = [&](int u, int32_t k, float (&x)[8]) {
    if (turn.on) {
      float y[8];
      if constexpr (SHFL) bf16x8(raw[u], y);  // (exchanged below)
      else bf16x8(other[u], y);
      turn.angles(a, turns + k * a.rot_dim, e);
      turn.apply(x, y, a.minus_zero);
    }
  };
  while (at.k < nt) {
    if (!SHFL && a.q_out == a.q) __syncthreads();  // (a thread's partners have been read before they are overwritten)
    Cursor c = at;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c.k >= nt) break;  // (the same for the whole CTA)
      const bool known = tok.seq[c.k] < a.batch;
      float x[8];
      bf16x8(raw[u], x);
      const uint4 own = raw[u];
      if constexpr (SHFL) {
        if (a.rot_dim > 0) {
          const int from = (threadIdx.x & 31) + turn.partner / 8;
          raw[u] = make_uint4(__shfl_sync(0xffffffffu, own.x, from), __shfl_sync(0xffffffffu, own.y, from),
                              __shfl_sync(0xffffffffu, own.z, from), __shfl_sync(0xffffffffu, own.w, from));
        }
      }
      if (c.p < q_passes) {
        const int32_t h = c.p * lanes + slot;
        turned(u, c.k, x);
        if (known && slot < lanes && h < a.num_q_heads) {
          const uint4 o = turn.on ? make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                               pack_bf16x2(x[6], x[7]))
                                  : own;
          *reinterpret_cast<uint4*>(a.q_out + static_cast<int64_t>(t0 + c.k) * a.out_token + h * a.out_head + e) = o;
        }
      } else if constexpr (kQuant) {
        const int32_t r = (c.p - q_passes) * lanes + slot;
        if (r < a.num_kv_heads) turned(u, c.k, x);
        __half scale;
        const uint2 code = block_codes<KIND>(x, scale);
        if (known && slot < lanes && r < kv_rows && tok.page[c.k] >= 0) {
          const int32_t kv = r < a.num_kv_heads ? 0 : 1;
          const int64_t row = ((static_cast<int64_t>(tok.page[c.k]) * a.n_kv + kv) * a.num_kv_heads + r - kv * a.num_kv_heads) *
                                  a.page_size + tok.off[c.k];
          *reinterpret_cast<uint2*>(a.codes + row * a.head_dim + e) = code;
          if (KindTraits<KIND>::kScaled && i % 4 == 0)
            static_cast<__half*>(a.scales)[row * (a.head_dim / kBlock) + i / 4] = scale;
        }
      }
      c.next(chunk, a.row_chunks, passes);
    }
    at = c;
    if (at.k < nt) load(at);
  }
}

// grid: the check, then (tokens, row chunk), row chunks fastest
template <int KIND, bool SHFL>
__global__ void __launch_bounds__(kThreads, 4) append_rows_kernel(const AppendArgs a) {
  extern __shared__ __align__(16) float turns[];
  __shared__ Tokens tok;
  if (blockIdx.x == 0) return append_check(a);
  const int32_t at = blockIdx.x - 1, t = at / a.row_chunks * a.tokens;
  append_rows<KIND, SHFL>(a, t, min(a.tokens, a.total - t), at % a.row_chunks, tok, turns);
}

// The least e with m <= 448 * 2^e (448 = 1.75 * 2^8), within the exponents that a page's scale may have.
__device__ __forceinline__ int32_t page_exponent(float m) {
  const int32_t bits = __float_as_int(m);
  const int32_t e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000 ? 1 : 0);
  return min(max(e, kPageScaleMin), kPageScaleMax);
}

__device__ __forceinline__ float power_of_two(int32_t e) { return __int_as_float((e + 127) << 23); }

// Pages before sequence b in the order of the grid: at least as many as b's predecessors touch, from q_start alone (n
// tokens touch at most (n + 14) / 16 + 1 pages, and floors only grow with the sum).
__device__ __forceinline__ int64_t pages_before(int32_t b, int32_t q0) {
  return (static_cast<int64_t>(q0) + 14LL * b) / kPage + b;
}

// grid: the check, (page, chunk of its 2 * heads parts), then (tokens, row chunk) of the queries
template <int D>
__global__ void __launch_bounds__(kThreads, D == 256 ? 2 : 3) append_pages_kernel(const AppendArgs a) {
  constexpr int PER_ROW = D / 8;               // threads of a row
  constexpr int ROWS = 32 / PER_ROW;           // rows of a pass
  constexpr int PASSES = kPage / ROWS;
  extern __shared__ __align__(16) float turns[];
  __shared__ Tokens tok;
  if (blockIdx.x == 0) return append_check(a);
  const int32_t at = blockIdx.x - 1;
  if (at >= a.page_ctas) {
    const int32_t q = static_cast<int32_t>(at - a.page_ctas), t = q / a.row_chunks * a.tokens;
    append_rows<KVQ_FP8_E4M3_PAGE, true>(a, t, min(a.tokens, a.total - t), q % a.row_chunks, tok, turns);
    return;
  }
  const int32_t item = at / a.part_chunks, chunk = at % a.part_chunks;
  // the sequence among whose pages the item lies, and which of them
  const int32_t b = append_find(a, [&](int32_t s, int32_t q0, int32_t n, int32_t len) {
    if (n == 0) return false;
    const int64_t j = item - pages_before(s, q0);
    return j >= 0 && j <= (len - 1) / kPage - (len - n) / kPage;
  });
  if (b >= a.batch) return;
  int32_t q0, n, len;
  append_sequence(a, b, q0, n, len);
  const int32_t j = static_cast<int32_t>(item - pages_before(b, q0)) + (len - n) / kPage;
  const int32_t page = append_page(a, b, j);
  if (page < 0) return;
  const int32_t lo = max(len - n - j * kPage, 0), hi = min(len - j * kPage, kPage);  // new rows of the page
  const int32_t t0 = q0 + j * kPage - (len - n);                                     // row r of it is the call's row t0 + r
  const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t part = chunk * kWarps + warp, parts = 2 * a.num_kv_heads;
  const int32_t kv = part / a.num_kv_heads, h = part - kv * a.num_kv_heads;
  const int32_t e = lane % PER_ROW * 8, sub = lane / PER_ROW;
  // ---- the new rows, all loads at once
  uint4 raw[PASSES];
#pragma unroll
  for (int x = 0; x < PASSES; ++x) {
    const int32_t r = x * ROWS + sub;
    const int64_t t = t0 + r;
    raw[x] = make_uint4(0u, 0u, 0u, 0u);
    if (part < parts && r >= lo && r < hi)
      raw[x] = __ldg(reinterpret_cast<const uint4*>(
          (kv == 0 ? a.k + t * a.k_token + h * a.k_head : a.v + t * a.v_token + h * a.v_head) + e));
  }
  // ---- meanwhile their angles
  if (a.rot_dim > 0 && chunk * kWarps < a.num_kv_heads) {
    const int32_t quads = a.rot_dim / 4;
    for (int32_t x = threadIdx.x; x < kPage * quads; x += kThreads) {
      const int32_t r = x / quads;
      if (r >= lo && r < hi)
        reinterpret_cast<float4*>(turns)[r * quads + quad_place(a, x - r * quads)] = __ldg(
            reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(append_position(a, t0 + r, j * kPage + r)) * a.rot_dim) +
            (x - r * quads));
    }
    __syncthreads();
  }
  if (part >= parts) return;
  const int64_t row0 = (static_cast<int64_t>(page) * 2 + kv) * a.num_kv_heads + h;
  uint8_t* codes = a.codes + row0 * kPage * D + e;
  float* scale = static_cast<float*>(a.scales) + row0;

  Turn turn;
  turn.place(a, e);
  const bool turns_too = kv == 0 && a.rot_dim > 0;  // (the same for the whole warp)
  auto value = [&](int pass, float (&x)[8]) {  // the thread's elements of row pass * ROWS + sub
    const uint4 own = raw[pass];
    bf16x8(own, x);
    if (turns_too) {
      const int from = lane + turn.partner / 8;
      const uint4 other = make_uint4(__shfl_sync(0xffffffffu, own.x, from), __shfl_sync(0xffffffffu, own.y, from),
                                     __shfl_sync(0xffffffffu, own.z, from), __shfl_sync(0xffffffffu, own.w, from));
      const int32_t r = pass * ROWS + sub;
      if (turn.on && r >= lo && r < hi) {
        float y[8];
        bf16x8(other, y);
        turn.angles(a, turns + r * a.rot_dim, e);
        turn.apply(x, y, a.minus_zero);
      }
    }
  };
  const float had = lo > 0 ? *scale : 0.0f;
  float m = 0.0f;
#pragma unroll
  for (int x = 0; x < PASSES; ++x) {
    if (x * ROWS + ROWS <= lo || x * ROWS >= hi) continue;  // (the same for the whole warp)
    float y[8];
    value(x, y);
    m = fmaxf(m, amax8(y));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  int32_t exp = page_exponent(m);
  if (lo > 0) {
    const int32_t old = min(max(((__float_as_int(had) >> 23) & 255) - 127, kPageScaleMin), kPageScaleMax);
    if (exp > old) {
      const float f = power_of_two(old - exp);
      for (int32_t r = sub; r < lo; r += ROWS) {
        const uint2 c = *reinterpret_cast<const uint2*>(codes + r * D);
        uint32_t w[4];
        codes_to_f16x2<KVQ_FP8_E4M3>(c.x, w[0], w[1]);
        codes_to_f16x2<KVQ_FP8_E4M3>(c.y, w[2], w[3]);
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = half_bits_to_float(lo16(w[i])) * f;
          x[2 * i + 1] = half_bits_to_float(hi16(w[i])) * f;
        }
        *reinterpret_cast<uint2*>(codes + r * D) = fp8x8<__NV_E4M3>(x);
      }
    }
    exp = max(exp, old);
  }
  const float inv = power_of_two(-exp);
#pragma unroll
  for (int x = 0; x < PASSES; ++x) {
    const int32_t r = x * ROWS + sub;
    if (x * ROWS + ROWS <= lo || x * ROWS >= hi) continue;
    asm volatile("" : "+r"(raw[x].x), "+r"(raw[x].y), "+r"(raw[x].z), "+r"(raw[x].w));  // (turned again: registers are scarcer)
    float y[8];
    value(x, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= inv;
    if (r >= lo && r < hi) *reinterpret_cast<uint2*>(codes + r * D) = fp8x8<__NV_E4M3>(y);
  }
  if (lane == 0) *scale = power_of_two(exp);
}

template <typename Kernel>
kvq_status launch(Kernel kern, const AppendArgs& a, int64_t grid, cudaStream_t stream) {
  const size_t smem = std::max(a.tokens, a.page_ctas > 0 ? kPage : 0) * a.rot_dim * sizeof(float);
  kern<<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

}  // namespace

bool append_supported(int32_t head_dim, kvq_kind kind) {
  if (kind == KVQ_FP8_E4M3_PAGE) return head_dim == 64 || head_dim == 128 || head_dim == 256;
  return head_dim / 8 <= kThreads;
}

int64_t append_grid(AppendArgs* a, int32_t sms) {
  const int32_t lanes = kThreads / (a->head_dim / 8);
  const bool pages = a->kind == KVQ_FP8_E4M3_PAGE;
  const int32_t kv_rows = pages ? 0 : a->n_kv * a->num_kv_heads, rows = a->num_q_heads + kv_rows;
  const int32_t passes = (a->num_q_heads + lanes - 1) / lanes + (kv_rows + lanes - 1) / lanes;
  // a token's rows are spread over CTAs while these would not fill the GPU
  a->row_chunks = static_cast<int32_t>(
      std::max<int64_t>(1, std::min<int64_t>(passes, 4LL * sms / std::max(1, a->total))));
  // ... and several tokens are one CTA's when there are many, which then looks for their sequences but once
  const int64_t room = a->rot_dim > 0 ? std::max(1, 16384 / (a->rot_dim * 4)) : kTokens;  // angles in shared memory
  a->tokens = static_cast<int32_t>(
      std::max<int64_t>(1, std::min<int64_t>({kTokens, room, a->total / (8LL * sms), 64 / std::max(passes, 1)})));
  a->part_chunks = (2 * a->num_kv_heads + kWarps - 1) / kWarps;
  const int64_t items = pages ? (static_cast<int64_t>(a->total) + 14LL * a->batch) / kPage + a->batch : 0;
  a->page_ctas = items * a->part_chunks;
  return 1 + a->page_ctas + (rows > 0 ? (static_cast<int64_t>(a->total) + a->tokens - 1) / a->tokens * a->row_chunks : 0);
}

kvq_status launch_append(const AppendArgs& a, int64_t grid, cudaStream_t stream) {
  const bool shfl = a.head_dim == 64 || a.head_dim == 128 || a.head_dim == 256;  // rows lie in one warp
  switch (a.kind) {
#define KVQ_APPEND_ROWS(K) \
  case K: return shfl ? launch(append_rows_kernel<K, true>, a, grid, stream) : launch(append_rows_kernel<K, false>, a, grid, stream);
    KVQ_APPEND_ROWS(KVQ_FP8_E4M3)
    KVQ_APPEND_ROWS(KVQ_Q8_0)
    KVQ_APPEND_ROWS(KVQ_FP8_E4M3_UNSCALED)
    KVQ_APPEND_ROWS(KVQ_FP8_E5M2_UNSCALED)
#undef KVQ_APPEND_ROWS
    case KVQ_FP8_E4M3_PAGE:
      if (a.head_dim == 64) return launch(append_pages_kernel<64>, a, grid, stream);
      if (a.head_dim == 128) return launch(append_pages_kernel<128>, a, grid, stream);
      return launch(append_pages_kernel<256>, a, grid, stream);
  }
  return KVQ_EKIND;
}

}  // namespace kvq
