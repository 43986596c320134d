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
// elements of a row (16 bytes), four lanes a block of 32; a CTA takes a token, so that its place, page and angles are
// found once, and walks its rows.
// append_pages_kernel: KVQ_FP8_E4M3_PAGE.  A warp owns one (page, K or V, head): its scale is a power of two that only
// grows, s = 2^e with the least e that lets every row stored since the page was opened fit (|x| <= 448 s), so a page that outgrows
// its scale has its older codes multiplied by 2^(e_old - e_new): exact but for values that fall below E4M3's normal
// range.  The rows are read twice, for the maximum and for the codes, the second time from L1.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void append_report(const AppendArgs& a, uint32_t code) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the clearing kernel before this one has completed
  set_status(a.status, code);
}

// Whether sequence b's numbers agree; q0, n and len are its first row, new tokens and stored tokens.
__device__ __forceinline__ bool append_sequence(const AppendArgs& a, int32_t b, int32_t& q0, int32_t& n, int32_t& len) {
  q0 = __ldg(a.q_start + b);
  const int64_t q1 = __ldg(a.q_start + b + 1);
  len = __ldg(a.seq_lens + b);
  n = static_cast<int32_t>(q1 - q0);
  return q0 >= 0 && q1 >= q0 && q1 <= a.total && n <= len && len <= static_cast<int64_t>(a.max_pages) * a.page_size;
}

// One CTA of the call reports inconsistent sequences; all of them skip these.
__device__ __forceinline__ void append_check(const AppendArgs& a) {
  int32_t q0, n, len;
  bool bad = false;
  for (int32_t b = threadIdx.x; b < a.batch; b += kThreads) bad |= !append_sequence(a, b, q0, n, len);
  if (bad) append_report(a, kStatusBadExtend);
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
  if (page < a.num_pages) return page;
  append_report(a, kStatusBadPage);
  return -1;
}

// The angles of row t, at place p of its sequence: cos of rot_dim / 2, then sin.
__device__ __forceinline__ const float* append_angles(const AppendArgs& a, int32_t t, int32_t p) {
  if (a.rot_dim == 0) return nullptr;
  int32_t at = a.positions ? __ldg(a.positions + t) : p;
  if (at < 0 || at >= a.max_position) {
    append_report(a, kStatusBadExtend);
    at = at < 0 ? 0 : a.max_position - 1;
  }
  return a.cos_sin + static_cast<int64_t>(at) * a.rot_dim;
}

__device__ __forceinline__ void bf16x8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void floats8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
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
    const int32_t half = a.rot_dim / 2;
    if (a.interleaved) {
      const float* p = row + (e - a.rot_offset) / 2;
      const float4 x = __ldg(reinterpret_cast<const float4*>(p)), y = __ldg(reinterpret_cast<const float4*>(p + half));
      c[0] = x.x; c[1] = x.y; c[2] = x.z; c[3] = x.w;
      s[0] = y.x; s[1] = y.y; s[2] = y.z; s[3] = y.w;
    } else {
      const float* p = row + (e - a.rot_offset) - (low ? 0 : half);
      floats8(p, c);
      floats8(p + half, s);
    }
  }
  // x: the thread's elements, y: their partners
  __device__ __forceinline__ void apply(float (&x)[8], const float (&y)[8]) const {
    if (!on) return;
    if (partner == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = x[2 * i], v = x[2 * i + 1];
        x[2 * i] = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(v, s[i]));
        x[2 * i + 1] = __fadd_rn(__fmul_rn(v, c[i]), __fmul_rn(u, s[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = __fmul_rn(x[i], c[i]), q = __fmul_rn(y[i], s[i]);
        x[i] = low ? __fsub_rn(p, q) : __fadd_rn(p, q);
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

// The rows of token t, from row r0 on `step` at a time: first the queries' heads, then (KIND != KVQ_FP8_E4M3_PAGE) the
// keys' and the values'.  All threads of the CTA call it; thread i of a row's D / 8 takes its elements 8 i ...
template <int KIND>
__device__ __forceinline__ void append_rows(const AppendArgs& a, int32_t t, int32_t r0, int32_t step) {
  constexpr bool kQuant = KIND != KVQ_FP8_E4M3_PAGE;
  const int32_t b = append_find(
      a, [&](int32_t, int32_t q0, int32_t n, int32_t) { return t >= q0 && t - q0 < n; });
  if (b >= a.batch) return;
  int32_t q0, n, len;
  append_sequence(a, b, q0, n, len);
  const int32_t place = len - n + (t - q0);
  const int32_t per_row = a.head_dim / 8, lanes = kThreads / per_row;
  const int32_t i = threadIdx.x % per_row, slot = threadIdx.x / per_row, e = i * 8;
  const int32_t rows = a.num_q_heads + (kQuant ? a.n_kv * a.num_kv_heads : 0);
  Turn turn;
  turn.place(a, e);
  const float* angles = append_angles(a, t, place);
  if (angles) turn.angles(a, angles, e);
  else turn.on = false;
  int32_t page = -1, off = 0;
  if (kQuant) {
    page = append_page(a, b, place / a.page_size);
    off = place % a.page_size;
  }
  for (int32_t base = r0; base < rows; base += step) {
    const int32_t r = base + slot;
    const bool live = slot < lanes && r < rows;
    const bool is_q = r < a.num_q_heads;
    const int32_t kv = is_q || r - a.num_q_heads < a.num_kv_heads ? 0 : 1;
    const int32_t h = is_q ? r : r - a.num_q_heads - kv * a.num_kv_heads;
    float x[8];
    if (live) {
      const uint16_t* row = is_q   ? a.q + t * a.q_token + h * a.q_head
                            : kv == 0 ? a.k + t * a.k_token + h * a.k_head
                                      : a.v + t * a.v_token + h * a.v_head;
      bf16x8(__ldg(reinterpret_cast<const uint4*>(row + e)), x);
      if (kv == 0 && turn.on) {
        float y[8];
        if (turn.partner != 0) bf16x8(__ldg(reinterpret_cast<const uint4*>(row + e + turn.partner)), y);
        turn.apply(x, y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    }
    if (a.q_out == a.q) __syncthreads();  // (a thread's partners have been read before they are overwritten)
    if (live && is_q) {
      uint4 o = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                           pack_bf16x2(x[6], x[7]));
      *reinterpret_cast<uint4*>(a.q_out + t * a.out_token + h * a.out_head + e) = o;
    }
    if constexpr (kQuant) {
      __half scale;
      const uint2 c = block_codes<KIND>(x, scale);
      if (live && !is_q && page >= 0) {
        const int64_t row = ((static_cast<int64_t>(page) * a.n_kv + kv) * a.num_kv_heads + h) * a.page_size + off;
        *reinterpret_cast<uint2*>(a.codes + row * a.head_dim + e) = c;
        if (KindTraits<KIND>::kScaled && i % 4 == 0)
          static_cast<__half*>(a.scales)[row * (a.head_dim / kBlock) + i / 4] = scale;
      }
    }
  }
}

// grid: (token, row chunk), row chunks fastest
template <int KIND>
__global__ void __launch_bounds__(kThreads) append_rows_kernel(const AppendArgs a) {
  if (blockIdx.x == 0) append_check(a);
  const int32_t lanes = kThreads / (a.head_dim / 8);
  const int32_t t = blockIdx.x / a.row_chunks, chunk = blockIdx.x % a.row_chunks;
  append_rows<KIND>(a, t, chunk * lanes, a.row_chunks * lanes);
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

// grid: (page, chunk of its 2 * heads parts) first, then (token, row chunk) of the queries
template <int D>
__global__ void __launch_bounds__(kThreads) append_pages_kernel(const AppendArgs a) {
  constexpr int PER_ROW = D / 8;               // threads of a row
  constexpr int ROWS = 32 / PER_ROW;           // rows of a pass
  if (blockIdx.x == 0) append_check(a);
  if (blockIdx.x >= a.page_ctas) {
    const int32_t lanes = kThreads / PER_ROW, q = blockIdx.x - a.page_ctas;
    append_rows<KVQ_FP8_E4M3_PAGE>(a, q / a.row_chunks, q % a.row_chunks * lanes, a.row_chunks * lanes);
    return;
  }
  const int32_t item = blockIdx.x / a.part_chunks, chunk = blockIdx.x % a.part_chunks;
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
  const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t part = chunk * kWarps + warp;
  if (part >= 2 * a.num_kv_heads) return;
  const int32_t page = append_page(a, b, j);
  if (page < 0) return;
  const int32_t kv = part / a.num_kv_heads, h = part - kv * a.num_kv_heads;
  const int32_t lo = max(len - n - j * kPage, 0), hi = min(len - j * kPage, kPage);  // new rows of the page
  const int32_t e = lane % PER_ROW * 8, sub = lane / PER_ROW;
  const int64_t row0 = (static_cast<int64_t>(page) * 2 + kv) * a.num_kv_heads + h;
  uint8_t* codes = a.codes + row0 * kPage * D + e;
  float* scale = static_cast<float*>(a.scales) + row0;

  Turn turn;
  turn.place(a, e);
  turn.on &= kv == 0 && a.rot_dim > 0;
  auto load = [&](int32_t r, float (&x)[8]) {  // row r of the page
    const int32_t p = j * kPage + r, t = q0 + p - (len - n);
    const uint16_t* row = kv == 0 ? a.k + t * a.k_token + h * a.k_head : a.v + t * a.v_token + h * a.v_head;
    bf16x8(__ldg(reinterpret_cast<const uint4*>(row + e)), x);
    if (turn.on) {
      turn.angles(a, append_angles(a, t, p), e);
      float y[8];
      if (turn.partner != 0) bf16x8(__ldg(reinterpret_cast<const uint4*>(row + e + turn.partner)), y);
      turn.apply(x, y);
    }
  };
  const float had = lo > 0 ? *scale : 0.0f;
  float m = 0.0f;
#pragma unroll 4
  for (int32_t r = lo + sub; r < hi; r += ROWS) {
    float x[8];
    load(r, x);
    m = fmaxf(m, amax8(x));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  int32_t exp = page_exponent(m);
  if (lo > 0) {
    const int32_t old = min(max(((__float_as_int(had) >> 23) & 255) - 127, kPageScaleMin), kPageScaleMax);
    if (exp > old) {
      const float f = power_of_two(old - exp);
#pragma unroll 4
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
#pragma unroll 4
  for (int32_t r = lo + sub; r < hi; r += ROWS) {
    float x[8];
    load(r, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= inv;
    *reinterpret_cast<uint2*>(codes + r * D) = fp8x8<__NV_E4M3>(x);
  }
  if (lane == 0) *scale = power_of_two(exp);
}

// Clears the status word; the append is its programmatic dependent and touches the word only after a wait.
__global__ void append_clear_kernel(uint32_t* word) {
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) *word = 0;
}

template <typename Kernel>
kvq_status launch(Kernel kern, const AppendArgs& a, int64_t grid, cudaStream_t stream) {
  append_clear_kernel<<<1, 32, 0, stream>>>(a.status);
  if (cudaGetLastError() != cudaSuccess) return KVQ_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

}  // namespace

bool append_supported(int32_t head_dim, kvq_kind kind) {
  if (kind == KVQ_FP8_E4M3_PAGE) return head_dim == 64 || head_dim == 128 || head_dim == 256;
  return head_dim / 8 <= kThreads;
}

int64_t append_grid(AppendArgs* a, int32_t sms) {
  const int32_t lanes = kThreads / (a->head_dim / 8);
  const bool pages = a->kind == KVQ_FP8_E4M3_PAGE;
  const int32_t rows = a->num_q_heads + (pages ? 0 : a->n_kv * a->num_kv_heads);
  const int32_t passes = (rows + lanes - 1) / lanes;
  // a token's rows are spread over CTAs while these would not fill the GPU
  a->row_chunks = static_cast<int32_t>(
      std::max<int64_t>(1, std::min<int64_t>(passes, 4LL * sms / std::max(1, a->total))));
  a->part_chunks = (2 * a->num_kv_heads + kWarps - 1) / kWarps;
  const int64_t items = pages ? (static_cast<int64_t>(a->total) + 14LL * a->batch) / kPage + a->batch : 0;
  a->page_ctas = items * a->part_chunks;
  return a->page_ctas + (rows > 0 ? static_cast<int64_t>(a->total) * a->row_chunks : 0);
}

kvq_status launch_append(const AppendArgs& a, int64_t grid, cudaStream_t stream) {
  switch (a.kind) {
    case KVQ_FP8_E4M3: return launch(append_rows_kernel<KVQ_FP8_E4M3>, a, grid, stream);
    case KVQ_Q8_0: return launch(append_rows_kernel<KVQ_Q8_0>, a, grid, stream);
    case KVQ_FP8_E4M3_UNSCALED: return launch(append_rows_kernel<KVQ_FP8_E4M3_UNSCALED>, a, grid, stream);
    case KVQ_FP8_E5M2_UNSCALED: return launch(append_rows_kernel<KVQ_FP8_E5M2_UNSCALED>, a, grid, stream);
    case KVQ_FP8_E4M3_PAGE:
      if (a.head_dim == 64) return launch(append_pages_kernel<64>, a, grid, stream);
      if (a.head_dim == 128) return launch(append_pages_kernel<128>, a, grid, stream);
      return launch(append_pages_kernel<256>, a, grid, stream);
  }
  return KVQ_EKIND;
}

}  // namespace kvq
