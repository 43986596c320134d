// kvq_page.cuh -- pieces shared by the kernels over a KVQ_FP8_E4M3_PAGE cache: how a call's work is cut into equal runs,
// output stores.
#pragma once

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr float kNoMax = -0x1.fffffep127f;  // reference of a row that has seen nothing: below every finite score
constexpr float kHead = 7.0f;     // log2 of the largest p when a row's reference moves ...
constexpr float kLimit = 15.0f;   // ... and at most (P is f16, which ends at 2^16)

// Every CTA reports into a word of its own behind the runs, and the joining kernel, which waits for them all, collects these: a
// status word shared by the CTAs would have to be cleared by a launch of its own (2 us of a small call).  A single CTA has the
// status word itself.
__device__ __forceinline__ uint32_t* page_words(const PageArgs& a) {
  return reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.runs) + static_cast<size_t>(a.grid) * kPageRunMost);
}
__device__ __forceinline__ uint32_t* page_word(const PageArgs& a) {
  return a.grid == 1 ? a.status : page_words(a) + blockIdx.x;
}
__device__ __forceinline__ void page_clear(const PageArgs& a) {  // before the CTA's first barrier
  if (threadIdx.x == 0) *page_word(a) = 0;
}
__device__ __forceinline__ void page_report(const PageArgs& a, uint32_t code) { set_status(page_word(a), code); }
__device__ __forceinline__ void page_collect(const PageArgs& a) {  // by the joining kernel, once the CTAs have ended
  if (blockIdx.x != 0 || blockIdx.y != 0 || threadIdx.x >= 32) return;
  uint32_t code = 0;
  for (int32_t c = threadIdx.x; c < a.grid; c += 32) code = max(code, page_words(a)[c]);
  code = __reduce_max_sync(0xffffffffu, code);
  if (threadIdx.x == 0) *a.status = code;
}

// A kernel that may start before the one in front of it in the stream has ended.
template <typename Kernel, typename... Args>
bool launch_dependent(Kernel kern, dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

// One sequence's query rows and stored tokens; n = 0: nothing to do.
struct PageSeq {
  int32_t q0, n, len;
};

__device__ __forceinline__ PageSeq page_sequence(const PageArgs& a, int32_t b, bool& bad) {
  PageSeq s;
  const int32_t room = a.max_pages * kPage;
  s.len = __ldg(a.seq_lens + b);
  if (a.q_start == nullptr) {  // one row per sequence
    s.q0 = b;
    s.n = 1;
    s.len = min(max(s.len, 0), room);
    return s;
  }
  s.q0 = __ldg(a.q_start + b);
  const int64_t q1 = __ldg(a.q_start + b + 1), n = q1 - s.q0;
  const bool ok = s.q0 >= 0 && n >= 0 && q1 <= a.total_q && n <= s.len && s.len <= room;
  bad |= !ok;
  s.n = ok ? static_cast<int32_t>(n) : 0;
  return s;
}

// All units of a call lie in one order, sequence by sequence.  U of them are shared by C CTAs, each taking an equal
// run, whatever the lengths.
__device__ __forceinline__ int32_t sharers(int64_t U, int32_t grid, int32_t least) {
  return static_cast<int32_t>(min(static_cast<int64_t>(grid), max(U / least, static_cast<int64_t>(1))));
}
__device__ __forceinline__ int64_t first_unit(int64_t U, int32_t C, int32_t c) { return U * c / C; }

// The CTA among whose units u is.
__device__ __forceinline__ int32_t owner_of(int64_t U, int32_t C, int64_t u) {
  int32_t c = static_cast<int32_t>(u * C / U);
  while (c > 0 && first_unit(U, C, c) > u) --c;
  while (c + 1 < C && first_unit(U, C, c + 1) <= u) ++c;
  return c;
}

// The slot of partial sums that CTA c has for a tile whose first unit is `first`: a run's tile that began before it, or
// fills it, has the first of the two.
__device__ __forceinline__ int64_t part_slot(int64_t U, int32_t C, int32_t c, int64_t first) {
  return 2 * static_cast<int64_t>(c) + (first > first_unit(U, C, c) ? 1 : 0);
}

// The sequence in which unit want(total) lies, and the units before it.
struct Place {
  int64_t total, before;
  int32_t b;  // -1: none
};

// units(b): a sequence's units; every thread of the CTA (of WARPS warps) calls it.  total_out, where not null, receives
// the units of the call.
template <int WARPS, typename Units, typename Want>
__device__ __forceinline__ Place page_place(int32_t batch, int64_t* total_out, Units units, Want want_of) {
  __shared__ int64_t s_sum[WARPS];
  __shared__ Place s_place;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t per = (batch + WARPS * 32 - 1) / (WARPS * 32);
  const int32_t b0 = min(tid * per, batch), b1 = min(b0 + per, batch);
  int64_t mine = 0;
  for (int32_t b = b0; b < b1; ++b) mine += units(b);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sum[warp] = incl;
  if (tid == 0) s_place.b = -1;
  __syncthreads();
  int64_t run = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) run += s_sum[w];
    total += s_sum[w];
  }
  const int64_t want = want_of(total);
  if (total_out != nullptr && tid == 0) *total_out = total;
  for (int32_t b = b0; b < b1; ++b) {
    const int64_t u = per == 1 ? mine : units(b);
    if (want >= run && want < run + u) {
      s_place.b = b;
      s_place.before = run;
    }
    run += u;
  }
  __syncthreads();
  Place p = s_place;
  p.total = total;
  return p;
}

// Four neighbouring outputs x * scale from element `at` on (a multiple of 4), bf16 or fp32.
__device__ __forceinline__ void page_store_out(const PageArgs& a, int64_t at, float4 x, float scale) {
  x.x *= scale;
  x.y *= scale;
  x.z *= scale;
  x.w *= scale;
  if (a.out_dtype == KVQ_OUT_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = x;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// P, the f16 that meets a token's V codes, is 2^(score + ev - m).  A page whose V scale 2^e is far below that of pages before it
// would leave P too few bits (f16 has 2^-14 to 2^15 in full), so its codes take up to 2^-14 of the scale, exactly: a code
// is 2^-9 at the least and 4 bits wide.  `ref` is the largest e of the run so far, so the scales' part in P is within
// 2^4 while pages' scales are within 2^18; P is then off by at most 2^-11 of itself or 2^-25 2^m, which is 2^-28 of the row's
// largest p; further down by as much more.
constexpr int kNearScales = 4;  // powers of two within which codes stay as they are: no product a code where scales are alike
__device__ __forceinline__ int32_t codes_down(int32_t e, int32_t ref) {
  return ref - e > kNearScales ? min(ref - e, 14) : 0;
}
__device__ __forceinline__ uint32_t f16x2_power(int32_t down) { return (15u - down) * 0x04000400u; }  // 2^-down, twice
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The exponent of a page's scale; 2^-e.
__device__ __forceinline__ int32_t scale_exponent(float s) { return (__float_as_int(s) >> 23) - 127; }
__device__ __forceinline__ float power_inverse(int32_t e) { return __int_as_float((127 - e) << 23); }

}  // namespace
}  // namespace kvq
