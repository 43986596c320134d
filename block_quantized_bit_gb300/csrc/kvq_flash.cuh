// kvq_flash.cuh -- pieces shared by the flash-style tcgen05 kernels (extend, tree, prompt): 128 query rows are the
// MMA's M, S and O live in tensor memory with one row per lane, P goes back to tensor memory as bf16.
#pragma once

#include "kvq_tc.cuh"

namespace kvq {
namespace {

// kind::f16 instruction descriptor: fp32 accumulate, bf16 A and B, M = 128, the given N; A K-major.
__device__ __forceinline__ uint32_t x_idesc(int n, bool b_mn_major) {
  uint32_t d = 0;
  d |= 1u << 4;   // D: f32
  d |= 1u << 7;   // A: bf16
  d |= 1u << 10;  // B: bf16
  d |= static_cast<uint32_t>(b_mn_major) << 16;
  d |= static_cast<uint32_t>(n >> 3) << 17;
  d |= static_cast<uint32_t>(128 >> 4) << 24;
  return d;
}

__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Tensor-memory loads and stores of 32 consecutive columns of this warp's 32 lanes.  A load's registers are
// valid only after tcgen05.wait::ld; the waits below take them as operands, so no use moves above the wait.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  tmem_ld32_issue(taddr, r);
  tmem_wait_ld32(r);
}

// The same load with the maximum of the 32 columns of each lane beside them (the reduction rides on the load).
__device__ __forceinline__ void tmem_ld32_max_issue(uint32_t taddr, uint32_t* r, uint32_t& top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(top)
      : "r"(taddr));
}

// ... whose wait takes the maximum as an operand as well.
__device__ __forceinline__ void tmem_wait_max(uint32_t& top) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(top) : : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32"
      "};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// 2^x by the hardware approximation (relative error far below the bf16 rounding that follows); 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^x on the FMA pipe, for a share of the probabilities (the MUFU unit alone would pace the softmax):
// x = j + f with j = round(x) by the 1.5 * 2^23 addition (the sum's low mantissa bits hold j) and f in
// [-0.5, 0.5]; 2^f by a cubic; j added to the exponent field.  The cubic's coefficients are a minimax fit of
// 2^f on [-0.5, 0.5] for relative error, computed by Lawson's iteratively reweighted least squares on
// Chebyshev nodes (the weights grow where the error is largest until it equioscillates), then rounded to
// fp32.  Relative error at most 1.5e-4 over [-126, 8] (kvq_exp2_probe exposes this routine so that a test
// checks the bound on the GPU), far below the bf16 rounding of P that follows.  x is clamped at -126 (the
// result is then about 2^-126, not 0: callers zero masked keys themselves).
__device__ __forceinline__ float ex2_fma(float x) {
  x = fmaxf(x, -126.0f);
  const float t = x + 12582912.0f;
  const int j = __float_as_int(t) - 0x4B400000;
  const float f = x - (t - 12582912.0f);
  const float p = fmaf(fmaf(fmaf(0.0551716685f, f, 0.2426111251f), f, 0.6932609677f), f, 0.9999280572f);
  return __int_as_float(__float_as_int(p) + (j << 23));
}

// Four MMAs of which two read A at a0 and two at a1 (8 columns apart each).
__device__ __forceinline__ void mma2x2_bf16_tmem_a(uint32_t d_tmem, uint32_t a0, uint32_t a1, uint64_t b, uint64_t b_step,
                                                   uint32_t idesc, uint32_t acc_first) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "add.u32 a2, %1, 8;\n\tadd.u32 a3, %5, 8;\n\t"
      "add.u64 b1, %2, %6;\n\tadd.u64 b2, b1, %6;\n\tadd.u64 b3, b2, %6;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b1, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], b2, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d_tmem),
      "r"(a0), "l"(b), "r"(idesc), "r"(acc_first), "r"(a1), "l"(b_step)
      : "memory");
}

// Shared-memory descriptor of an operand in 128-byte swizzled rows (1024-byte aligned groups of eight).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return smem_desc(addr, lbo, sbo) | (static_cast<uint64_t>(2) << 61);  // 128-byte swizzle
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

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 bytes that are read once: no line is kept in L1.
__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Four MMAs from a single elect.sync, A in tensor memory (a_step in columns); as mma8_bf16_tmem_a.
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

// A bounded wait that the whole warp agrees on: no lane runs ahead into a warp-collective tcgen05 instruction
// while another gave up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}

// The same with everything behind the first try out of line: where several roles share an SM's instruction cache,
// each wait's unlikely part costs the others misses (prompt 16384 x 32 heads 1455 -> 1405 us, tree at head_dim 128
// 139 -> 132 us; the tree kernel at 256, whose registers spill around the call, keeps the other: 180 against 256 us).
__device__ __noinline__ bool mbar_wait_rest(uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity); }

__device__ __forceinline__ bool warp_wait_far(uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_rest(bar, parity));
}

}  // namespace
}  // namespace kvq
