// kvq_page.cuh -- pieces shared by the kernels over a KVQ_FP8_E4M3_PAGE cache: output stores.
#pragma once

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

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

}  // namespace
}  // namespace kvq
