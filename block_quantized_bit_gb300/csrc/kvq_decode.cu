// kvq_decode.cu -- split-K decode attention over the 8-bit paged pool, CUDA-core path, and the merge.
//
// "feat(kvcache): 8-bit KV cache (q8_0 / fp8_e4m3) behind --kv-cache-dtype", section "What": the scale
// varies along head_dim, the reduction dim, so K and V are dequantized to bf16 before the dot.
// "feat(kvcache): 8-bit DSV4 window/compressed KV", section "Testing": the split-k decode kernel and
// masked (-1) columns; section "What this adds": an MLA latent row serves as both K and V.
//
// Work decomposition (computed identically by every CTA from seq_lens, so no planning launch and no
// host read-back is needed; CTA 0 also leaves each sequence's first item and split count for the merge):
//   query group qg = (kv head g, head tile ht): `heads_per_item` query heads that share kv head g;
//   pages of sequence b are cut into splits of C pages; one work item = (b, qg, split);
//   C = pages_per_split, or max(4, ceil(sum_b pages_b * groups / target)) when automatic, target a little
//   under two waves of the resident CTAs (the host's plan).
// One CTA runs one item.  Each of its warps walks every WARPS-th page of the split with its own
// STAGES-deep pipeline of 1-D bulk copies (codes and scales of the page's K and V chunks into shared
// memory, completion on an mbarrier).  Lanes read 16-byte code chunks, dequantize to bf16-exact fp32,
// and run the fp32 online softmax in the exp2 domain; the CTA combines its warps and writes one
// (m, l, acc) partial per query head.  The CTA that finishes the last split of a (b, qg) merges the
// group's partials itself (a split counter in the workspace), so this path needs no merge launch; a
// group with one split writes its output directly.  The merge kernel below combines the partials of
// the tensor-core kernels.
#include <math.h>

#include <algorithm>

#include "kvq_decode_cc.cuh"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_plan.cuh"

namespace kvq {

namespace {

// ------------------------------------------------------------------------------------- merge
constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMergeSubs = 4;  // splits a warp reads at once: 8 lanes x float4 = the 32 dims of a slice

// One CTA per (sequence, query group, head of the item, 32-dim slice of v): the log-sum-exp merge of
// the sequence's split partials, out = sum_s 2^(m_s - M) acc_s / sum_s 2^(m_s - M) l_s, M = max_s m_s.
// A warp reads four splits at a time (lanes 8j..8j+7 take split j, four dims each), so the CTA has 32
// splits' loads in flight per round; the sums are reduced across the lane groups and the warps.  The
// decode kernel's CTA 0 left each sequence's first item and split count in plan_tab, so no plan is
// recomputed here.
template <typename OutT>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(KParams p, OutT* __restrict__ out, int32_t heads_per_item,
                                                              int32_t DV, int32_t units_per_seq) {
  __shared__ float s_m[kMergeWarps];
  __shared__ __align__(16) float s_a[kMergeWarps][32];
  __shared__ float s_l[kMergeWarps];
  // Launched as a programmatic dependent of the decode kernel: its CTAs may start while the decode's last
  // CTAs still run; this waits until that grid has completed and its partials are visible.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane >> 3, q = lane & 7;  // split of the four, float4 of the slice
  const int32_t b = blockIdx.x / units_per_seq;
  const int32_t u = blockIdx.x - b * units_per_seq;
  const int32_t slices = DV / 32;
  const int32_t slice = u % slices;
  const int32_t h = (u / slices) % heads_per_item;
  const int32_t qg = u / (slices * heads_per_item);
  const int32_t g = qg / p.head_tiles, ht = qg - g * p.head_tiles;
  const int32_t head = g * p.group + ht * heads_per_item + h;
  int32_t ns = p.plan_tab[2 * b + 1];
  const int64_t first = static_cast<int64_t>(p.plan_tab[2 * b]) + static_cast<int64_t>(qg) * ns;
  if (ns < 0 || first < 0 || first + ns > p.max_items) {  // cannot happen when the workspace bound holds
    if (tid == 0) set_status(p.status, kStatusBadPage);
    ns = 0;
  }
  float M = -INFINITY;
  for (int32_t s = tid; s < ns; s += kMergeThreads) M = fmaxf(M, p.part_ml[((first + s) * heads_per_item + h) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) s_m[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) M = fmaxf(M, s_m[w]);
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f;
  if (M != -INFINITY) {
    const float* acc = p.part_acc + slice * 32 + q * 4;
#pragma unroll 2
    for (int32_t s = warp * kMergeSubs + sub; s < ns; s += kMergeWarps * kMergeSubs) {
      const int64_t it = (first + s) * heads_per_item + h;
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + it * 2);
      const float w = (ml.x == -INFINITY) ? 0.0f : exp2f(ml.x - M);
      const float4 v = *reinterpret_cast<const float4*>(acc + it * DV);
      a.x = fmaf(v.x, w, a.x);
      a.y = fmaf(v.y, w, a.y);
      a.z = fmaf(v.z, w, a.z);
      a.w = fmaf(v.w, w, a.w);
      l = fmaf(ml.y, w, l);
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {  // over the four lane groups (the same q)
    a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
    l += __shfl_xor_sync(0xffffffffu, l, o);
  }
  if (lane < 8) *reinterpret_cast<float4*>(&s_a[warp][q * 4]) = a;
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (warp == 0) {
    float at = 0.0f, lt = 0.0f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      at += s_a[w][lane];
      lt += s_l[w];
    }
    const float o = (lt > 0.0f) ? at / lt : 0.0f;
    const int64_t dst = (static_cast<int64_t>(b) * p.num_q_heads + head) * DV + slice * 32 + lane;
    if constexpr (sizeof(OutT) == 2)
      out[dst] = __float2bfloat16_rn(o);
    else
      out[dst] = o;
  }
}

// The merge of drafted tokens' splits (kvq_tree over the MLA row): a warp per output row, since a call has thousands
// of rows (a CTA per 32 outputs, as above, took 3.4 ms for 1024 drafted tokens of 128 heads).  Rows with one split are
// final already; rows that no sequence covers are left as they are.
template <int DV>
__global__ void __launch_bounds__(kMergeThreads) merge_rows_kernel(KParams p, int32_t heads_per_item) {
  constexpr int V4 = DV / 128;  // float4 per lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
  const int32_t b = static_cast<int32_t>(row / p.num_q_heads);
  if (b >= p.batch || uncovered(p, b)) return;
  const int32_t head = static_cast<int32_t>(row - static_cast<int64_t>(b) * p.num_q_heads);
  const int32_t qg = head / heads_per_item, h = head - qg * heads_per_item;
  const int32_t ns = p.plan_tab[2 * b + 1];
  const int64_t first = static_cast<int64_t>(p.plan_tab[2 * b]) + static_cast<int64_t>(qg) * ns;
  if (ns <= 1 || first < 0 || first + ns > p.max_items) return;
  float M = -INFINITY;
  for (int32_t s = lane; s < ns; s += 32) M = fmaxf(M, p.part_ml[((first + s) * heads_per_item + h) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float4 a[V4];
#pragma unroll
  for (int j = 0; j < V4; ++j) a[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f;
#pragma unroll 2
  for (int32_t s = 0; s < ns; ++s) {
    const int64_t it = (first + s) * heads_per_item + h;
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + it * 2);
    const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - M);
    l = fmaf(ml.y, w, l);
#pragma unroll
    for (int j = 0; j < V4; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(p.part_acc + it * DV + j * 128 + lane * 4);
      a[j].x = fmaf(v.x, w, a[j].x);
      a[j].y = fmaf(v.y, w, a[j].y);
      a[j].z = fmaf(v.z, w, a[j].z);
      a[j].w = fmaf(v.w, w, a[j].w);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int j = 0; j < V4; ++j) {
    const int64_t at = row * DV + j * 128 + lane * 4;
    const float4 o = make_float4(a[j].x * inv, a[j].y * inv, a[j].z * inv, a[j].w * inv);
    if (p.out_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = o;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
          make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  }
}

// --------------------------------------------------------------------------------- dequant probe
template <int KIND>
__global__ void dequant_probe_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                                     uint16_t* __restrict__ out, int64_t nchunks) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t c = i; c < nchunks; c += stride) {
    const uint4 code = reinterpret_cast<const uint4*>(codes)[c];
    uint32_t kd[8];
    dequant16<KIND>(code, KindTraits<KIND>::kScaled ? scales[c] : kHalfOne, kd);
    uint4* dst = reinterpret_cast<uint4*>(out + c * 16);
    dst[0] = make_uint4(kd[0], kd[1], kd[2], kd[3]);
    dst[1] = make_uint4(kd[4], kd[5], kd[6], kd[7]);
  }
}

}  // namespace

int32_t cc_heads_per_item(int32_t group, int32_t head_dim, int32_t mla) {
  const int32_t cap = mla ? 2 : 4;
  int32_t gt = 1;
  while (gt * 2 <= cap && group % (gt * 2) == 0) gt *= 2;
  (void)head_dim;
  return gt;
}

// CTAs per SM that launch_decode_cc's configuration keeps resident (its MINB).
int32_t cc_ctas_per_sm(int32_t head_dim, int32_t mla, int32_t gt) {
  if (mla) return 1;
  if (head_dim == 64) return 4;
  if (head_dim == 128) return gt == 2 ? 5 : 4;
  return 3;
}

bool decode_cc_supported(int32_t head_dim, int32_t v_dim, int32_t mla) {
  if (mla) return head_dim == 576 && v_dim == 512;
  return v_dim == head_dim && (head_dim == 64 || head_dim == 128 || head_dim == 256);
}

kvq_status launch_decode_cc(const DecodeArgs& a, cudaStream_t stream) {
  return a.tree_mask != nullptr ? launch_decode_cc_masked(a, stream) : launch_cc_shape<false>(a, stream);
}

kvq_status launch_merge(const DecodeArgs& a, int32_t query_groups, cudaStream_t stream) {
  const KParams p = make_kparams(a);
  const int32_t units = query_groups * a.heads_per_item * (a.v_dim / 32);
  const bool rows = a.tree_mask != nullptr && a.v_dim == 512;  // drafted tokens over the MLA row
  const int64_t grid = rows ? (static_cast<int64_t>(a.batch) * a.num_q_heads + kMergeWarps - 1) / kMergeWarps
                            : static_cast<int64_t>(a.batch) * units;
  if (grid == 0) return KVQ_OK;
  // programmatic stream serialization: the merge grid launches as the decode grid winds down instead of after it
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (rows)
    e = cudaLaunchKernelEx(&cfg, merge_rows_kernel<512>, p, a.heads_per_item);
  else if (a.out_dtype == KVQ_OUT_BF16)
    e = cudaLaunchKernelEx(&cfg, merge_kernel<__nv_bfloat16>, p, static_cast<__nv_bfloat16*>(a.out), a.heads_per_item,
                           a.v_dim, units);
  else
    e = cudaLaunchKernelEx(&cfg, merge_kernel<float>, p, static_cast<float*>(a.out), a.heads_per_item, a.v_dim,
                           units);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? KVQ_OK : KVQ_ECUDA;
}

// ------------------------------------------------------------------------------------ wait probe
// One thread initialises an mbarrier expecting one arrival that never comes, and waits on it with
// mbar_wait_bounded, the wait every decode kernel uses; it gives up after kWaitLimitNs and reports the
// timeout exactly as a decode kernel would.
__global__ void wait_probe_kernel(uint32_t* status) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x != 0) return;
  mbar_init(&bar, 1);
  fence_mbar_init();
  if (!mbar_wait_bounded(&bar, 0)) set_status(status, kStatusTimeout);
}

kvq_status launch_wait_probe(uint32_t* status, cudaStream_t stream) {
  wait_probe_kernel<<<1, 32, 0, stream>>>(status);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

kvq_status launch_dequant_probe(kvq_kind kind, const uint8_t* codes, const uint16_t* scales, uint16_t* out,
                                int64_t n, cudaStream_t stream) {
  const int64_t nchunks = n / 16;
  if (nchunks == 0) return KVQ_OK;
  const int threads = 256;
  const int64_t grid = std::min<int64_t>((nchunks + threads - 1) / threads, 152 * 16);
  const unsigned g = static_cast<unsigned>(grid);
  switch (kind) {
    case KVQ_FP8_E4M3: dequant_probe_kernel<KVQ_FP8_E4M3><<<g, threads, 0, stream>>>(codes, scales, out, nchunks); break;
    case KVQ_Q8_0: dequant_probe_kernel<KVQ_Q8_0><<<g, threads, 0, stream>>>(codes, scales, out, nchunks); break;
    case KVQ_FP8_E4M3_UNSCALED:
      dequant_probe_kernel<KVQ_FP8_E4M3_UNSCALED><<<g, threads, 0, stream>>>(codes, scales, out, nchunks);
      break;
    case KVQ_FP8_E5M2_UNSCALED:
      dequant_probe_kernel<KVQ_FP8_E5M2_UNSCALED><<<g, threads, 0, stream>>>(codes, scales, out, nchunks);
      break;
  }
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

}  // namespace kvq
