// kvq_prompt.cuh -- pieces shared by the two kernels of the prompt attention (kvq_prompt): items and their order,
// TMA boxes of packed rows, swizzled shared-memory descriptors.
#pragma once

#include "kvq_flash.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kM = 128;                // rows of a tile (the MMA M)
constexpr int kTmemCols = 512;
constexpr float kLazyRescale = 8.0f;   // log2 headroom before the running max must move

// A published item: one or two tiles of (sequence, kv head); q0: the sequence's first row; len: its tokens; per
// tile its token block (-1: no such tile) and query head.
struct Item {
  int32_t q0, len, g, blk[2], head[2], live;
};
static_assert(sizeof(Item) == 32, "item slots");

// One box: 64 elements (128 bytes) of `head`, the map's number of rows from `row`.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int head, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(row), "r"(smem_u32(bar))
      : "memory");
}

// Items of a sequence of len tokens: ceil(len / 128) token blocks of G heads, TILES of them at a time.
template <int TILES>
__device__ __forceinline__ int32_t prompt_items(int32_t len, int32_t G) {
  return ((len + kM - 1) / kM * G + TILES - 1) / TILES;
}

// tab[b] = items per kv head of sequence b (0 for an inconsistent one, which CTA 0 reports).
template <int TILES>
__device__ __forceinline__ void prompt_table(const PromptArgs& a, int32_t* tab) {
  for (int32_t b = threadIdx.x; b < a.batch; b += blockDim.x) {
    const int32_t q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1);
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.total;
    if (!ok && blockIdx.x == 0) set_status(a.status, kStatusBadExtend);
    tab[b] = ok ? prompt_items<TILES>(q1 - q0, a.num_q_heads / a.num_kv_heads) : 0;
  }
}

// The items of the call in order of falling level p, so that the longest start first: level p holds item p of every
// sequence that has one, times the kv heads.  All 32 lanes of the warp call its members.
template <int TILES>
struct ItemSource {
  const PromptArgs& a;
  const int32_t* tab;
  int32_t top;      // items of the longest sequence
  bool narrow;      // sums over the sequences fit 32 bits
  int64_t n_items;
  __device__ __forceinline__ ItemSource(const PromptArgs& args, const int32_t* table) : a(args), tab(table) {
    const int lane = threadIdx.x & 31;
    top = 0;
    for (int32_t b = lane; b < a.batch; b += 32) top = max(top, tab[b]);
    top = __reduce_max_sync(0xffffffffu, top);
    narrow = static_cast<int64_t>(top) * a.batch < (1LL << 31);
    n_items = above(-1);
  }
  // items of levels > p
  __device__ __forceinline__ int64_t above(int32_t p) const {
    int64_t s = 0;
    for (int32_t b = threadIdx.x & 31; b < a.batch; b += 32) s += max(tab[b] - p - 1, 0);
    if (narrow) return static_cast<int64_t>(__reduce_add_sync(0xffffffffu, static_cast<int32_t>(s))) * a.num_kv_heads;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s * a.num_kv_heads;
  }
  __device__ __forceinline__ Item get(int64_t idx) const {
    Item it;
    it.live = idx < n_items;
    if (!it.live) return it;
    const int lane = threadIdx.x & 31;
    const int32_t G = a.num_q_heads / a.num_kv_heads;
    int32_t lo = 0, hi = top - 1;  // smallest p with above(p) <= idx
    while (lo < hi) {
      const int32_t mid = (lo + hi) >> 1;
      if (above(mid) <= idx) hi = mid;
      else lo = mid + 1;
    }
    const int32_t p = lo;
    const int32_t q = static_cast<int32_t>(idx - above(p));  // below batch * kv heads
    int32_t rank = q / a.num_kv_heads, b = 0;
    it.g = q - rank * a.num_kv_heads;
    for (int32_t b0 = 0; b0 < a.batch; b0 += 32) {  // the rank-th sequence with more than p items
      const uint32_t m = __ballot_sync(0xffffffffu, b0 + lane < a.batch && tab[b0 + lane] > p);
      const int32_t c = __popc(m);
      if (rank < c) {  // the lane whose bit is the rank-th of the mask (from 0)
        const bool hit = ((m >> lane) & 1u) && __popc(m & ((1u << lane) - 1u)) == rank;
        b = b0 + __ffs(__ballot_sync(0xffffffffu, hit)) - 1;
        break;
      }
      rank -= c;
    }
    it.q0 = __ldg(a.q_start + b);
    it.len = __ldg(a.q_start + b + 1) - it.q0;
    const int32_t tiles = (it.len + kM - 1) / kM * G;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int32_t t = TILES * p + w;
      it.blk[w] = w < TILES && t < tiles ? t / G : -1;
      it.head[w] = it.g * G + t % G;
    }
    return it;
  }
};

// Clears the rows from `from` on of a tile of CHUNKS column chunks of ROWS rows: the V rows of keys behind the
// sequence's end, which no probability but 0 meets.
template <int CHUNKS, int ROWS>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int32_t from) {
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c)
#pragma unroll 4
    for (int32_t o = from * 128 + (threadIdx.x & 31) * 16; o < ROWS * 128; o += 512)
      *reinterpret_cast<uint4*>(tile + c * ROWS * 128 + o) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// One row's 32 output columns o * scale, at element `at` of the output.
__device__ __forceinline__ void store_row32(const PromptArgs& a, int64_t at, const uint32_t (&ov)[32], float scale) {
  float o[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(ov[e]) * scale;
  if (a.out_dtype == KVQ_OUT_F32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
#pragma unroll
    for (int q4 = 0; q4 < 8; ++q4) dst[q4] = make_float4(o[4 * q4], o[4 * q4 + 1], o[4 * q4 + 2], o[4 * q4 + 3]);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at);
#pragma unroll
    for (int h8 = 0; h8 < 4; ++h8)
      dst[h8] = make_uint4(pack_bf16x2(o[8 * h8], o[8 * h8 + 1]), pack_bf16x2(o[8 * h8 + 2], o[8 * h8 + 3]),
                           pack_bf16x2(o[8 * h8 + 4], o[8 * h8 + 5]), pack_bf16x2(o[8 * h8 + 6], o[8 * h8 + 7]));
  }
}

// (element, head, token) view of a bf16 tensor [total][heads][D] with the given strides in elements; a box is 64
// elements of `rows` tokens of one head.
inline bool encode_rows(CUtensorMap* map, const void* x, int64_t total, int32_t heads, int D, int64_t token, int64_t head,
                        int32_t rows) {
  const EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(total)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(token) * 2};
  const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace kvq
