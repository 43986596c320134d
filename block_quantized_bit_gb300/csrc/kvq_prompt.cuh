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

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

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

// The clearing kernel before this one has completed from here on.
__device__ __forceinline__ void wait_cleared() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void prompt_report(const PromptArgs& a, uint32_t code) {
  wait_cleared();
  set_status(a.status, code);
}

// tab[b] = items per kv head of sequence b (0 for an inconsistent one, which CTA 0 reports).
template <int TILES>
__device__ __forceinline__ void prompt_table(const PromptArgs& a, int32_t* tab) {
  for (int32_t b = threadIdx.x; b < a.batch; b += blockDim.x) {
    const int32_t q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1);
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.total;
    if (!ok && blockIdx.x == 0) prompt_report(a, kStatusBadExtend);
    tab[b] = ok ? prompt_items<TILES>(q1 - q0, a.num_q_heads / a.num_kv_heads) : 0;
  }
}

// The items of the call in order of falling level p, so that the longest start first: level p holds item p of every
// sequence that has one, times the kv heads.  All 32 lanes of the warp call its members.  A lane keeps the first 32
// sequences' entry of the table in a register.
template <int TILES>
struct ItemSource {
  const PromptArgs& a;
  const int32_t* tab;
  int32_t tab0;     // tab[lane]
  int32_t top;      // items of the longest sequence
  bool narrow;      // sums over the sequences fit 32 bits
  __device__ __forceinline__ ItemSource(const PromptArgs& args, const int32_t* table) : a(args), tab(table) {
    const int lane = threadIdx.x & 31;
    tab0 = lane < a.batch ? tab[lane] : 0;
    top = tab0;
    for (int32_t b = lane + 32; b < a.batch; b += 32) top = max(top, tab[b]);
    top = __reduce_max_sync(0xffffffffu, top);
    narrow = static_cast<int64_t>(top) * a.batch < (1LL << 31);
  }
  // items of levels > p
  __device__ __forceinline__ int64_t above(int32_t p) const {
    int64_t s = max(tab0 - p - 1, 0);
    for (int32_t b = (threadIdx.x & 31) + 32; b < a.batch; b += 32) s += max(tab[b] - p - 1, 0);
    if (narrow) return static_cast<int64_t>(__reduce_add_sync(0xffffffffu, static_cast<int32_t>(s))) * a.num_kv_heads;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s * a.num_kv_heads;
  }
  __device__ __forceinline__ Item get(int64_t idx) const {
    Item it;
    it.live = 0;
    const int lane = threadIdx.x & 31;
    const int32_t G = a.num_q_heads / a.num_kv_heads;
    int32_t lo = 0, hi = top - 1;  // smallest p >= 0 with above(p) <= idx
    int64_t before = 0;            // above(hi)
    while (lo < hi) {
      const int32_t mid = (lo + hi) >> 1;
      const int64_t s = above(mid);
      if (s <= idx) {
        hi = mid;
        before = s;
      } else {
        lo = mid + 1;
      }
    }
    const int32_t p = lo;
    if (p >= top || idx - before >= static_cast<int64_t>(a.batch) * a.num_kv_heads) return it;
    const int32_t q = static_cast<int32_t>(idx - before);  // below batch * kv heads
    int32_t rank = q / a.num_kv_heads, b = -1;
    it.g = q - rank * a.num_kv_heads;
    for (int32_t b0 = 0; b0 < a.batch; b0 += 32) {  // the rank-th sequence with more than p items
      const int32_t x = b0 == 0 ? tab0 : b0 + lane < a.batch ? tab[b0 + lane] : 0;
      const uint32_t m = __ballot_sync(0xffffffffu, x > p);
      const int32_t c = __popc(m);
      if (rank < c) {  // the lane whose bit is the rank-th of the mask (from 0)
        const bool hit = ((m >> lane) & 1u) && __popc(m & ((1u << lane) - 1u)) == rank;
        b = b0 + __ffs(__ballot_sync(0xffffffffu, hit)) - 1;
        break;
      }
      rank -= c;
    }
    if (b < 0) return it;  // past the last item
    it.live = 1;
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

// 32 output columns o * scale of a warp's 32 rows, one row per lane; row 0's first column is element `at` of the output,
// `rows` of the rows are the sequence's.  16 bytes per lane straight from the registers would touch 32 lines per
// store, so the rows pass through the warp's 2 KB at `stg` (XOR of the 16-byte chunks: no bank conflicts), from where
// four lanes write 64 bytes of one row.
template <bool F32>
__device__ __forceinline__ void store_rows32(const PromptArgs& a, uint8_t* stg, int64_t at, int32_t rows,
                                             const uint32_t (&ov)[32], float scale) {
  const int lane = threadIdx.x & 31, r0 = lane >> 2, c = lane & 3;
  auto put = [&](int h, uint4 x) {
    *reinterpret_cast<uint4*>(stg + lane * 64 + ((h ^ ((lane >> 1) & 3)) << 4)) = x;
  };
  auto copy = [&](uint8_t* dst, int64_t step) {  // dst: this lane's piece of row r0; step: bytes of 8 rows
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 8 * i;
      const uint4 x = *reinterpret_cast<const uint4*>(stg + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
      if (r < rows) *reinterpret_cast<uint4*>(dst + i * step) = x;
    }
    __syncwarp();
  };
  float o[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(ov[e]) * scale;
  const int64_t first = at + r0 * a.out_token;
  if constexpr (F32) {
#pragma unroll
    for (int f = 0; f < 2; ++f) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float* x = o + 16 * f + 4 * h;
        put(h, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])));
      }
      copy(static_cast<uint8_t*>(a.out) + (first + 16 * f + 4 * c) * 4, a.out_token * 32);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 4; ++h)
      put(h, make_uint4(pack_bf16x2(o[8 * h], o[8 * h + 1]), pack_bf16x2(o[8 * h + 2], o[8 * h + 3]),
                        pack_bf16x2(o[8 * h + 4], o[8 * h + 5]), pack_bf16x2(o[8 * h + 6], o[8 * h + 7])));
    copy(static_cast<uint8_t*>(a.out) + (first + 8 * c) * 2, a.out_token * 16);
  }
}

// Clears the status word and the item counter.  The prompt kernel is its programmatic dependent: it sets itself up
// and loads its first tiles meanwhile, and touches the two only after its wait.
__global__ void prompt_clear_kernel(uint32_t* words) {
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x < 2) words[threadIdx.x] = 0;
}

// Launches the kernel as the clearing kernel's dependent.
template <typename Kernel>
inline kvq_status launch_cleared(Kernel kern, const PromptArgs& a, int64_t grid, int threads, int smem,
                                 const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  prompt_clear_kernel<<<1, 32, 0, stream>>>(a.status);
  if (cudaGetLastError() != cudaSuccess) return KVQ_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, q, k, v) == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
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
