// kvq_api.cu -- the C ABI of libkvq: argument validation, the pool cost model, workspace sizing and
// kernel dispatch.  Every check runs on the host before any launch; a rejected call touches nothing.
//
// Cost model: "feat(kvcache): 8-bit KV cache (q8_0 / fp8_e4m3) behind --kv-cache-dtype", section "What"
// (1.0625 bytes per element: one code byte plus an fp16 scale per 32 elements) and its review comment's
// "End-to-end numbers" (the KV pool grows by 2 / 1.0625 at the same budget).  "feat(kvcache): 8-bit
// DSV4 window/compressed KV", section "One ordering trap": the budget must be priced with the same
// bytes-per-token the pool uses, which is why both come from this one function.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <limits>

#include "../../include/kvq.h"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr size_t kAlign = 16;

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) % kAlign) == 0; }

int n_kv_of(const kvq_layout& L) { return L.mla ? 1 : 2; }

kvq_status check_layout(const kvq_layout* L) {
  if (L == nullptr) return KVQ_EINVAL;
  if (L->num_pages < 0 || L->page_size <= 0 || L->num_kv_heads <= 0) return KVQ_EINVAL;
  if (L->mla != 0 && L->mla != 1) return KVQ_EINVAL;
  if (L->head_dim <= 0 || L->head_dim % 32 != 0) return KVQ_EHEADDIM;
  if (L->v_dim <= 0 || L->v_dim % 32 != 0) return KVQ_EHEADDIM;
  if (!L->mla && L->v_dim != L->head_dim) return KVQ_EINVAL;
  if (L->mla && L->v_dim > L->head_dim) return KVQ_EINVAL;
  // element count must fit comfortably in int64 / size_t
  const double elems = static_cast<double>(L->num_pages) * n_kv_of(*L) * L->num_kv_heads * L->page_size *
                       static_cast<double>(L->head_dim);
  if (elems > 4.0e18) return KVQ_EINVAL;
  return KVQ_OK;
}

bool kind_ok(int kind) { return kind == KVQ_FP8_E4M3 || kind == KVQ_Q8_0; }

// Kinds the attention entry points read: the block-scaled ones and the unscaled fp8 casts.
bool kind_read_ok(int kind) { return kind_ok(kind) || kind == KVQ_FP8_E4M3_UNSCALED || kind == KVQ_FP8_E5M2_UNSCALED; }

// Kinds that kvq_append writes: these and the one whose scale belongs to a page and head.
bool kind_append_ok(int kind) { return kind_read_ok(kind) || kind == KVQ_FP8_E4M3_PAGE; }

// The unscaled kinds have no scale array: their scales pointer is ignored (it may be NULL).
bool has_scales(int kind) { return kind_ok(kind) || kind == KVQ_FP8_E4M3_PAGE; }

// SMs of the current device (the MLA tensor-core plan targets one work item per SM).
int32_t sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      sms <= 0)
    return kTargetItems;
  return sms;
}

size_t elems_of(const kvq_layout& L) {
  return static_cast<size_t>(L.num_pages) * n_kv_of(L) * L.num_kv_heads * L.page_size * L.head_dim;
}

struct WorkspacePlan {
  int32_t path;
  int32_t split_align;
  int32_t target_items;
  int32_t heads_per_item;
  int32_t query_groups;
  int64_t max_items;
  size_t cnt_offset, acc_offset, ml_offset, tab_offset, total;
};

// 1 = CUDA-core kernel, 2 = tensor-core kernel, -1 = the requested path has no kernel for this shape.
// Automatic: tensor cores where QK^T and PV are dense enough -- 8..16 query heads per kv head, or an MLA
// pool read by a multiple of 64 query heads whose block tables can hold at least kMlaTcMinTokens tokens
// in all (the MLA tensor-core kernel costs ~50 us however short the contexts: at batch 1 it measured 54
// us at 256 and 1024 tokens against 21 and 58 us on the CUDA cores); the GQA tensor-core kernel also
// runs 1..7 heads (padded), but measured slower there than the CUDA cores.
constexpr int64_t kMlaTcMinTokens = 1024;

int32_t choose_path(const kvq_layout& L, int32_t batch, int32_t num_q_heads, int32_t max_pages,
                    const kvq_decode_options* opt) {
  const int32_t group = num_q_heads / L.num_kv_heads;
  const bool tc = L.mla ? decode_mla_tc_supported(L.head_dim, L.v_dim, L.mla, group, batch)
                        : decode_tc_supported(L.head_dim, L.v_dim, L.mla, group, batch);
  const bool cc = decode_cc_supported(L.head_dim, L.v_dim, L.mla);
  const int32_t want = opt ? opt->path : 0;
  if (want == 2) return tc ? 2 : -1;
  if (want == 1) return cc ? 1 : -1;
  const bool long_mla = static_cast<int64_t>(batch) * max_pages * kPageTokens >= kMlaTcMinTokens;
  if (tc && (L.mla ? long_mla : group >= 8)) return 2;
  return cc ? 1 : -1;
}

bool plan_workspace(const kvq_layout& L, int32_t batch, int32_t num_q_heads, int32_t max_pages,
                    const kvq_decode_options* opt, WorkspacePlan* w) {
  if (batch < 0 || num_q_heads <= 0 || max_pages <= 0) return false;
  if (num_q_heads % L.num_kv_heads != 0) return false;
  const int32_t group = num_q_heads / L.num_kv_heads;
  const int32_t pps = opt ? opt->pages_per_split : 0;
  if (pps < 0) return false;
  const int32_t path = choose_path(L, batch, num_q_heads, max_pages, opt);
  w->path = path;
  if (path == 2 && L.mla) w->heads_per_item = decode_mla_tc_heads_per_item(group);
  else w->heads_per_item = (path == 2) ? group : cc_heads_per_item(group, L.head_dim, L.mla);
  w->split_align = (path == 2) ? 8 : 1;
  // Tensor-core items are expensive to start and finish (a pipeline fill, a q tile, an O readout, and
  // partials the merge must read): the GQA kernel aims at about two items per SM, the MLA kernel
  // (64 query rows of 576, 64 x 512 partial outputs) at one.
  // CUDA-core items: a little under two waves of the resident CTAs, because each sequence's last split
  // is partial and rounds the count up (qwen3_1p7b: 1240 items against 2 x 608 slots at the full two
  // waves).
  w->target_items = (path == 2) ? (L.mla ? sm_count() : 2 * sm_count())
                                : std::max<int32_t>(64, 19 * cc_ctas_per_sm(L.head_dim, L.mla, w->heads_per_item) *
                                                            sm_count() / 10);
  w->query_groups = L.num_kv_heads * (group / w->heads_per_item);
  w->max_items = max_work_items(batch, w->query_groups, max_pages, pps, w->target_items);
  const size_t acc = static_cast<size_t>(w->max_items) * w->heads_per_item * L.v_dim * sizeof(float);
  const size_t ml = static_cast<size_t>(w->max_items) * w->heads_per_item * 2 * sizeof(float);
  // split counters of the fused merge (CUDA-core path) follow the header: one memset clears both
  const size_t cnt = static_cast<size_t>(batch) * w->query_groups * sizeof(int32_t);
  w->cnt_offset = kWorkspaceHeader;
  w->acc_offset = w->cnt_offset + ((cnt + 255) / 256) * 256;
  w->ml_offset = w->acc_offset + ((acc + 255) / 256) * 256;
  w->tab_offset = w->ml_offset + ((ml + 255) / 256) * 256;
  const size_t tab = static_cast<size_t>(batch) * 2 * sizeof(int32_t);
  w->total = w->tab_offset + ((tab + 255) / 256) * 256;
  return true;
}

}  // namespace

int64_t max_work_items(int32_t batch, int32_t query_groups, int32_t max_pages, int32_t pages_per_split,
                       int32_t target_items) {
  const int64_t per_seq = static_cast<int64_t>(query_groups);
  if (pages_per_split > 0)
    return static_cast<int64_t>(batch) * per_seq * ((max_pages + pages_per_split - 1) / pages_per_split);
  const int64_t upper = static_cast<int64_t>(batch) * per_seq * ((max_pages + kMinPagesPerSplit - 1) / kMinPagesPerSplit);
  return std::min<int64_t>(upper, static_cast<int64_t>(target_items) + static_cast<int64_t>(batch) * per_seq);
}

}  // namespace kvq

using namespace kvq;

namespace {

// Masks of the decode's sequences when they are the rows of drafted trees (kvq_tree).
struct TreeRows {
  const int64_t* mask;
  const int32_t* base;
  int32_t words;
};

kvq_status decode_common(const void* q, const void* pool, const void* scales, const int32_t* block_table,
                         int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                         float sm_scale, void* out, kvq_out_dtype out_dtype, void* workspace,
                         size_t workspace_bytes, const kvq_layout* layout, kvq_kind kind,
                         const kvq_decode_options* options, void* stream, bool clear_status,
                         const int32_t* bt_row = nullptr, const TreeRows* tree = nullptr) {
  kvq_status st = check_layout(layout);
  if (st != KVQ_OK) return st;
  if (!kind_read_ok(kind)) return KVQ_EKIND;
  if (!has_scales(kind)) scales = nullptr;
  if (out_dtype != KVQ_OUT_BF16 && out_dtype != KVQ_OUT_F32) return KVQ_EINVAL;
  if (batch < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0) return KVQ_EINVAL;
  if (num_q_heads % layout->num_kv_heads != 0) return KVQ_EINVAL;
  if (!(sm_scale == sm_scale) || sm_scale > std::numeric_limits<float>::max() ||
      sm_scale < -std::numeric_limits<float>::max())
    return KVQ_EINVAL;
  if (options && (options->pages_per_split < 0 || options->path < 0 || options->path > 2)) return KVQ_EINVAL;
  if (layout->page_size != kPageTokens) return KVQ_EUNSUPPORTED;
  WorkspacePlan w;
  if (!plan_workspace(*layout, batch, num_q_heads, max_pages_per_seq, options, &w)) return KVQ_EINVAL;
  if (w.path < 0) return KVQ_EUNSUPPORTED;
  if (batch == 0) return KVQ_OK;
  if (!q || !pool || (has_scales(kind) && !scales) || !block_table || !seq_lens || !out || !workspace)
    return KVQ_EINVAL;
  if (workspace_bytes < w.total) return KVQ_EWORKSPACE;
  if (!aligned(q) || !aligned(pool) || !aligned(scales) || !aligned(out) || !aligned(workspace) ||
      (reinterpret_cast<uintptr_t>(block_table) % 4) != 0 || (reinterpret_cast<uintptr_t>(seq_lens) % 4) != 0)
    return KVQ_EALIGN;
  st = kvq_device_check();
  if (st != KVQ_OK) return st;

  DecodeArgs a;
  a.q = q;
  a.codes = static_cast<const uint8_t*>(pool);
  a.scales = static_cast<const uint16_t*>(scales);
  a.block_table = block_table;
  a.bt_row = bt_row;
  a.num_pages = layout->num_pages;
  a.max_pages = max_pages_per_seq;
  a.seq_lens = seq_lens;
  a.tree_mask = tree ? tree->mask : nullptr;
  a.tree_base = tree ? tree->base : nullptr;
  a.tree_words = tree ? tree->words : 0;
  a.batch = batch;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = layout->num_kv_heads;
  a.head_dim = layout->head_dim;
  a.v_dim = layout->v_dim;
  a.mla = layout->mla;
  a.sm_scale = sm_scale;
  a.out = out;
  a.out_dtype = out_dtype;
  a.kind = kind;
  a.pages_per_split = options ? options->pages_per_split : 0;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.part_acc = reinterpret_cast<float*>(ws + w.acc_offset);
  a.part_ml = reinterpret_cast<float*>(ws + w.ml_offset);
  a.plan_tab = reinterpret_cast<int32_t*>(ws + w.tab_offset);
  a.split_cnt = (w.path == 1) ? reinterpret_cast<int32_t*>(ws + w.cnt_offset) : nullptr;
  a.max_items = w.max_items;
  a.heads_per_item = w.heads_per_item;
  a.split_align = w.split_align;
  a.target_items = w.target_items;
  // the GQA tensor-core kernel: one item per SM when the splits come out even (no second pipeline fill
  // and O readout per SM, half the partials to merge), else about two
  a.one_wave_items = (w.path == 2 && !layout->mla) ? sm_count() : 0;
  a.min_one_split = (w.path == 1) ? 1 : 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // status word and split counters (the counters only on the CUDA-core path, which merges in-kernel)
  // (a caller that already recorded errors in the status word, the sparse decode, keeps it)
  const size_t clear = (w.path == 1) ? w.acc_offset : sizeof(uint32_t);
  const size_t from = clear_status ? 0 : kWorkspaceHeader;
  if (clear > from && cudaMemsetAsync(ws + from, 0, clear - from, s) != cudaSuccess) return KVQ_ECUDA;
  if (w.path == 2) st = a.mla ? launch_decode_mla_tc(a, s) : launch_decode_tc(a, s);
  else return launch_decode_cc(a, s);
  if (st != KVQ_OK) return st;
  return launch_merge(a, w.query_groups, s);
}

// Sparse decode: the dense decode's workspace first (its status word at offset 0 is the call's), then
// the compact pool, its block table and its sequence lengths.  cpages = ceil(topk / 16) pages per
// sequence hold every column a list can select.
struct SparsePlan {
  kvq_layout compact;
  int32_t cpages;
  size_t dense_bytes, codes_offset, scales_offset, table_offset, lens_offset, total;
};

bool plan_sparse(const kvq_layout* layout, int32_t batch, int32_t num_q_heads, int32_t topk, SparsePlan* sp) {
  if (check_layout(layout) != KVQ_OK) return false;
  if (batch < 0 || num_q_heads <= 0 || topk < 0 || topk > kMaxSparseTopk) return false;
  if (num_q_heads % layout->num_kv_heads != 0) return false;
  sp->cpages = std::max<int32_t>(1, (topk + kPageTokens - 1) / kPageTokens);
  sp->compact = *layout;
  sp->compact.num_pages = static_cast<int64_t>(std::max<int32_t>(batch, 1)) * sp->cpages;
  WorkspacePlan w;
  if (!plan_workspace(sp->compact, batch, num_q_heads, sp->cpages, nullptr, &w)) return false;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t n_kv = layout->mla ? 1 : 2;
  const size_t rows = static_cast<size_t>(sp->compact.num_pages) * kPageTokens * n_kv * layout->num_kv_heads;
  sp->dense_bytes = up(w.total);
  sp->codes_offset = sp->dense_bytes;
  sp->scales_offset = sp->codes_offset + up(rows * layout->head_dim);
  sp->table_offset = sp->scales_offset + up(rows * (layout->head_dim / 32) * sizeof(uint16_t));
  sp->lens_offset = sp->table_offset + up(static_cast<size_t>(sp->compact.num_pages) * sizeof(int32_t));
  sp->total = sp->lens_offset + up(static_cast<size_t>(std::max<int32_t>(batch, 1)) * sizeof(int32_t));
  return true;
}

// Extend by prefixes: every new token is a sequence of its own (its causal prefix, the block-table row of the
// sequence it belongs to), decoded in chunks of at most kExtendChunk tokens by the decode kernels.  This is
// how the MLA latent row is extended, and the GQA path when the flash kernel cannot serve the shape or the
// caller asks for fp32 probabilities.  Workspace: the decode workspace of one chunk (its status word at
// offset 0 is the call's), then the per-token prefix lengths and block-table rows.
constexpr int32_t kExtendChunk = 1024;

struct ExtendPlan {
  bool flash;              // the GQA flash-style tcgen05 kernel (else: prefixes through the decode kernels)
  bool split;              // the flash kernel feeds P as two bf16 terms
  kvq_decode_options dec;  // the decode kernel choice of the prefix path
  int32_t chunk;
  size_t dense_bytes, lens_offset, rows_offset, total;
};

// The extend's kernel choice and workspace.  False: invalid sizes or options, or no kernel for the shape.
bool plan_extend(const kvq_layout& L, int32_t total_q, int32_t num_q_heads, int32_t max_pages,
                 const kvq_extend_options* o, ExtendPlan* ep) {
  const int32_t path = o ? o->path : 0;
  const bool precise = o && o->precise_p != 0;
  if (path < 0 || path > 2 || total_q < 0 || num_q_heads <= 0 || max_pages <= 0) return false;
  if (num_q_heads % L.num_kv_heads != 0) return false;
  const int32_t group = num_q_heads / L.num_kv_heads;
  // the batch bound is checked per call; any batch up to it gives the same choice
  const bool flash_ok = extend_tc_supported(L.head_dim, L.v_dim, L.mla, group, 1);
  ep->flash = !L.mla && (path == 2 || (path == 0 && flash_ok));
  ep->split = ep->flash && precise;
  ep->dec.pages_per_split = 0;
  ep->dec.path = path == 1 ? 1 : (path == 2 ? 2 : 0);
  if (!ep->flash && precise) {
    if (path == 2) return false;  // the tensor-core decode keeps P in bf16
    ep->dec.path = 1;
  }
  if (ep->flash) {
    ep->chunk = 0;
    ep->dense_bytes = ep->lens_offset = ep->rows_offset = ep->total = kWorkspaceHeader;
    return flash_ok;
  }
  ep->chunk = std::max<int32_t>(1, std::min<int32_t>(total_q, kExtendChunk));
  WorkspacePlan w;
  if (!plan_workspace(L, ep->chunk, num_q_heads, max_pages, &ep->dec, &w) || w.path < 0) return false;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t n = static_cast<size_t>(std::max<int32_t>(total_q, 1)) * sizeof(int32_t);
  ep->dense_bytes = up(w.total);
  ep->lens_offset = ep->dense_bytes;
  ep->rows_offset = ep->lens_offset + up(n);
  ep->total = ep->rows_offset + up(n);
  return true;
}

kvq_status extend_prefixes(const ExtendPlan& ep, const void* q, const void* pool, const void* scales,
                           const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* seq_lens,
                           const int32_t* q_start, int32_t total_q, int32_t batch, int32_t num_q_heads, float sm_scale,
                           void* out, kvq_out_dtype out_dtype, void* workspace, const kvq_layout* layout,
                           kvq_kind kind, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* vlens = reinterpret_cast<int32_t*>(ws + ep.lens_offset);
  int32_t* vrow = reinterpret_cast<int32_t*>(ws + ep.rows_offset);
  // rows no sequence covers (an inconsistent q_start) keep length 0: zeros out
  if (cudaMemsetAsync(ws + ep.lens_offset, 0, ep.total - ep.lens_offset, s) != cudaSuccess) return KVQ_ECUDA;
  kvq_status st =
      launch_extend_expand(q_start, seq_lens, batch, total_q, vlens, vrow, reinterpret_cast<uint32_t*>(ws), s);
  if (st != KVQ_OK) return st;
  const size_t q_row = static_cast<size_t>(num_q_heads) * layout->head_dim * 2;
  const size_t o_row = static_cast<size_t>(num_q_heads) * layout->v_dim * (out_dtype == KVQ_OUT_F32 ? 4 : 2);
  for (int32_t c0 = 0; c0 < total_q; c0 += ep.chunk) {
    const int32_t n = std::min<int32_t>(ep.chunk, total_q - c0);
    st = decode_common(static_cast<const uint8_t*>(q) + c0 * q_row, pool, scales, block_table, max_pages_per_seq,
                       vlens + c0, n, num_q_heads, sm_scale, static_cast<uint8_t*>(out) + c0 * o_row, out_dtype,
                       workspace, ep.dense_bytes, layout, kind, &ep.dec, s, false, vrow + c0);
    if (st != KVQ_OK) return st;
  }
  return KVQ_OK;
}

// Attention of drafted tokens: the split-K flash kernel (GQA, head_dim 128 and 256), else every drafted token is
// a sequence of its own to the decode kernels, in chunks, with its mask.
struct TreePlan {
  bool flash;
  kvq_decode_options dec;
  int32_t chunk, grid;
  size_t tab_offset, seq_offset, st_offset, acc_offset, ml_offset;   // flash
  size_t dense_bytes, lens_offset, rows_offset, base_offset, total;  // rows through the decode kernels
};

bool plan_tree(const kvq_layout& L, int32_t batch, int32_t total_q, int32_t num_q_heads, int32_t max_pages, int32_t path,
               TreePlan* tp) {
  if (path < 0 || path > 2 || batch < 0 || total_q < 0 || num_q_heads <= 0 || max_pages <= 0 || max_pages > kMaxTreePages) return false;
  if (num_q_heads % L.num_kv_heads != 0) return false;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int64_t G = num_q_heads / L.num_kv_heads;
  // units (tiles of at least 64 keys, for blocks of 128 rows) and merge CTAs are counted in 32 bits
  // (for any q_start, consistent or not: at most 64 * kMaxMaskWords drafted tokens a sequence)
  const double units = static_cast<double>(batch) * (64.0 * kMaxMaskWords * G / 128 + 1) * L.num_kv_heads *
                       (static_cast<double>(max_pages) * L.page_size / 64 + 1);
  const bool flash_ok = tree_tc_supported(L.head_dim, L.v_dim, L.mla, batch) && units < 2.0e9 &&
                        static_cast<double>(total_q) * num_q_heads < 2.0e9;
  tp->flash = !L.mla && path != 1 && flash_ok;
  if (!L.mla && path == 2 && !flash_ok) return false;
  if (tp->flash) {
    tp->grid = sm_count();
    const size_t slots = 2 * static_cast<size_t>(tp->grid) * 128;
    tp->tab_offset = kWorkspaceHeader;
    tp->seq_offset = tp->tab_offset + up((static_cast<size_t>(batch) + 2) * sizeof(int32_t));
    tp->st_offset = tp->seq_offset + up(static_cast<size_t>(total_q) * sizeof(int32_t));
    tp->ml_offset = tp->st_offset + up(static_cast<size_t>(tp->grid) * sizeof(uint32_t));
    tp->acc_offset = tp->ml_offset + up(slots * 2 * sizeof(float));
    tp->total = tp->acc_offset + up(slots * L.head_dim * sizeof(float));
    return true;
  }
  tp->dec.pages_per_split = 0;
  tp->dec.path = L.mla ? path : 1;  // (the GQA tensor-core decode has no masks)
  tp->chunk = std::max<int32_t>(1, std::min<int32_t>(total_q, kExtendChunk));
  WorkspacePlan w;
  if (!plan_workspace(L, tp->chunk, num_q_heads, max_pages, &tp->dec, &w) || w.path < 0) return false;
  const size_t n = static_cast<size_t>(std::max<int32_t>(total_q, 1)) * sizeof(int32_t);
  tp->dense_bytes = up(w.total);
  tp->lens_offset = tp->dense_bytes;
  tp->base_offset = tp->lens_offset + up(n);
  tp->rows_offset = tp->base_offset + up(n);
  tp->total = tp->rows_offset + up(n);
  return true;
}

// Attention over a KVQ_FP8_E4M3_PAGE cache: the kernel and what joins its runs.  max_bytes caps the workspace, and
// with it the CTAs (0: no cap).
struct PagePlan {
  bool flash;  // the kernel for many query rows
  int32_t grid, tile;
  size_t ml_offset, acc_offset, total;
};

bool plan_page(const kvq_layout& L, int32_t batch, int32_t total_q, int32_t num_q_heads, int32_t max_pages,
               size_t max_bytes, PagePlan* pp) {
  if (batch < 0 || total_q < 0 || num_q_heads <= 0 || max_pages <= 0 || num_q_heads % L.num_kv_heads != 0) return false;
  if (L.mla || L.page_size != kPageTokens || !page_supported(L.head_dim)) return false;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  // A tile of the rows kernel holds a sequence's rows of a kv head, or the call is small for it, or the flash kernel takes
  // it, which starts and joins more slowly but reads K and V once for 256 rows instead of 16.  Small: as the table's width has it,
  // since lengths are not known here.  With 8 / 2 heads of 128 over 2048 tokens (rows kernel, flash kernel): 32 new
  // tokens, 2080 units, 29 and 41 us; 128 tokens, 8700 units, 39 and 47 us; over 8192 tokens 64 and 128 new ones, 16500 and
  // 33300 units, 47 and 49, 62 and 49 us; 32 / 8 heads over 512 tokens, 64 new ones, 4600 units, 37 and 31 us.
  const double rows = static_cast<double>(total_q) * (num_q_heads / L.num_kv_heads);
  pp->flash = total_q > batch && rows > static_cast<double>(kPageRowsTile) * batch &&
              rows / kPageRowsTile * L.num_kv_heads * max_pages > kPageRowsUnits;
  const int32_t tile = pp->tile = pp->flash ? page_flash_rows(L.head_dim) : rows <= 8.0 * batch ? 8 : kPageRowsTile;
  const int32_t least = pp->flash ? kPageFlashUnits : kPageMinUnits;
  const size_t slot = tile * (static_cast<size_t>(L.head_dim) + 2) * sizeof(float);
  // units of work at most: pages of tiles of 16 rows, or tiles of 64 keys or more of items (of half their rows at least)
  const double tiles = batch + rows / (pp->flash ? tile / 4 : tile) + (pp->flash ? total_q : 0);
  const double units = tiles * L.num_kv_heads * (pp->flash ? max_pages / 4 + 1.0 + kPageItemUnits : max_pages);
  if (units > 1e14) return false;  // (units times CTAs are counted in 64 bits)
  int64_t grid = pp->flash ? sm_count() : page_rows_grid(L.head_dim, tile, sm_count());
  if (units < static_cast<double>(grid) * least) grid = static_cast<int64_t>(units / least) + 1;
  if (max_bytes > 0) {
    if (max_bytes < kWorkspaceHeader + 1024) return false;
    grid = std::min<int64_t>(grid, (max_bytes - kWorkspaceHeader - 1024) / (2 * slot + kPageRunBytes));
  }
  if (grid < 1) return false;
  const size_t slots = 2 * static_cast<size_t>(grid);
  pp->grid = static_cast<int32_t>(grid);
  pp->ml_offset = kWorkspaceHeader + up(static_cast<size_t>(grid) * kPageRunBytes);
  pp->acc_offset = pp->ml_offset + up(slots * tile * 2 * sizeof(float));
  pp->total = pp->acc_offset + up(slots * tile * L.head_dim * sizeof(float));
  return true;
}

// q_start null: one row per sequence (kvq_decode).  The host's checks that the kinds share are done.
kvq_status page_common(const void* q, const void* pool, const void* scales, const int32_t* block_table, int32_t max_pages,
                       const int32_t* seq_lens, const int32_t* q_start, int32_t total_q, int32_t batch,
                       int32_t num_q_heads, float sm_scale, void* out, kvq_out_dtype out_dtype, void* workspace,
                       size_t workspace_bytes, const kvq_layout* layout, bool cap, cudaStream_t s) {
  if (layout->mla || layout->page_size != kPageTokens || !page_supported(layout->head_dim)) return KVQ_EUNSUPPORTED;
  if (static_cast<int64_t>(max_pages) * kPageTokens > std::numeric_limits<int32_t>::max()) return KVQ_EINVAL;
  if (static_cast<int64_t>(total_q) * num_q_heads > std::numeric_limits<int32_t>::max()) return KVQ_EUNSUPPORTED;
  PagePlan pp;
  if (!plan_page(*layout, batch, total_q, num_q_heads, max_pages, cap ? workspace_bytes : 0, &pp))
    return cap ? KVQ_EWORKSPACE : KVQ_EINVAL;
  const bool empty = batch == 0 || total_q == 0;
  if (!workspace) return empty && q_start == nullptr ? KVQ_OK : KVQ_EINVAL;
  if (workspace_bytes < pp.total) return KVQ_EWORKSPACE;
  if (!empty && (!q || !pool || !scales || !block_table || !seq_lens || !out)) return KVQ_EINVAL;
  if (!aligned(workspace) || !aligned(q) || !aligned(pool) || !aligned(scales) || !aligned(out)) return KVQ_EALIGN;
  for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(q_start)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return KVQ_EALIGN;
  const kvq_status st = kvq_device_check();
  if (st != KVQ_OK) return st;
  if (empty) return cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PageArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.codes = static_cast<const uint8_t*>(pool);
  a.scales = static_cast<const float*>(scales);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.q_start = q_start;
  a.out = out;
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.total = reinterpret_cast<int64_t*>(ws + 64);
  a.runs = ws + kWorkspaceHeader;
  a.part_ml = reinterpret_cast<float*>(ws + pp.ml_offset);
  a.part_acc = reinterpret_cast<float*>(ws + pp.acc_offset);
  a.num_pages = layout->num_pages;
  a.max_pages = max_pages;
  a.batch = batch;
  a.total_q = total_q;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = layout->num_kv_heads;
  a.head_dim = layout->head_dim;
  a.grid = pp.grid;
  a.tile = pp.tile;
  a.score_scale = sm_scale * 1.4426950408889634f;  // log2(e)
  a.out_dtype = out_dtype;
  return pp.flash ? launch_page_flash(a, s) : launch_page_rows(a, s);
}

kvq_status page_decode(const void* q, const void* pool, const void* scales, const int32_t* block_table, int32_t max_pages,
                       const int32_t* seq_lens, int32_t batch, int32_t num_q_heads, float sm_scale, void* out,
                       kvq_out_dtype out_dtype, void* workspace, size_t workspace_bytes, const kvq_layout* layout,
                       const kvq_decode_options* options, bool cap, void* stream) {
  const kvq_status st = check_layout(layout);
  if (st != KVQ_OK) return st;
  if (out_dtype != KVQ_OUT_BF16 && out_dtype != KVQ_OUT_F32) return KVQ_EINVAL;
  if (batch < 0 || num_q_heads <= 0 || max_pages <= 0) return KVQ_EINVAL;
  if (num_q_heads % layout->num_kv_heads != 0) return KVQ_EINVAL;
  if (!(sm_scale == sm_scale) || sm_scale > std::numeric_limits<float>::max() ||
      sm_scale < -std::numeric_limits<float>::max())
    return KVQ_EINVAL;
  if (options && (options->pages_per_split < 0 || options->path < 0 || options->path > 2)) return KVQ_EINVAL;
  if (options && (options->pages_per_split > 0 || options->path > 0)) return KVQ_EUNSUPPORTED;
  return page_common(q, pool, scales, block_table, max_pages, seq_lens, nullptr, batch, batch, num_q_heads, sm_scale, out,
                     out_dtype, workspace, workspace_bytes, layout, cap, static_cast<cudaStream_t>(stream));
}

// Workspace of a fork or a resize of n list entries: the status word, the entries, the free pages' bitmap with
// its prefixes, and the parents' rows.
struct PagesPlan {
  int32_t chunks;
  size_t entries, chunk_free, word_prefix, bits, rows, total;
};

bool plan_pages(const kvq_layout& L, int32_t n, int32_t max_pages, PagesPlan* pp) {
  if (n < 0 || n > kMaxPagesList || max_pages <= 0 || max_pages > kMaxPagesCols) return false;
  const int64_t chunks = (L.num_pages + kPagesChunk - 1) / kPagesChunk;
  if (chunks > kMaxPagesChunks) return false;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t words = static_cast<size_t>(chunks) * (kPagesChunk / 32);
  pp->chunks = static_cast<int32_t>(chunks);
  pp->entries = kWorkspaceHeader;
  pp->chunk_free = pp->entries + up(static_cast<size_t>(n) * sizeof(PagesEntry));
  pp->word_prefix = pp->chunk_free + up(static_cast<size_t>(chunks) * sizeof(int32_t));
  pp->bits = pp->word_prefix + up(words * sizeof(int32_t));
  pp->rows = pp->bits + up(words * sizeof(uint32_t));
  pp->total = pp->rows + up(static_cast<size_t>(n) * max_pages * sizeof(int32_t));
  return true;
}

// Checks and arguments that fork and resize share; KVQ_OK with a->n = 0 when there is nothing to do.
kvq_status pages_common(int32_t* block_table, int32_t max_pages, int32_t* seq_lens, int32_t batch, int32_t* page_refs,
                        const int32_t* dst, int32_t n, void* workspace, size_t workspace_bytes,
                        const kvq_layout* layout, PagesArgs* a) {
  kvq_status st = check_layout(layout);
  if (st != KVQ_OK) return st;
  if (batch < 0 || n < 0 || max_pages <= 0) return KVQ_EINVAL;
  if (static_cast<int64_t>(max_pages) * layout->page_size > std::numeric_limits<int32_t>::max()) return KVQ_EINVAL;
  PagesPlan pp;
  if (!plan_pages(*layout, n, max_pages, &pp)) return KVQ_EUNSUPPORTED;
  a->n = 0;
  if (n > 0 && (!block_table || !seq_lens || (!page_refs && layout->num_pages > 0) || !dst)) return KVQ_EINVAL;
  if (!workspace) return KVQ_EINVAL;
  if (workspace_bytes < pp.total) return KVQ_EWORKSPACE;
  if (!aligned(workspace)) return KVQ_EALIGN;
  for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(page_refs), static_cast<const void*>(dst)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return KVQ_EALIGN;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a->block_table = block_table;
  a->seq_lens = seq_lens;
  a->page_refs = page_refs;
  a->src = nullptr;
  a->dst = dst;
  a->new_lens = nullptr;
  a->copy_src = a->copy_dst = nullptr;
  a->batch = batch;
  a->max_pages = max_pages;
  a->n = n;
  a->page_size = layout->page_size;
  a->chunks = pp.chunks;
  a->num_pages = layout->num_pages;
  a->status = reinterpret_cast<uint32_t*>(ws);
  a->entries = reinterpret_cast<PagesEntry*>(ws + pp.entries);
  a->chunk_free = reinterpret_cast<int32_t*>(ws + pp.chunk_free);
  a->word_prefix = reinterpret_cast<int32_t*>(ws + pp.word_prefix);
  a->bits = reinterpret_cast<uint32_t*>(ws + pp.bits);
  a->rows = reinterpret_cast<int32_t*>(ws + pp.rows);
  return KVQ_OK;
}

bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return b != nullptr && x < y + b_bytes && y < x + a_bytes;
}

// The status word of a page call with an empty list.
kvq_status clear_status(void* workspace, cudaStream_t s) {
  return cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
}

}  // namespace

namespace kvq {
kvq_status decode_pages_capped(const void* q, const void* pool, const void* scales, const int32_t* block_table,
                               int32_t max_pages, const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                               float sm_scale, void* out, kvq_out_dtype out_dtype, void* workspace, size_t workspace_bytes,
                               const kvq_layout* layout, void* stream) {
  return page_decode(q, pool, scales, block_table, max_pages, seq_lens, batch, num_q_heads, sm_scale, out, out_dtype,
                     workspace, workspace_bytes, layout, nullptr, true, stream);
}
}  // namespace kvq

extern "C" {

const char* kvq_version(void) { return "0.1.0"; }

const char* kvq_strerror(kvq_status s) {
  switch (s) {
    case KVQ_OK: return "ok";
    case KVQ_EINVAL: return "invalid argument";
    case KVQ_EKIND:
      return "quantization kind not accepted by this call (the block-scaled stores take KVQ_FP8_E4M3 or KVQ_Q8_0; "
             "kvq_store_unscaled the unscaled kinds; the attention calls all four; KVQ_FP8_E4M3_PAGE belongs to kvq_append, "
             "kvq_decode, kvq_extend and kvq_pages_copy)";
    case KVQ_EHEADDIM: return "head_dim and v_dim must be positive multiples of 32 (the quantization block)";
    case KVQ_EALIGN: return "device pointers must be 16-byte aligned";
    case KVQ_EWORKSPACE: return "workspace smaller than kvq_decode_workspace_bytes()";
    case KVQ_EARCH: return "current device is not compute capability 10.3 (GB300, sm_103a)";
    case KVQ_ECUDA: return "a CUDA call or kernel launch failed";
    case KVQ_EUNSUPPORTED: return "no decode kernel for this page size / head_dim / path";
    case KVQ_ETIMEOUT: return "a kernel gave up a bounded wait; its output is not valid";
    case KVQ_ENOPAGES: return "not enough free pages; the call changed nothing";
  }
  return "unknown status";
}

size_t kvq_pool_bytes(const kvq_layout* layout) {
  if (check_layout(layout) != KVQ_OK) return 0;
  return elems_of(*layout);
}

size_t kvq_scale_bytes(const kvq_layout* layout) {
  if (check_layout(layout) != KVQ_OK) return 0;
  return elems_of(*layout) / 32 * 2;
}

double kvq_bytes_per_token(const kvq_layout* layout) {
  if (check_layout(layout) != KVQ_OK) return -1.0;
  const double elems = static_cast<double>(n_kv_of(*layout)) * layout->num_kv_heads * layout->head_dim;
  return elems + elems / 32.0 * 2.0;
}

int64_t kvq_num_pages(const kvq_layout* layout, size_t budget_bytes) {
  if (check_layout(layout) != KVQ_OK) return -1;
  const uint64_t elems_per_page =
      static_cast<uint64_t>(n_kv_of(*layout)) * layout->num_kv_heads * layout->page_size * layout->head_dim;
  const uint64_t bytes_per_page = elems_per_page + elems_per_page / 32 * 2;
  return static_cast<int64_t>(budget_bytes / bytes_per_page);
}

double kvq_bytes_per_token_ex(const kvq_layout* layout, kvq_kind kind) {
  if (check_layout(layout) != KVQ_OK || !kind_append_ok(kind)) return -1.0;
  if (kind_ok(kind)) return kvq_bytes_per_token(layout);
  const double rows = static_cast<double>(n_kv_of(*layout)) * layout->num_kv_heads;
  return rows * layout->head_dim + (kind == KVQ_FP8_E4M3_PAGE ? rows * sizeof(float) / layout->page_size : 0.0);
}

int64_t kvq_num_pages_ex(const kvq_layout* layout, kvq_kind kind, size_t budget_bytes) {
  if (check_layout(layout) != KVQ_OK || !kind_append_ok(kind)) return -1;
  if (kind_ok(kind)) return kvq_num_pages(layout, budget_bytes);
  const uint64_t rows = static_cast<uint64_t>(n_kv_of(*layout)) * layout->num_kv_heads;
  const uint64_t bytes_per_page =
      rows * layout->page_size * layout->head_dim + (kind == KVQ_FP8_E4M3_PAGE ? rows * sizeof(float) : 0);
  return static_cast<int64_t>(budget_bytes / bytes_per_page);
}

kvq_status kvq_device_check(void) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ECUDA;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return KVQ_ECUDA;
  if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) return KVQ_ECUDA;
  if (major != 10 || minor != 3) return KVQ_EARCH;
  return KVQ_OK;
}

kvq_status kvq_store(void* pool, void* scales, const void* k, const void* v, const int64_t* slot_mapping,
                     int64_t num_tokens, const kvq_layout* layout, kvq_kind kind, void* stream) {
  kvq_status st = check_layout(layout);
  if (st != KVQ_OK) return st;
  if (!kind_ok(kind)) return KVQ_EKIND;
  if (num_tokens < 0) return KVQ_EINVAL;
  if (layout->mla ? (v != nullptr) : false) return KVQ_EINVAL;
  if (num_tokens == 0) return KVQ_OK;
  if (!pool || !scales || !k || !slot_mapping || (!layout->mla && !v)) return KVQ_EINVAL;
  if (!aligned(pool) || !aligned(scales) || !aligned(k) || (v && !aligned(v)) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) % 8) != 0)
    return KVQ_EALIGN;
  st = kvq_device_check();
  if (st != KVQ_OK) return st;
  return launch_store(pool, scales, k, v, slot_mapping, num_tokens, *layout, kind,
                      static_cast<cudaStream_t>(stream));
}

int32_t kvq_decode_path(const kvq_layout* layout, int32_t batch, int32_t num_q_heads, int32_t max_pages_per_seq,
                        const kvq_decode_options* options) {
  if (check_layout(layout) != KVQ_OK) return KVQ_EINVAL;
  if (batch < 0 || num_q_heads <= 0 || num_q_heads % layout->num_kv_heads != 0) return KVQ_EINVAL;
  if (max_pages_per_seq <= 0) return KVQ_EINVAL;
  if (options && (options->pages_per_split < 0 || options->path < 0 || options->path > 2)) return KVQ_EINVAL;
  if (layout->page_size != kPageTokens) return KVQ_EUNSUPPORTED;
  const int32_t path = choose_path(*layout, batch, num_q_heads, max_pages_per_seq, options);
  return path < 0 ? static_cast<int32_t>(KVQ_EUNSUPPORTED) : path;
}

size_t kvq_decode_workspace_bytes_ex(const kvq_layout* layout, int32_t batch, int32_t num_q_heads,
                                     int32_t max_pages_per_seq, const kvq_decode_options* options) {
  if (check_layout(layout) != KVQ_OK) return 0;
  WorkspacePlan w;
  if (!plan_workspace(*layout, batch, num_q_heads, max_pages_per_seq, options, &w)) return 0;
  return w.total;
}

size_t kvq_decode_workspace_bytes(const kvq_layout* layout, int32_t batch, int32_t num_q_heads,
                                  int32_t max_pages_per_seq) {
  return kvq_decode_workspace_bytes_ex(layout, batch, num_q_heads, max_pages_per_seq, nullptr);
}

kvq_status kvq_decode_ex(const void* q, const void* pool, const void* scales, const int32_t* block_table,
                         int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                         float sm_scale, void* out, kvq_out_dtype out_dtype, void* workspace,
                         size_t workspace_bytes, const kvq_layout* layout, kvq_kind kind,
                         const kvq_decode_options* options, void* stream) {
  if (kind == KVQ_FP8_E4M3_PAGE)
    return page_decode(q, pool, scales, block_table, max_pages_per_seq, seq_lens, batch, num_q_heads, sm_scale, out,
                       out_dtype, workspace, workspace_bytes, layout, options, false, stream);
  return decode_common(q, pool, scales, block_table, max_pages_per_seq, seq_lens, batch, num_q_heads, sm_scale, out,
                       out_dtype, workspace, workspace_bytes, layout, kind, options, stream, true);
}

kvq_status kvq_decode(const void* q, const void* pool, const void* scales, const int32_t* block_table,
                      int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                      float sm_scale, void* out, kvq_out_dtype out_dtype, void* workspace, size_t workspace_bytes,
                      const kvq_layout* layout, kvq_kind kind, void* stream) {
  return kvq_decode_ex(q, pool, scales, block_table, max_pages_per_seq, seq_lens, batch, num_q_heads, sm_scale, out,
                       out_dtype, workspace, workspace_bytes, layout, kind, nullptr, stream);
}

size_t kvq_decode_workspace_bytes_kind(const kvq_layout* layout, kvq_kind kind, int32_t batch, int32_t num_q_heads,
                                       int32_t max_pages_per_seq, const kvq_decode_options* options) {
  if (check_layout(layout) != KVQ_OK) return 0;
  if (kind_read_ok(kind)) return kvq_decode_workspace_bytes_ex(layout, batch, num_q_heads, max_pages_per_seq, options);
  PagePlan pp;
  if (kind != KVQ_FP8_E4M3_PAGE || (options && (options->pages_per_split != 0 || options->path != 0)) ||
      !plan_page(*layout, batch, batch, num_q_heads, max_pages_per_seq, 0, &pp))
    return 0;
  return pp.total;
}

size_t kvq_decode_sparse_workspace_bytes(const kvq_layout* layout, int32_t batch, int32_t num_q_heads, int32_t topk) {
  SparsePlan sp;
  if (!plan_sparse(layout, batch, num_q_heads, topk, &sp)) return 0;
  return sp.total;
}

kvq_status kvq_decode_sparse(const void* q, const void* pool, const void* scales, const int32_t* block_table,
                             int32_t max_pages_per_seq, const int32_t* seq_lens, const int32_t* indices, int32_t topk,
                             int32_t batch, int32_t num_q_heads, float sm_scale, void* out, kvq_out_dtype out_dtype,
                             void* workspace, size_t workspace_bytes, const kvq_layout* layout, kvq_kind kind,
                             void* stream) {
  kvq_status st = check_layout(layout);
  if (st != KVQ_OK) return st;
  if (!kind_read_ok(kind)) return KVQ_EKIND;
  if (!has_scales(kind)) scales = nullptr;
  if (out_dtype != KVQ_OUT_BF16 && out_dtype != KVQ_OUT_F32) return KVQ_EINVAL;
  if (max_pages_per_seq <= 0) return KVQ_EINVAL;
  SparsePlan sp;
  if (!plan_sparse(layout, batch, num_q_heads, topk, &sp)) return KVQ_EINVAL;
  if (layout->page_size != kPageTokens || layout->head_dim % 64 != 0) return KVQ_EUNSUPPORTED;
  if (batch == 0) return KVQ_OK;
  if (!q || !pool || (has_scales(kind) && !scales) || !block_table || !seq_lens || (topk > 0 && !indices) || !out ||
      !workspace)
    return KVQ_EINVAL;
  if (workspace_bytes < sp.total) return KVQ_EWORKSPACE;
  if (!aligned(pool) || !aligned(scales) || !aligned(workspace) || (reinterpret_cast<uintptr_t>(block_table) % 4) != 0 ||
      (reinterpret_cast<uintptr_t>(seq_lens) % 4) != 0 || (reinterpret_cast<uintptr_t>(indices) % 4) != 0)
    return KVQ_EALIGN;
  st = kvq_device_check();
  if (st != KVQ_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(ws, 0, sizeof(uint32_t), s) != cudaSuccess) return KVQ_ECUDA;
  SparseGatherArgs g;
  g.codes = static_cast<const uint8_t*>(pool);
  g.scales = static_cast<const uint16_t*>(scales);
  g.block_table = block_table;
  g.seq_lens = seq_lens;
  g.indices = indices;
  g.dst_codes = ws + sp.codes_offset;
  g.dst_scales = has_scales(kind) ? reinterpret_cast<uint16_t*>(ws + sp.scales_offset) : nullptr;
  g.dst_table = reinterpret_cast<int32_t*>(ws + sp.table_offset);
  g.dst_lens = reinterpret_cast<int32_t*>(ws + sp.lens_offset);
  g.status = reinterpret_cast<uint32_t*>(ws);
  g.num_pages = layout->num_pages;
  g.max_pages = max_pages_per_seq;
  g.batch = batch;
  g.topk = topk;
  g.cpages = sp.cpages;
  g.n_kv = layout->mla ? 1 : 2;
  g.Hkv = layout->num_kv_heads;
  g.D = layout->head_dim;
  st = launch_sparse_gather(g, s);
  if (st != KVQ_OK) return st;
  return decode_common(q, g.dst_codes, g.dst_scales, g.dst_table, sp.cpages, g.dst_lens, batch, num_q_heads, sm_scale,
                       out, out_dtype, workspace, sp.dense_bytes, &sp.compact, kind, nullptr, stream, false);
}

size_t kvq_extend_workspace_bytes(void) { return kWorkspaceHeader; }

size_t kvq_extend_workspace_bytes_ex(const kvq_layout* layout, int32_t total_q, int32_t num_q_heads,
                                     int32_t max_pages_per_seq, const kvq_extend_options* options) {
  if (check_layout(layout) != KVQ_OK || layout->page_size != kPageTokens) return 0;
  ExtendPlan ep;
  if (!plan_extend(*layout, total_q, num_q_heads, max_pages_per_seq, options, &ep)) return 0;
  return ep.total;
}

size_t kvq_extend_workspace_bytes_kind(const kvq_layout* layout, kvq_kind kind, int32_t batch, int32_t total_q,
                                       int32_t num_q_heads, int32_t max_pages_per_seq, const kvq_extend_options* options) {
  if (check_layout(layout) != KVQ_OK) return 0;
  if (kind_read_ok(kind))
    return kvq_extend_workspace_bytes_ex(layout, total_q, num_q_heads, max_pages_per_seq, options);
  PagePlan pp;
  if (kind != KVQ_FP8_E4M3_PAGE || (options && (options->path != 0 || options->precise_p != 0)) ||
      !plan_page(*layout, batch, total_q, num_q_heads, max_pages_per_seq, 0, &pp))
    return 0;
  return pp.total;
}

int32_t kvq_extend_path(const kvq_layout* layout, int32_t total_q, int32_t num_q_heads, int32_t max_pages_per_seq,
                        const kvq_extend_options* options) {
  if (check_layout(layout) != KVQ_OK) return KVQ_EINVAL;
  if (total_q < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 || num_q_heads % layout->num_kv_heads != 0)
    return KVQ_EINVAL;
  if (options && (options->path < 0 || options->path > 2)) return KVQ_EINVAL;
  if (layout->page_size != kPageTokens) return KVQ_EUNSUPPORTED;
  ExtendPlan ep;
  if (!plan_extend(*layout, total_q, num_q_heads, max_pages_per_seq, options, &ep)) return KVQ_EUNSUPPORTED;
  if (ep.flash) return ep.split ? 4 : 3;
  WorkspacePlan w;
  plan_workspace(*layout, ep.chunk, num_q_heads, max_pages_per_seq, &ep.dec, &w);
  return w.path;
}

kvq_status kvq_extend(const void* q, const void* pool, const void* scales, const int32_t* block_table,
                      int32_t max_pages_per_seq, const int32_t* seq_lens, const int32_t* q_start, int32_t total_q,
                      int32_t batch, int32_t num_q_heads, float sm_scale, void* out, kvq_out_dtype out_dtype,
                      void* workspace, size_t workspace_bytes, const kvq_layout* layout, kvq_kind kind, void* stream) {
  return kvq_extend_ex(q, pool, scales, block_table, max_pages_per_seq, seq_lens, q_start, total_q, batch,
                       num_q_heads, sm_scale, out, out_dtype, workspace, workspace_bytes, layout, kind, nullptr,
                       stream);
}

kvq_status kvq_extend_ex(const void* q, const void* pool, const void* scales, const int32_t* block_table,
                         int32_t max_pages_per_seq, const int32_t* seq_lens, const int32_t* q_start,
                         int32_t total_q, int32_t batch, int32_t num_q_heads, float sm_scale, void* out,
                         kvq_out_dtype out_dtype, void* workspace, size_t workspace_bytes, const kvq_layout* layout,
                         kvq_kind kind, const kvq_extend_options* options, void* stream) {
  kvq_status st = check_layout(layout);
  if (st != KVQ_OK) return st;
  if (!kind_read_ok(kind) && kind != KVQ_FP8_E4M3_PAGE) return KVQ_EKIND;
  if (!has_scales(kind)) scales = nullptr;
  if (out_dtype != KVQ_OUT_BF16 && out_dtype != KVQ_OUT_F32) return KVQ_EINVAL;
  if (batch < 0 || total_q < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0) return KVQ_EINVAL;
  if (num_q_heads % layout->num_kv_heads != 0) return KVQ_EINVAL;
  if (options && (options->path < 0 || options->path > 2)) return KVQ_EINVAL;
  if (static_cast<int64_t>(total_q) * (num_q_heads / layout->num_kv_heads) > std::numeric_limits<int32_t>::max() - 128)
    return KVQ_EINVAL;  // the kernel counts query rows per sequence in 32 bits
  if (!(sm_scale > 0.0f) || sm_scale > std::numeric_limits<float>::max()) return KVQ_EINVAL;  // finite, > 0
  if (layout->page_size != kPageTokens) return KVQ_EUNSUPPORTED;
  if (batch > kMaxExtendBatch) return KVQ_EUNSUPPORTED;
  if (kind == KVQ_FP8_E4M3_PAGE) {
    if (options && (options->path != 0 || options->precise_p != 0)) return KVQ_EUNSUPPORTED;
    if (!q_start && batch > 0 && total_q > 0) return KVQ_EINVAL;
    return page_common(q, pool, scales, block_table, max_pages_per_seq, seq_lens, q_start, total_q, batch, num_q_heads,
                       sm_scale, out, out_dtype, workspace, workspace_bytes, layout, false,
                       static_cast<cudaStream_t>(stream));
  }
  ExtendPlan ep;
  if (!plan_extend(*layout, total_q, num_q_heads, max_pages_per_seq, options, &ep)) return KVQ_EUNSUPPORTED;
  if (!workspace) return KVQ_EINVAL;
  if (workspace_bytes < ep.total) return KVQ_EWORKSPACE;
  if (!aligned(workspace)) return KVQ_EALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) != cudaSuccess) return KVQ_ECUDA;
  if (batch == 0 || total_q == 0) return KVQ_OK;
  if (!q || !pool || (has_scales(kind) && !scales) || !block_table || !seq_lens || !q_start || !out)
    return KVQ_EINVAL;
  if (!aligned(q) || !aligned(pool) || !aligned(scales) || !aligned(out) ||
      (reinterpret_cast<uintptr_t>(block_table) % 4) != 0 || (reinterpret_cast<uintptr_t>(seq_lens) % 4) != 0 ||
      (reinterpret_cast<uintptr_t>(q_start) % 4) != 0)
    return KVQ_EALIGN;
  st = kvq_device_check();
  if (st != KVQ_OK) return st;
  if (!ep.flash)
    return extend_prefixes(ep, q, pool, scales, block_table, max_pages_per_seq, seq_lens, q_start, total_q, batch,
                           num_q_heads, sm_scale, out, out_dtype, workspace, layout, kind, s);
  ExtendArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.codes = static_cast<const uint8_t*>(pool);
  a.scales = static_cast<const uint16_t*>(scales);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.q_start = q_start;
  a.out = out;
  a.status = static_cast<uint32_t*>(workspace);
  a.num_pages = layout->num_pages;
  a.max_pages = max_pages_per_seq;
  a.batch = batch;
  a.total_q = total_q;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = layout->num_kv_heads;
  a.head_dim = layout->head_dim;
  a.score_scale = sm_scale * 1.4426950408889634f;  // log2(e)
  a.out_dtype = out_dtype;
  a.kind = kind;
  a.split_p = ep.split ? 1 : 0;
  return launch_extend_tc(a, s);
}

size_t kvq_tree_workspace_bytes(const kvq_layout* layout, int32_t batch, int32_t total_q, int32_t num_q_heads,
                                int32_t max_pages_per_seq, int32_t path) {
  TreePlan tp;
  if (check_layout(layout) != KVQ_OK || layout->page_size != kPageTokens) return 0;
  if (!plan_tree(*layout, batch, total_q, num_q_heads, max_pages_per_seq, path, &tp)) return 0;
  return tp.total;
}

kvq_status kvq_tree(const void* q, const void* pool, const void* scales, const int32_t* block_table,
                    int32_t max_pages_per_seq, const int32_t* seq_lens, const int32_t* q_start, const int64_t* tree_mask,
                    int32_t mask_words, int32_t total_q, int32_t batch, int32_t num_q_heads, float sm_scale, void* out,
                    kvq_out_dtype out_dtype, void* workspace, size_t workspace_bytes, const kvq_layout* layout,
                    kvq_kind kind, int32_t path, void* stream) {
  kvq_status st = check_layout(layout);
  if (st != KVQ_OK) return st;
  if (!kind_read_ok(kind)) return KVQ_EKIND;
  if (!has_scales(kind)) scales = nullptr;
  if (out_dtype != KVQ_OUT_BF16 && out_dtype != KVQ_OUT_F32) return KVQ_EINVAL;
  if (batch < 0 || total_q < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 || mask_words <= 0) return KVQ_EINVAL;
  if (num_q_heads % layout->num_kv_heads != 0 || path < 0 || path > 2) return KVQ_EINVAL;
  if (!(sm_scale > 0.0f) || sm_scale > std::numeric_limits<float>::max()) return KVQ_EINVAL;  // finite, > 0
  if (layout->page_size != kPageTokens || mask_words > kMaxMaskWords) return KVQ_EUNSUPPORTED;
  if (static_cast<int64_t>(max_pages_per_seq) * kPageTokens > std::numeric_limits<int32_t>::max()) return KVQ_EINVAL;
  if (max_pages_per_seq > kMaxTreePages) return KVQ_EUNSUPPORTED;
  TreePlan tp;
  if (!plan_tree(*layout, batch, total_q, num_q_heads, max_pages_per_seq, path, &tp)) return KVQ_EUNSUPPORTED;
  if (!workspace) return KVQ_EINVAL;
  if (workspace_bytes < tp.total) return KVQ_EWORKSPACE;
  const bool empty = batch == 0 || total_q == 0;
  if (!empty && (!q || !pool || (has_scales(kind) && !scales) || !block_table || !seq_lens || !q_start || !tree_mask || !out))
    return KVQ_EINVAL;
  if (!aligned(workspace) || !aligned(q) || !aligned(pool) || !aligned(scales) || !aligned(out) ||
      (reinterpret_cast<uintptr_t>(tree_mask) % 8) != 0)
    return KVQ_EALIGN;
  for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(q_start)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return KVQ_EALIGN;
  st = kvq_device_check();
  if (st != KVQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) return clear_status(workspace, s);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (!tp.flash) {
    st = clear_status(workspace, s);
    if (st != KVQ_OK) return st;
    int32_t* vlens = reinterpret_cast<int32_t*>(ws + tp.lens_offset);
    int32_t* vbase = reinterpret_cast<int32_t*>(ws + tp.base_offset);
    int32_t* vrow = reinterpret_cast<int32_t*>(ws + tp.rows_offset);
    // rows that no sequence covers keep length 0 and row -1: they are left as they are
    if (cudaMemsetAsync(vlens, 0, tp.rows_offset - tp.lens_offset, s) != cudaSuccess ||
        cudaMemsetAsync(vrow, 0xFF, tp.total - tp.rows_offset, s) != cudaSuccess)
      return KVQ_ECUDA;
    st = launch_tree_expand(q_start, seq_lens, batch, total_q, mask_words,
                            static_cast<int64_t>(max_pages_per_seq) * kPageTokens, vlens, vrow, vbase,
                            reinterpret_cast<uint32_t*>(ws), s);
    if (st != KVQ_OK) return st;
    const size_t q_row = static_cast<size_t>(num_q_heads) * layout->head_dim * 2;
    const size_t o_row = static_cast<size_t>(num_q_heads) * layout->v_dim * (out_dtype == KVQ_OUT_F32 ? 4 : 2);
    for (int32_t c0 = 0; c0 < total_q; c0 += tp.chunk) {
      const int32_t n = std::min<int32_t>(tp.chunk, total_q - c0);
      const TreeRows rows = {tree_mask + static_cast<int64_t>(c0) * mask_words, vbase + c0, mask_words};
      st = decode_common(static_cast<const uint8_t*>(q) + c0 * q_row, pool, scales, block_table, max_pages_per_seq,
                         vlens + c0, n, num_q_heads, sm_scale, static_cast<uint8_t*>(out) + c0 * o_row, out_dtype,
                         workspace, tp.dense_bytes, layout, kind, &tp.dec, s, false, vrow + c0, &rows);
      if (st != KVQ_OK) return st;
    }
    return KVQ_OK;
  }
  TreeArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.codes = static_cast<const uint8_t*>(pool);
  a.scales = static_cast<const uint16_t*>(scales);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.q_start = q_start;
  a.mask = tree_mask;
  a.out = out;
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.tab = reinterpret_cast<int32_t*>(ws + tp.tab_offset);
  a.row_seq = reinterpret_cast<int32_t*>(ws + tp.seq_offset);
  a.cta_status = reinterpret_cast<uint32_t*>(ws + tp.st_offset);
  a.part_acc = reinterpret_cast<float*>(ws + tp.acc_offset);
  a.part_ml = reinterpret_cast<float*>(ws + tp.ml_offset);
  a.num_pages = layout->num_pages;
  a.max_pages = max_pages_per_seq;
  a.batch = batch;
  a.total_q = total_q;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = layout->num_kv_heads;
  a.head_dim = layout->head_dim;
  a.mask_words = mask_words;
  a.grid = tp.grid;
  a.score_scale = sm_scale * 1.4426950408889634f;  // log2(e)
  a.out_dtype = out_dtype;
  a.kind = kind;
  return launch_tree_tc(a, s);
}

size_t kvq_prompt_workspace_bytes(void) { return kWorkspaceHeader; }

kvq_status kvq_prompt(const void* q, const void* k, const void* v, const int32_t* q_start, int32_t total, int32_t batch,
                      int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float sm_scale, void* out,
                      kvq_out_dtype out_dtype, const kvq_prompt_strides* strides, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (out_dtype != KVQ_OUT_BF16 && out_dtype != KVQ_OUT_F32) return KVQ_EINVAL;
  if (total < 0 || batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0)
    return KVQ_EINVAL;
  if (head_dim <= 0 || head_dim % 32 != 0) return KVQ_EHEADDIM;
  if (!(sm_scale > 0.0f) || sm_scale > std::numeric_limits<float>::max()) return KVQ_EINVAL;  // finite, > 0
  if (!prompt_supported(head_dim, batch)) return KVQ_EUNSUPPORTED;
  // rows of tiles, and the items of the longest sequence, are counted in 32 bits
  if (static_cast<int64_t>(total) + 128 > std::numeric_limits<int32_t>::max() ||
      (static_cast<int64_t>(total) / 128 + 1) * num_q_heads > std::numeric_limits<int32_t>::max() / 2)
    return KVQ_EUNSUPPORTED;
  PromptArgs a;
  const int64_t d = head_dim;
  a.q_head = a.k_head = a.v_head = a.out_head = d;
  a.q_token = a.out_token = num_q_heads * d;
  a.k_token = a.v_token = num_kv_heads * d;
  if (strides != nullptr) {
    // 16-byte rows; a stride says nothing along a dimension of one
    auto take = [&](int64_t token, int64_t head, int32_t heads, int64_t* t, int64_t* h) {
      if (heads > 1) *h = head;
      if (total > 1) *t = token;
      return *t > 0 && *h > 0 && *t % 8 == 0 && *h % 8 == 0 && *t < (1LL << 39) && *h < (1LL << 39);
    };
    if (!take(strides->q_token, strides->q_head, num_q_heads, &a.q_token, &a.q_head) ||
        !take(strides->k_token, strides->k_head, num_kv_heads, &a.k_token, &a.k_head) ||
        !take(strides->v_token, strides->v_head, num_kv_heads, &a.v_token, &a.v_head) ||
        !take(strides->out_token, strides->out_head, num_q_heads, &a.out_token, &a.out_head))
      return KVQ_EINVAL;
  }
  if (!workspace) return KVQ_EINVAL;
  if (workspace_bytes < kWorkspaceHeader) return KVQ_EWORKSPACE;
  const bool empty = batch == 0 || total == 0;
  if (!empty && (!q || !k || !v || !q_start || !out)) return KVQ_EINVAL;
  if (!aligned(workspace) || !aligned(q) || !aligned(k) || !aligned(v) || !aligned(out) ||
      (reinterpret_cast<uintptr_t>(q_start) % 4) != 0)
    return KVQ_EALIGN;
  const kvq_status st = kvq_device_check();
  if (st != KVQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) return cudaMemsetAsync(workspace, 0, 2 * sizeof(uint32_t), s) == cudaSuccess ? KVQ_OK : KVQ_ECUDA;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_start = q_start;
  a.out = out;
  a.status = static_cast<uint32_t*>(workspace);
  a.counter = a.status + 1;
  a.total = total;
  a.batch = batch;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.sms = sm_count();
  a.score_scale = sm_scale * 1.4426950408889634f;  // log2(e)
  a.out_dtype = out_dtype;
  return launch_prompt(a, s);
}

size_t kvq_append_workspace_bytes(void) { return kWorkspaceHeader; }

kvq_status kvq_append(void* pool, void* scales, const void* q, const void* k, const void* v, const int32_t* block_table,
                      int32_t max_pages_per_seq, const int32_t* seq_lens, const int32_t* q_start,
                      const int32_t* positions, int32_t total, int32_t batch, int32_t num_q_heads, void* q_out,
                      const kvq_rope* rope, const kvq_prompt_strides* strides, void* workspace, size_t workspace_bytes,
                      const kvq_layout* layout, kvq_kind kind, void* stream) {
  kvq_status st = check_layout(layout);
  if (st != KVQ_OK) return st;
  if (!kind_append_ok(kind)) return KVQ_EKIND;
  if (!has_scales(kind)) scales = nullptr;
  if (total < 0 || batch < 0 || num_q_heads < 0 || max_pages_per_seq <= 0) return KVQ_EINVAL;
  if (static_cast<int64_t>(max_pages_per_seq) * layout->page_size > std::numeric_limits<int32_t>::max()) return KVQ_EINVAL;
  if ((num_q_heads == 0) != (q == nullptr) || (q == nullptr) != (q_out == nullptr)) return KVQ_EINVAL;
  if (layout->mla && v != nullptr) return KVQ_EINVAL;
  const int64_t d = layout->head_dim;
  AppendArgs a;
  a.cos_sin = nullptr;
  a.max_position = a.rot_dim = a.rot_offset = a.interleaved = 0;
  if (rope != nullptr) {
    if (rope->cos_sin == nullptr || rope->max_position <= 0 || (rope->interleaved != 0 && rope->interleaved != 1))
      return KVQ_EINVAL;
    // pieces of 8 elements lie in one half of a rotation, or outside
    if (rope->rot_dim <= 0 || rope->rot_dim % 16 != 0 || rope->rot_offset < 0 || rope->rot_offset % 8 != 0 ||
        rope->rot_dim > d || rope->rot_offset > d - rope->rot_dim)
      return KVQ_EINVAL;
    if (!aligned(rope->cos_sin)) return KVQ_EALIGN;
    a.cos_sin = rope->cos_sin;
    a.max_position = rope->max_position;
    a.rot_dim = rope->rot_dim;
    a.rot_offset = rope->rot_offset;
    a.interleaved = rope->interleaved;
  }
  if (kind == KVQ_FP8_E4M3_PAGE && (layout->mla || layout->page_size != kPageTokens)) return KVQ_EUNSUPPORTED;
  if (!append_supported(layout->head_dim, kind)) return KVQ_EUNSUPPORTED;
  a.q_head = a.k_head = a.v_head = a.out_head = d;
  a.q_token = a.out_token = num_q_heads * d;
  a.k_token = a.v_token = layout->num_kv_heads * d;
  if (strides != nullptr) {
    auto take = [&](int64_t token, int64_t head, int32_t heads, int64_t* t, int64_t* h) {
      if (heads > 1) *h = head;
      if (total > 1) *t = token;
      return *t > 0 && *h > 0 && *t % 8 == 0 && *h % 8 == 0 && *t < (1LL << 39) && *h < (1LL << 39);
    };
    if ((num_q_heads > 0 && (!take(strides->q_token, strides->q_head, num_q_heads, &a.q_token, &a.q_head) ||
                             !take(strides->out_token, strides->out_head, num_q_heads, &a.out_token, &a.out_head))) ||
        !take(strides->k_token, strides->k_head, layout->num_kv_heads, &a.k_token, &a.k_head) ||
        (!layout->mla && !take(strides->v_token, strides->v_head, layout->num_kv_heads, &a.v_token, &a.v_head)))
      return KVQ_EINVAL;
  }
  if (q != nullptr && q == q_out && total > 0 && (a.q_token != a.out_token || a.q_head != a.out_head)) return KVQ_EINVAL;
  a.num_kv_heads = layout->num_kv_heads;
  a.num_q_heads = num_q_heads;
  a.n_kv = n_kv_of(*layout);
  a.head_dim = layout->head_dim;
  a.page_size = layout->page_size;
  a.max_pages = max_pages_per_seq;
  a.batch = batch;
  a.total = total;
  a.kind = kind;
  a.num_pages = layout->num_pages;
  if (!workspace) return KVQ_EINVAL;
  if (workspace_bytes < kWorkspaceHeader) return KVQ_EWORKSPACE;
  const bool empty = batch == 0 || total == 0;
  if (!empty && (!pool || (has_scales(kind) && !scales) || !k || (!layout->mla && !v) || !block_table || !seq_lens || !q_start))
    return KVQ_EINVAL;
  if (!aligned(workspace) || !aligned(pool) || !aligned(scales) || !aligned(q) || !aligned(k) || !aligned(v) || !aligned(q_out))
    return KVQ_EALIGN;
  for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(q_start), static_cast<const void*>(positions)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return KVQ_EALIGN;
  const int64_t grid = append_grid(&a, sm_count());
  if (grid > std::numeric_limits<int32_t>::max()) return KVQ_EUNSUPPORTED;  // a grid dimension
  st = kvq_device_check();
  if (st != KVQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) return clear_status(workspace, s);
  a.codes = static_cast<uint8_t*>(pool);
  a.scales = scales;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.q_start = q_start;
  a.positions = positions;
  a.status = static_cast<uint32_t*>(workspace);
  return launch_append(a, grid, s);
}

size_t kvq_pages_workspace_bytes(const kvq_layout* layout, int32_t n, int32_t max_pages_per_seq) {
  PagesPlan pp;
  if (check_layout(layout) != KVQ_OK || !plan_pages(*layout, n, max_pages_per_seq, &pp)) return 0;
  return pp.total;
}

kvq_status kvq_pages_copy(void* pool, void* scales, const int32_t* src, const int32_t* dst, int32_t n,
                          const kvq_layout* layout, kvq_kind kind, void* stream) {
  kvq_status st = check_layout(layout);
  if (st != KVQ_OK) return st;
  if (!kind_append_ok(kind)) return KVQ_EKIND;
  if (!has_scales(kind)) scales = nullptr;
  if (n < 0) return KVQ_EINVAL;
  const int64_t page_bytes =
      static_cast<int64_t>(n_kv_of(*layout)) * layout->num_kv_heads * layout->page_size * layout->head_dim;
  const bool by_page = kind == KVQ_FP8_E4M3_PAGE;
  if (by_page && layout->mla) return KVQ_EUNSUPPORTED;
  const int64_t scale_bytes = by_page         ? static_cast<int64_t>(2 * sizeof(float)) * layout->num_kv_heads
                              : kind_ok(kind) ? page_bytes / 16
                                              : 0;
  if ((!by_page && scale_bytes % 16 != 0) || page_bytes > (1LL << 34)) return KVQ_EUNSUPPORTED;  // whole 16-byte pieces, 32-bit counts
  if (n == 0) return KVQ_OK;
  if (!pool || (has_scales(kind) && !scales) || !src || !dst) return KVQ_EINVAL;
  if (!aligned(pool) || !aligned(scales) || (reinterpret_cast<uintptr_t>(src) % 4) != 0 ||
      (reinterpret_cast<uintptr_t>(dst) % 4) != 0)
    return KVQ_EALIGN;
  st = kvq_device_check();
  if (st != KVQ_OK) return st;
  return launch_copy_pages(pool, scales, src, dst, n, layout->num_pages, static_cast<uint32_t>(page_bytes / 16),
                           static_cast<uint32_t>(scale_bytes), static_cast<cudaStream_t>(stream));
}

kvq_status kvq_pages_fork(int32_t* block_table, int32_t max_pages_per_seq, int32_t* seq_lens, int32_t batch,
                          int32_t* page_refs, const int32_t* src, const int32_t* dst, int32_t n, int32_t* copy_src,
                          int32_t* copy_dst, void* workspace, size_t workspace_bytes, const kvq_layout* layout,
                          void* stream) {
  PagesArgs a;
  kvq_status st = pages_common(block_table, max_pages_per_seq, seq_lens, batch, page_refs, dst, n, workspace,
                               workspace_bytes, layout, &a);
  if (st != KVQ_OK) return st;
  if (n > 0 && (!src || !copy_src || !copy_dst)) return KVQ_EINVAL;
  for (const void* p : {static_cast<const void*>(src), static_cast<const void*>(copy_src),
                        static_cast<const void*>(copy_dst)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return KVQ_EALIGN;
  st = kvq_device_check();
  if (st != KVQ_OK) return st;
  if (n == 0) return clear_status(workspace, static_cast<cudaStream_t>(stream));
  a.src = src;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  return launch_fork_pages(a, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_pages_resize(int32_t* block_table, int32_t max_pages_per_seq, int32_t* seq_lens, int32_t batch,
                            int32_t* page_refs, const int32_t* seqs, const int32_t* new_lens, int32_t n,
                            void* workspace, size_t workspace_bytes, const kvq_layout* layout, void* stream) {
  PagesArgs a;
  kvq_status st = pages_common(block_table, max_pages_per_seq, seq_lens, batch, page_refs, seqs, n, workspace,
                               workspace_bytes, layout, &a);
  if (st != KVQ_OK) return st;
  if (n > 0 && !new_lens) return KVQ_EINVAL;
  if (reinterpret_cast<uintptr_t>(new_lens) % 4 != 0) return KVQ_EALIGN;
  st = kvq_device_check();
  if (st != KVQ_OK) return st;
  if (n == 0) return clear_status(workspace, static_cast<cudaStream_t>(stream));
  a.new_lens = new_lens;
  return launch_resize_pages(a, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_pages_compact(void* pool, void* scales, const int32_t* block_table, int32_t max_pages_per_seq,
                             const int32_t* seq_lens, const int32_t* q_start, const int64_t* keep, int32_t mask_words,
                             int32_t batch, int32_t* new_lens, const int32_t* page_refs, void* workspace,
                             size_t workspace_bytes, const kvq_layout* layout, kvq_kind kind, void* stream) {
  kvq_status st = check_layout(layout);
  if (st != KVQ_OK) return st;
  if (!kind_read_ok(kind)) return KVQ_EKIND;
  if (!has_scales(kind)) scales = nullptr;
  if (batch < 0 || max_pages_per_seq <= 0 || mask_words <= 0) return KVQ_EINVAL;
  if (mask_words > kMaxMaskWords) return KVQ_EUNSUPPORTED;
  if (!workspace) return KVQ_EINVAL;
  if (workspace_bytes < kWorkspaceHeader) return KVQ_EWORKSPACE;
  const int64_t kv_rows = static_cast<int64_t>(n_kv_of(*layout)) * layout->num_kv_heads;
  if (kv_rows > 65535) return KVQ_EUNSUPPORTED;  // a grid dimension
  if (batch > 0 && (!pool || (has_scales(kind) && !scales) || !block_table || !seq_lens || !q_start || !keep || !new_lens))
    return KVQ_EINVAL;
  if (!aligned(workspace) || !aligned(pool) || !aligned(scales) || (reinterpret_cast<uintptr_t>(keep) % 8) != 0)
    return KVQ_EALIGN;
  for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(q_start), static_cast<const void*>(new_lens),
                        static_cast<const void*>(page_refs)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return KVQ_EALIGN;
  // new_lens is written while other CTAs still read the rest
  const size_t b = batch, ints = b * sizeof(int32_t);
  if (overlap(new_lens, ints, seq_lens, ints) || overlap(new_lens, ints, q_start, ints + sizeof(int32_t)) ||
      overlap(new_lens, ints, block_table, ints * max_pages_per_seq) ||
      overlap(new_lens, ints, keep, b * mask_words * sizeof(int64_t)) ||
      overlap(new_lens, ints, page_refs, static_cast<size_t>(layout->num_pages) * sizeof(int32_t)))
    return KVQ_EINVAL;
  st = kvq_device_check();
  if (st != KVQ_OK) return st;
  if (batch == 0) return clear_status(workspace, static_cast<cudaStream_t>(stream));
  CompactArgs a;
  a.codes = static_cast<uint8_t*>(pool);
  a.scales = static_cast<uint16_t*>(scales);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.q_start = q_start;
  a.keep = keep;
  a.page_refs = page_refs;
  a.new_lens = new_lens;
  a.status = static_cast<uint32_t*>(workspace);
  a.num_pages = layout->num_pages;
  a.max_pages = max_pages_per_seq;
  a.batch = batch;
  a.mask_words = mask_words;
  a.page_size = layout->page_size;
  a.kv_rows = static_cast<int32_t>(kv_rows);
  a.head_dim = layout->head_dim;
  return launch_compact(a, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_workspace_status(const void* workspace, void* stream) {
  if (!workspace) return KVQ_EINVAL;
  uint32_t word = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost, s) != cudaSuccess) return KVQ_ECUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return KVQ_ECUDA;
  if (word == 0) return KVQ_OK;
  if (word == kStatusNoPagesWord) return KVQ_ENOPAGES;
  return word == kStatusTimeoutWord ? KVQ_ETIMEOUT : KVQ_EINVAL;
}

kvq_status kvq_encode_probe(kvq_kind kind, const float* y, uint8_t* codes, int64_t n, void* stream) {
  if (!kind_ok(kind)) return KVQ_EKIND;
  if (n < 0) return KVQ_EINVAL;
  if (n == 0) return KVQ_OK;
  if (!y || !codes) return KVQ_EINVAL;
  kvq_status st = kvq_device_check();
  if (st != KVQ_OK) return st;
  return launch_encode_probe(kind, y, codes, n, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_quantize_probe(kvq_kind kind, const uint16_t* x, int64_t nx, const uint16_t* s, int64_t ns,
                              uint8_t* codes, void* stream) {
  if (!kind_ok(kind)) return KVQ_EKIND;
  if (nx < 0 || ns < 0) return KVQ_EINVAL;
  if (nx == 0 || ns == 0) return KVQ_OK;
  if (!x || !s || !codes) return KVQ_EINVAL;
  kvq_status st = kvq_device_check();
  if (st != KVQ_OK) return st;
  return launch_quantize_probe(kind, x, nx, s, ns, codes, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_dequant_probe(kvq_kind kind, const uint8_t* codes, const uint16_t* scales, uint16_t* out, int64_t n,
                             void* stream) {
  if (!kind_read_ok(kind)) return KVQ_EKIND;
  if (!has_scales(kind)) scales = nullptr;
  if (n < 0 || n % 16 != 0) return KVQ_EINVAL;
  if (n == 0) return KVQ_OK;
  if (!codes || (has_scales(kind) && !scales) || !out) return KVQ_EINVAL;
  if (!aligned(codes) || !aligned(out)) return KVQ_EALIGN;
  kvq_status st = kvq_device_check();
  if (st != KVQ_OK) return st;
  return launch_dequant_probe(kind, codes, scales, out, n, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_exp2_probe(const float* x, float* y, int64_t n, void* stream) {
  if (n < 0) return KVQ_EINVAL;
  if (n == 0) return KVQ_OK;
  if (!x || !y) return KVQ_EINVAL;
  if ((reinterpret_cast<uintptr_t>(x) % 4) != 0 || (reinterpret_cast<uintptr_t>(y) % 4) != 0) return KVQ_EALIGN;
  const kvq_status st = kvq_device_check();
  if (st != KVQ_OK) return st;
  return launch_exp2_probe(x, y, n, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_wait_probe(void* workspace, void* stream) {
  if (!workspace) return KVQ_EINVAL;
  if (!aligned(workspace)) return KVQ_EALIGN;
  kvq_status st = kvq_device_check();
  if (st != KVQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) != cudaSuccess) return KVQ_ECUDA;
  return launch_wait_probe(static_cast<uint32_t*>(workspace), s);
}

}  // extern "C"
