// kvq_internal.h -- launchers shared between the libkvq translation units (host side).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kvq.h"

namespace kvq {

// Arguments of one decode call after host validation.
struct DecodeArgs {
  const void* q;
  const uint8_t* codes;
  const uint16_t* scales;
  const int32_t* block_table;
  const int32_t* bt_row;  // block-table row of each sequence, or null (row b); set by the MLA extend
  int64_t num_pages;
  int32_t max_pages;
  const int32_t* seq_lens;
  const int64_t* tree_mask;  // per sequence, the drafted tokens it sees, or null; set by kvq_tree (with bt_row)
  const int32_t* tree_base;
  int32_t tree_words;
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t v_dim;
  int32_t mla;
  float sm_scale;
  void* out;
  kvq_out_dtype out_dtype;
  kvq_kind kind;
  int32_t pages_per_split;  // 0 = automatic
  // workspace carve-up
  uint32_t* status;
  float* part_acc;   // [max_items][heads_per_item][v_dim]
  float* part_ml;    // [max_items][heads_per_item][2]
  int32_t* plan_tab; // [batch][2]: first item and split count of each sequence (written by the decode)
  int32_t* split_cnt; // [batch][query groups]: splits finished, zeroed per call; set when the decode
                      // kernel merges its own partials (the last split of a group merges), else null
  int64_t max_items;
  int32_t heads_per_item;  // query heads one work item covers (a tile of the group)
  int32_t split_align;     // automatic split sizes are a multiple of this many pages
  int32_t target_items;    // automatic split sizes aim at about this many work items
  int32_t one_wave_items;  // nonzero: first try splits sized for this many items (one per resident CTA),
                           // kept when the batch's items fit; else target_items
  int32_t min_one_split;   // nonzero: every (sequence, group) has at least one split (an empty one when
                           // the sequence has no page), as the kernel that merges in-kernel needs
};

// Tokens per page the decode kernels support, and the workspace's leading status block.
constexpr int kPageTokens = 16;
constexpr size_t kWorkspaceHeader = 256;
// Status words.  Of two reports the larger one stays, so a wait that was given up, after which no output is valid, has
// the largest.
constexpr uint32_t kStatusNoPagesWord = 0x7500u;  // a page call found too few free pages
constexpr uint32_t kStatusTimeoutWord = 0x7F00u;  // a kernel gave up a bounded wait

// Work-item planning constants shared by the host (workspace bound) and the kernels.
constexpr int kTargetItems = 1216;  // items when the host sets no target; also the SM count assumed without a device
constexpr int kMinPagesPerSplit = 4;

// Heads of one query group that a CUDA-core work item covers.
int32_t cc_heads_per_item(int32_t group, int32_t head_dim, int32_t mla);
// Upper bound on work items for the given sizes (used for workspace sizing and the grid).
int64_t max_work_items(int32_t batch, int32_t query_groups, int32_t max_pages, int32_t pages_per_split,
                       int32_t target_items);

kvq_status launch_store(void* pool, void* scales, const void* k, const void* v, const int64_t* slot_mapping,
                        int64_t num_tokens, const kvq_layout& L, kvq_kind kind, cudaStream_t stream);
kvq_status launch_encode_probe(kvq_kind kind, const float* y, uint8_t* codes, int64_t n, cudaStream_t stream);
kvq_status launch_quantize_probe(kvq_kind kind, const uint16_t* x, int64_t nx, const uint16_t* s, int64_t ns,
                                 uint8_t* codes, cudaStream_t stream);
kvq_status launch_dequant_probe(kvq_kind kind, const uint8_t* codes, const uint16_t* scales, uint16_t* out,
                                int64_t n, cudaStream_t stream);
kvq_status launch_wait_probe(uint32_t* status, cudaStream_t stream);
bool decode_cc_supported(int32_t head_dim, int32_t v_dim, int32_t mla);
int32_t cc_ctas_per_sm(int32_t head_dim, int32_t mla, int32_t heads_per_item);
bool decode_tc_supported(int32_t head_dim, int32_t v_dim, int32_t mla, int32_t group, int32_t batch);
bool decode_mla_tc_supported(int32_t head_dim, int32_t v_dim, int32_t mla, int32_t group, int32_t batch);
int32_t decode_mla_tc_heads_per_item(int32_t group);
kvq_status launch_decode_mla_tc(const DecodeArgs& a, cudaStream_t stream);
kvq_status launch_decode_tc(const DecodeArgs& a, cudaStream_t stream);
kvq_status launch_decode_cc(const DecodeArgs& a, cudaStream_t stream);
kvq_status launch_decode_cc_masked(const DecodeArgs& a, cudaStream_t stream);  // with a.tree_mask
kvq_status launch_merge(const DecodeArgs& a, int32_t query_groups, cudaStream_t stream);

// Sparse decode: the gather of the selected columns into a compact pool (pages b * cpages ..).
struct SparseGatherArgs {
  const uint8_t* codes;
  const uint16_t* scales;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* indices;   // [batch][topk]
  uint8_t* dst_codes;
  uint16_t* dst_scales;
  int32_t* dst_table;       // [batch][cpages]
  int32_t* dst_lens;        // [batch]
  uint32_t* status;
  int64_t num_pages;
  int32_t max_pages;
  int32_t batch;
  int32_t topk;
  int32_t cpages;
  int32_t n_kv, Hkv, D;
};
constexpr int32_t kMaxSparseTopk = 8192;
kvq_status launch_sparse_gather(const SparseGatherArgs& g, cudaStream_t stream);

// Extend (prefill) attention: the new tokens of every sequence attend causally over the pool.
struct ExtendArgs {
  const uint16_t* q;          // [total_q][num_q_heads][head_dim] bf16
  const uint8_t* codes;
  const uint16_t* scales;
  const int32_t* block_table; // [batch][max_pages]
  const int32_t* seq_lens;    // [batch]
  const int32_t* q_start;     // [batch + 1]
  void* out;                  // [total_q][num_q_heads][v_dim]
  uint32_t* status;
  int64_t num_pages;
  int32_t max_pages;
  int32_t batch;
  int32_t total_q;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  float score_scale;          // sm_scale * log2(e): the kernels work in the exp2 domain
  kvq_out_dtype out_dtype;
  kvq_kind kind;
  int32_t split_p;            // nonzero: P enters the PV MMA as two bf16 terms (hi + lo)
};
constexpr int32_t kMaxExtendBatch = 2048;  // sequences whose item bases fit the kernel's shared table
bool extend_tc_supported(int32_t head_dim, int32_t v_dim, int32_t mla, int32_t group, int32_t batch);
kvq_status launch_extend_tc(const ExtendArgs& a, cudaStream_t stream);
kvq_status launch_exp2_probe(const float* x, float* y, int64_t n, cudaStream_t stream);
// MLA extend: each new token's causal prefix length and block-table row (rows of inconsistent sequences
// are left as they are and flagged in the status word).
kvq_status launch_extend_expand(const int32_t* q_start, const int32_t* seq_lens, int32_t batch, int32_t total_q,
                                int32_t* vlens, int32_t* vrow, uint32_t* status, cudaStream_t stream);

// Attention of drafted tokens over the cache (kvq_tree): the split-K flash kernel.
struct TreeArgs {
  const uint16_t* q;          // [total_q][num_q_heads][head_dim] bf16
  const uint8_t* codes;
  const uint16_t* scales;
  const int32_t* block_table; // [batch][max_pages]
  const int32_t* seq_lens;    // [batch]
  const int32_t* q_start;     // [batch + 1]
  const int64_t* mask;        // [total_q][mask_words]
  void* out;                  // [total_q][num_q_heads][head_dim]
  uint32_t* status;
  int32_t* tab;               // [batch + 1] work units before each sequence, then [1] CTAs that share them
  int32_t* row_seq;           // [total_q] sequence of each query row, or -1
  uint32_t* cta_status;       // [CTAs]
  float* part_acc;            // [2 * CTAs][128][head_dim]
  float* part_ml;             // [2 * CTAs][128][2]
  int64_t num_pages;
  int32_t max_pages;
  int32_t batch;
  int32_t total_q;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t mask_words;
  int32_t grid;               // CTAs launched
  float score_scale;          // sm_scale * log2(e)
  kvq_out_dtype out_dtype;
  kvq_kind kind;
};
constexpr int32_t kMaxTreePages = (0x7fffffff - 127) / kPageTokens;  // lengths are rounded up to tiles in 32 bits
constexpr int32_t kMaxTreeBatch = 2048;  // sequences whose unit prefixes fit the kernel's shared table
bool tree_tc_supported(int32_t head_dim, int32_t v_dim, int32_t mla, int32_t batch);
kvq_status launch_tree_tc(const TreeArgs& a, cudaStream_t stream);
// Per query row: stored tokens, block-table row and first drafted position of its sequence; rows that no
// (consistent) sequence covers get length 0 and row -1.
kvq_status launch_tree_expand(const int32_t* q_start, const int32_t* seq_lens, int32_t batch, int32_t total_q,
                              int32_t mask_words, int64_t max_tokens, int32_t* vlens, int32_t* vrow, int32_t* vbase,
                              uint32_t* status, cudaStream_t stream);

// Causal attention over packed prompts (kvq_prompt).  Strides in elements.
struct PromptArgs {
  const void* q;              // [total][num_q_heads][head_dim] bf16
  const void* k;              // [total][num_kv_heads][head_dim] bf16
  const void* v;
  const int32_t* q_start;     // [batch + 1]
  void* out;                  // [total][num_q_heads][head_dim]
  uint32_t* status;
  uint32_t* counter;          // items handed out, zeroed per call
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;
  int32_t total;
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t sms;
  float score_scale;          // sm_scale * log2(e)
  kvq_out_dtype out_dtype;
};
constexpr int32_t kMaxPromptBatch = 2048;  // sequences whose tile counts fit the kernel's shared table
bool prompt_supported(int32_t head_dim, int32_t batch);
kvq_status launch_prompt(const PromptArgs& a, cudaStream_t stream);
kvq_status launch_prompt_wide(const PromptArgs& a, cudaStream_t stream);

// Appends with the position rotation (kvq_append).  Strides in elements.
struct AppendArgs {
  uint8_t* codes;
  void* scales;
  const uint16_t* q;          // [total][num_q_heads][head_dim] bf16, or null with num_q_heads = 0
  const uint16_t* k;          // [total][num_kv_heads][head_dim] bf16
  const uint16_t* v;          // null: the latent row
  uint16_t* q_out;
  const int32_t* block_table; // [batch][max_pages]
  const int32_t* seq_lens;    // [batch]
  const int32_t* q_start;     // [batch + 1]
  const int32_t* positions;   // [total], or null: the places in the sequences
  const float* cos_sin;       // [max_position][rot_dim]
  uint32_t* status;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;
  int64_t num_pages;
  float minus_zero = -0.0f;
  int64_t page_ctas;          // CTAs of the pages kernel that write pages (append_grid)
  int32_t max_pages, batch, total, num_q_heads, num_kv_heads, n_kv, head_dim, page_size;
  int32_t max_position, rot_dim, rot_offset, interleaved;  // rot_dim 0: no rotation
  int32_t row_chunks, part_chunks;                         // CTAs of one token, of one page (append_grid)
  int32_t tokens;                                          // tokens of one CTA (append_grid)
  kvq_kind kind;
};
// Exponents that the power of two of a KVQ_FP8_E4M3_PAGE page may have: codes from 2^-41 to 448 * 2^32.
constexpr int32_t kPageScaleMin = -32, kPageScaleMax = 32;
bool append_supported(int32_t head_dim, kvq_kind kind);
int64_t append_grid(AppendArgs* a, int32_t sms);  // sets the chunks; CTAs of the call
kvq_status launch_append(const AppendArgs& a, int64_t grid, cudaStream_t stream);

// Attention over a KVQ_FP8_E4M3_PAGE cache.
struct PageArgs {
  const uint16_t* q;          // [total_q][num_q_heads][head_dim] bf16
  const uint8_t* codes;
  const float* scales;        // [num_pages][2][num_kv_heads]
  const int32_t* block_table; // [batch][max_pages]
  const int32_t* seq_lens;    // [batch]
  const int32_t* q_start;     // [batch + 1], or null: one row per sequence
  void* out;                  // [total_q][num_q_heads][head_dim]
  uint32_t* status;
  int64_t* total;             // the call's units
  void* runs;                 // [grid] each CTA's first run, then [grid] words: what it reports
  float* part_acc;            // [2 * grid][rows][head_dim], rows: tile
  float* part_ml;             // [2 * grid][rows][2]
  int64_t num_pages;
  int32_t max_pages, batch, total_q, num_q_heads, num_kv_heads, head_dim;
  int32_t grid;               // CTAs launched
  int32_t tile;               // query rows of a unit of work
  float score_scale;          // sm_scale * log2(e)
  kvq_out_dtype out_dtype;
};
constexpr int kPageRowsTile = 16;  // query rows of a tile of the rows kernel at most (8 or 16)
constexpr double kPageRowsUnits = 4096;  // (tile, page) units up to which several tiles of a sequence stay with the rows kernel
constexpr int kPageMinUnits = 8;   // (tile, page) units that are worth a CTA
constexpr int kPageRunMost = 60;   // bytes of a CTA's first run, at most ...
constexpr int kPageRunBytes = kPageRunMost + 4;  // ... and its report
constexpr int kPageItemUnits = 6;   // key tiles' time that an item's start and end take (measured at head_dim 128, used at all)
constexpr int kPageFlashUnits = 10; // units (key tiles and items' starts) that are worth a CTA of the flash kernel
bool page_supported(int32_t head_dim);
int32_t page_rows_grid(int32_t head_dim, int32_t tile, int32_t sms);  // CTAs that are resident at once
kvq_status launch_page_rows(const PageArgs& a, cudaStream_t stream);
int32_t page_flash_rows(int32_t head_dim);  // query rows of an item of the flash kernel
kvq_status launch_page_flash(const PageArgs& a, cudaStream_t stream);
// kvq_decode of that kind with no more CTAs than the workspace has room for.
kvq_status decode_pages_capped(const void* q, const void* pool, const void* scales, const int32_t* block_table,
                               int32_t max_pages, const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                               float sm_scale, void* out, kvq_out_dtype out_dtype, void* workspace, size_t workspace_bytes,
                               const kvq_layout* layout, void* stream);

// Pages of the cache (kvq_pages_*).
constexpr int32_t kPagesChunk = 8192;       // pages whose counts one CTA of the plan reads
constexpr int32_t kMaxPagesChunks = 8192;   // chunks whose prefixes fit the apply kernel's shared memory
constexpr int32_t kPagesSlice = 2048;       // block-table columns one CTA of a fork or a resize works on
constexpr int32_t kMaxPagesCols = 65535 * kPagesSlice;  // slices are a grid's y dimension
constexpr int32_t kMaxPagesList = 0x7fffffff - kMaxPagesChunks;  // entries and chunks are its x dimension
constexpr int32_t kMaxMaskWords = 4;        // 64-bit words of a drafted token's mask: 256 drafted tokens

// What the plan finds for one list entry of a fork or a resize.
struct PagesEntry {
  int32_t row;       // block-table row that changes, -1: a bad entry
  int32_t used_old;  // pages it holds
  int32_t used_new;  // pages it will hold
  int32_t new_len;   // tokens it will hold
  int32_t tail;      // (fork) the parent's partly filled last page, or -1
  int32_t need;      // free pages it takes
};

struct PagesArgs {
  int32_t* block_table;      // [batch][max_pages]
  int32_t* seq_lens;         // [batch]
  int32_t* page_refs;        // [num_pages]
  const int32_t* src;        // [n] (fork) parents
  const int32_t* dst;        // [n] rows that change
  const int32_t* new_lens;   // [n] (resize)
  int32_t* copy_src;         // [n] (fork)
  int32_t* copy_dst;         // [n] (fork)
  int32_t batch, max_pages, n, page_size, chunks;
  int64_t num_pages;
  // workspace carve-up
  uint32_t* status;
  PagesEntry* entries;       // [n]
  int32_t* chunk_free;       // [chunks] free pages of each chunk
  int32_t* word_prefix;      // [chunks][kPagesChunk / 32] free pages of the chunk before each word
  uint32_t* bits;            // [chunks][kPagesChunk / 32] free pages
  int32_t* rows;             // [n][max_pages] the parents' rows (fork)
};

struct CompactArgs {
  uint8_t* codes;
  uint16_t* scales;          // null: an unscaled pool
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* q_start;    // [batch + 1]
  const int64_t* keep;       // [batch][mask_words]
  const int32_t* page_refs;  // [num_pages] or null
  int32_t* new_lens;         // [batch]
  uint32_t* status;
  int64_t num_pages;
  int32_t max_pages, batch, mask_words, page_size, kv_rows, head_dim;
};

kvq_status launch_copy_pages(void* codes, void* scales, const int32_t* src, const int32_t* dst, int32_t n,
                             int64_t num_pages, uint32_t code_vecs, uint32_t scale_bytes, cudaStream_t stream);
kvq_status launch_fork_pages(const PagesArgs& a, cudaStream_t stream);
kvq_status launch_resize_pages(const PagesArgs& a, cudaStream_t stream);
kvq_status launch_compact(const CompactArgs& a, cudaStream_t stream);
}  // namespace kvq
