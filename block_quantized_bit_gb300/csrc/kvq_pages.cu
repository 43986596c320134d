// kvq_pages.cu -- pages of the cache: copies, forks, growth and release, and the compaction of drafted tokens.
//
// A page p of the pool is held by page_refs[p] block-table rows and is free while that count is 0.  The free
// list is never stored: the calls that take pages read the counts and take the lowest-numbered free pages, in
// the order of their list, so a call's result does not depend on the order in which earlier pages were
// released, and pages that one call releases are free from the next call on.
//
// fork and resize share two kernels:
//   plan   one CTA (times column slices) per list entry checks the entry, finds how many pages it needs and
//          (fork) copies the parent's row to the workspace, since another entry may replace that row; further
//          CTAs turn 8192 counts each into a bitmap of free pages with per-word prefixes and a total.
//   apply  starts when the plan is complete (programmatic dependent launch).  If an entry was bad or the free
//          pages do not suffice, it changes nothing and says so in the status word.  Else every column is
//          one thread's work: find the r-th free page by binary search over the bitmap's prefixes, change
//          the two counts, write the entry.  Counts change by atomic adds of integers: any order gives the
//          same result.
// The bitmap is a snapshot, so apply never reads a count that another CTA of it may have changed.
//
// Both move few bytes (4 B per page of the rows, 4 B per page of the pool); they are bound by the latency of
// two dependent launches: in a graph a fork of 64 rows takes 8 us, of 32 rows over 2048 columns 12 us, a resize of 1 to
// 64 rows 5 to 6 us.  A caller that launches them one by one waits for the host instead (9 us per call from Python).
//
// copy is bound by HBM: 16384 pages (570 MB read and written) 87.9 us, 6.5 TB/s, 96% of the measured copy rate; a call of
// some pages takes 2.7 us in a graph.  compact moves the few kept rows of each sequence, a CTA per (sequence, K or V,
// head), and is bound by its chain of dependent loads: 4 to 6 us in a graph.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// ------------------------------------------------------------------------------------------ page copies
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;  // 16-byte pieces in flight per thread

// Piece u of the call: piece u % per_page of pair u / per_page; a page's code pieces come first, then its
// scale pieces.  Every CTA moves kCopyThreads * kCopyVecs consecutive pieces, all loads before the stores.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(uint4* codes, uint4* scales, const int32_t* __restrict__ src,
                                                                  const int32_t* __restrict__ dst, int32_t n,
                                                                  int64_t num_pages, uint32_t code_vecs,
                                                                  uint32_t scale_vecs) {
  const uint32_t per_page = code_vecs + scale_vecs;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kCopyThreads * kCopyVecs);
  const int64_t pair0 = first / per_page;
  const uint32_t rem0 = static_cast<uint32_t>(first - pair0 * per_page);
  uint4 v[kCopyVecs];
  uint4* to[kCopyVecs];
#pragma unroll
  for (int j = 0; j < kCopyVecs; ++j) {
    const uint32_t local = rem0 + j * kCopyThreads + threadIdx.x;
    const uint32_t skip = local / per_page, u = local - skip * per_page;
    const int64_t pair = pair0 + skip;
    to[j] = nullptr;
    if (pair >= n) continue;
    const int64_t s = __ldg(src + pair), d = __ldg(dst + pair);
    if (s < 0 || d < 0 || s >= num_pages || d >= num_pages) continue;
    const bool code = u < code_vecs;
    const uint4* from = code ? codes + s * code_vecs + u : scales + s * scale_vecs + (u - code_vecs);
    to[j] = code ? codes + d * code_vecs + u : scales + d * scale_vecs + (u - code_vecs);
    v[j] = *from;
  }
#pragma unroll
  for (int j = 0; j < kCopyVecs; ++j)
    if (to[j] != nullptr) *to[j] = v[j];
}

// --------------------------------------------------------------------------------------- fork and resize
constexpr int kPlanThreads = 256;
constexpr int kChunkPages = kPagesChunk;           // pages one CTA of the plan looks at
constexpr int kChunkWords = kChunkPages / 32;
constexpr int kSliceCols = kPagesSlice;            // block-table columns one CTA works on
static_assert(kSliceCols % kPlanThreads == 0, "whole rounds of a CTA's threads");

__device__ __forceinline__ int32_t pages_of(int32_t tokens, int32_t page_size) {
  return static_cast<int32_t>((static_cast<int64_t>(tokens) + page_size - 1) / page_size);
}

// One chunk of counts -> bitmap words, per-word exclusive prefixes and the chunk's total.
__device__ void plan_chunk(const PagesArgs& a, int32_t chunk) {
  __shared__ int32_t s_tot[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  static_assert(kChunkWords == kPlanThreads, "one word per thread");
  const int64_t base = static_cast<int64_t>(chunk) * kChunkPages + warp * 1024;
  uint32_t word = 0;
#pragma unroll 8
  for (int w = 0; w < 32; ++w) {
    const int64_t p = base + w * 32 + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, p < a.num_pages && a.page_refs[p] == 0);
    word = (w == lane) ? m : word;
  }
  const int32_t c = __popc(word);
  int32_t incl = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_tot[warp] = incl;
  __syncthreads();
  int32_t off = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    off += w < warp ? s_tot[w] : 0;
    tot += s_tot[w];
  }
  a.bits[static_cast<int64_t>(chunk) * kChunkWords + threadIdx.x] = word;
  a.word_prefix[static_cast<int64_t>(chunk) * kChunkWords + threadIdx.x] = off + incl - c;
  if (threadIdx.x == 0) a.chunk_free[chunk] = tot;
}

template <bool FORK>
__global__ void __launch_bounds__(kPlanThreads) plan_pages_kernel(PagesArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  if (static_cast<int32_t>(blockIdx.x) >= a.n) {
    if (blockIdx.y == 0) plan_chunk(a, static_cast<int32_t>(blockIdx.x) - a.n);
    return;
  }
  const int32_t i = blockIdx.x, tid = threadIdx.x;
  if (i == 0 && blockIdx.y == 0 && tid == 0) *a.status = 0;
  const int64_t max_tok = static_cast<int64_t>(a.max_pages) * a.page_size;
  const int32_t d = __ldg(a.dst + i);
  const int32_t s = FORK ? __ldg(a.src + i) : d;
  bool ok = s >= 0 && s < a.batch && d >= 0 && d < a.batch;
  const int32_t old_len = ok ? a.seq_lens[d] : 0;
  const int32_t new_len = !ok ? 0 : (FORK ? a.seq_lens[s] : a.new_lens[i]);
  ok = ok && old_len >= 0 && old_len <= max_tok && new_len >= 0 && new_len <= max_tok;
  // another entry with the same row; (fork) the parent's row is replaced; an earlier child of the parent
  bool dup = false, gone = false, earlier = false;
  for (int32_t j = tid; j < a.n; j += kPlanThreads) {
    const int32_t dj = __ldg(a.dst + j);
    dup |= j != i && dj == d;
    if (FORK) {
      gone |= dj == s;
      earlier |= j < i && __ldg(a.src + j) == s;
    }
  }
  dup = __syncthreads_or(dup);
  if (FORK) {
    gone = __syncthreads_or(gone);
    earlier = __syncthreads_or(earlier);
  }
  ok = ok && !dup;
  if (!FORK && ok && new_len > old_len && old_len % a.page_size != 0) {
    // the new tokens' first rows would go into a page that another row reads
    const int32_t p = a.block_table[static_cast<int64_t>(d) * a.max_pages + old_len / a.page_size];
    ok = !(p >= 0 && p < a.num_pages && a.page_refs[p] > 1);
  }
  const int32_t used_new = ok ? pages_of(new_len, a.page_size) : 0;
  const int32_t used_old = ok ? pages_of(old_len, a.page_size) : 0;
  const int32_t* row = a.block_table + static_cast<int64_t>(ok ? s : 0) * a.max_pages;
  if (blockIdx.y == 0 && tid == 0) {
    int32_t need = max(used_new - used_old, 0), tail = -1;
    if (FORK) {
      // the partly filled last page of the parent goes on with one row: the parent's own, or where that is
      // replaced the first child in the list; every other child gets a copy, and so does that one when a row
      // besides the parent holds the page (a row cut back into a page that it had shared when it was full)
      need = 0;
      if (ok && new_len % a.page_size != 0) {
        tail = row[used_new - 1];
        need = tail >= 0 && tail < a.num_pages && (!gone || earlier || a.page_refs[tail] > 1);
      }
    }
    PagesEntry e;
    e.row = ok ? d : -1;
    e.used_old = used_old;
    e.used_new = used_new;
    e.new_len = new_len;
    e.tail = tail;
    e.need = need;
    a.entries[i] = e;
  }
  if (FORK) {
    const int32_t c0 = blockIdx.y * kSliceCols, c1 = min(c0 + kSliceCols, used_new);
    for (int32_t c = c0 + tid; c < c1; c += kPlanThreads) a.rows[static_cast<int64_t>(i) * a.max_pages + c] = row[c];
  }
}

// Position of the k-th (from 0) set bit of w, which has more than k.
__device__ __forceinline__ int32_t nth_bit(uint32_t w, int32_t k) {
  int32_t at = 0;
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) {
    const int32_t c = __popc((w >> at) & ((1u << s) - 1u));
    if (k >= c) {
      k -= c;
      at += s;
    }
  }
  return at;
}

// The r-th lowest free page of the snapshot; s_pre[c]: free pages before chunk c.
__device__ __forceinline__ int32_t free_page(const PagesArgs& a, const int32_t* s_pre, int32_t r) {
  int32_t lo = 0, hi = a.chunks;  // last chunk with s_pre <= r
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (s_pre[mid] <= r) lo = mid;
    else hi = mid;
  }
  const int32_t k = r - s_pre[lo];
  const int32_t* wp = a.word_prefix + static_cast<int64_t>(lo) * kChunkWords;
  int32_t w = 0, wh = kChunkWords;
  while (wh - w > 1) {
    const int32_t mid = (w + wh) >> 1;
    if (wp[mid] <= k) w = mid;
    else wh = mid;
  }
  const uint32_t bits = a.bits[static_cast<int64_t>(lo) * kChunkWords + w];
  return lo * kChunkPages + w * 32 + nth_bit(bits, k - wp[w]);
}

// One row less holds page p.  A count that is 0 already (a table that lists a page nobody counted) stays 0 and
// is reported: that the page was free before the call is in the bitmap, since another row may have taken it by now.
__device__ __forceinline__ void release_page(const PagesArgs& a, int32_t p) {
  if (p < 0 || p >= a.num_pages) return;
  const bool was_free = (a.bits[p >> 5] >> (p & 31)) & 1u;
  if (atomicSub(a.page_refs + p, 1) <= 0 || was_free) {
    atomicAdd(a.page_refs + p, 1);
    set_status(a.status, kStatusBadPages);
  }
}

template <bool FORK>
__global__ void __launch_bounds__(kPlanThreads) apply_pages_kernel(PagesArgs a) {
  extern __shared__ int32_t s_pre[];  // [chunks] free pages before each chunk
  __shared__ uint32_t s_need[2][kPlanThreads / 32];
  __shared__ int32_t s_free[kPlanThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // pages needed by the entries before this one and by all; is every entry good?  (The demand may pass 32 bits: sums
  // stop at a number that no pool has.)
  constexpr uint32_t kTooMany = 1u << 27;
  static_assert(kTooMany > static_cast<int64_t>(kMaxPagesChunks) * kPagesChunk, "more than the pages of any pool");
  uint32_t before = 0, total = 0;
  bool bad = false;
  for (int32_t j = tid; j < a.n; j += kPlanThreads) {
    const PagesEntry& e = a.entries[j];
    const uint32_t need = e.need;
    total = min(total + need, kTooMany);
    before = min(before + (j < i ? need : 0u), kTooMany);
    bad |= e.row < 0;
  }
  // exclusive prefix over the chunks, kPlanThreads at a time
  int32_t free_total = 0;
  for (int32_t c0 = 0; c0 < a.chunks; c0 += kPlanThreads) {
    const int32_t c = c0 + tid;
    const int32_t x = c < a.chunks ? a.chunk_free[c] : 0;
    int32_t incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_free[warp] = incl;
    __syncthreads();
    int32_t off = 0, tot = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      off += w < warp ? s_free[w] : 0;
      tot += s_free[w];
    }
    if (c < a.chunks) s_pre[c] = free_total + off + incl - x;
    free_total += tot;
    __syncthreads();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before = min(before + __shfl_xor_sync(0xffffffffu, before, o), kTooMany);
    total = min(total + __shfl_xor_sync(0xffffffffu, total, o), kTooMany);
  }
  if (lane == 0) {
    s_need[0][warp] = before;
    s_need[1][warp] = total;
  }
  bad = __syncthreads_or(bad);
  before = total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    before = min(before + s_need[0][w], kTooMany);
    total = min(total + s_need[1][w], kTooMany);
  }
  if (bad || total > static_cast<uint32_t>(free_total)) {
    if (i == 0 && blockIdx.y == 0 && tid == 0) set_status(a.status, bad ? kStatusBadPages : kStatusNoPages);
    if (FORK && blockIdx.y == 0 && tid == 0) a.copy_src[i] = a.copy_dst[i] = -1;
    return;
  }
  const int32_t rank = static_cast<int32_t>(before);  // (at most the free pages)
  const PagesEntry e = a.entries[i];
  int32_t* row = a.block_table + static_cast<int64_t>(e.row) * a.max_pages;
  const int32_t c0 = blockIdx.y * kSliceCols, c1 = min(c0 + kSliceCols, a.max_pages);
  if (FORK) {
    const int32_t* from = a.rows + static_cast<int64_t>(i) * a.max_pages;
    const int32_t tail_col = e.need ? e.used_new - 1 : -1;
    for (int32_t c = c0 + tid; c < c1; c += kPlanThreads) {
      const int32_t old = row[c];
      int32_t now = c < e.used_new ? from[c] : -1;
      if (c == tail_col) {
        now = free_page(a, s_pre, rank);
        a.copy_src[i] = e.tail;
        a.copy_dst[i] = now;
      }
      const bool held = c < e.used_old;
      if (now == old && held == (c < e.used_new)) continue;  // the same page in the same place
      if (c < e.used_new && now >= 0 && now < a.num_pages) atomicAdd(a.page_refs + now, 1);
      if (held) release_page(a, old);
      if (now != old) row[c] = now;
    }
    if (blockIdx.y == 0 && tid == 0 && !e.need) a.copy_src[i] = a.copy_dst[i] = -1;
  } else {
    const int32_t lo = max(min(e.used_old, e.used_new), c0), hi = min(max(e.used_old, e.used_new), c1);
    for (int32_t c = lo + tid; c < hi; c += kPlanThreads) {
      if (e.used_new > e.used_old) {
        const int32_t p = free_page(a, s_pre, rank + c - e.used_old);
        atomicAdd(a.page_refs + p, 1);  // (0 -> 1; a wrong table may release the page at the same time)
        row[c] = p;
      } else {
        release_page(a, row[c]);
        row[c] = -1;
      }
    }
  }
  if (blockIdx.y == 0 && tid == 0) a.seq_lens[e.row] = e.new_len;
}

// ------------------------------------------------------------------------------------------- compaction
constexpr int kCompactThreads = 128;
constexpr int kCompactVecs = 8;                                // 16-byte pieces held per thread
constexpr int kCompactPieces = kCompactThreads * kCompactVecs; // pieces one round moves

// The drafted tokens of sequence b: number, first position, whether the sequence can be compacted.
struct Drafted {
  int32_t n, base, len;
  bool ok;
};

__device__ __forceinline__ Drafted drafted(const CompactArgs& a, int32_t b) {
  Drafted t;
  const int32_t q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1);
  t.len = __ldg(a.seq_lens + b);
  t.n = q1 - q0;
  t.ok = q0 >= 0 && q1 >= q0 && t.n <= 64 * a.mask_words && t.n <= t.len &&
         t.len <= static_cast<int64_t>(a.max_pages) * a.page_size;
  if (!t.ok) t.n = 0;
  t.base = t.len - t.n;
  return t;
}

__device__ __forceinline__ uint64_t keep_word(const CompactArgs& a, int32_t b, int32_t w, int32_t n) {
  const int32_t left = n - 64 * w;
  if (left <= 0) return 0;
  const uint64_t m = static_cast<uint64_t>(__ldg(reinterpret_cast<const long long*>(a.keep) +
                                                 static_cast<int64_t>(b) * a.mask_words + w));
  return left >= 64 ? m : m & ((1ull << left) - 1ull);
}

// Kept tokens of sequence b, or -1 when it cannot be compacted: a page of the drafted tokens is masked or past
// the pool, or (with counts) a page that rows move to is held by another sequence too.
__device__ int32_t kept_tokens(const CompactArgs& a, int32_t b, const Drafted& t) {
  if (!t.ok) return -1;
  int32_t kept = 0, still = 0;  // still: leading kept tokens that stay where they are
  bool run = true;
  for (int32_t w = 0; w < a.mask_words; ++w) {
    const uint64_t m = keep_word(a, b, w, t.n);
    kept += __popcll(m);
    if (run) {
      const int32_t ones = m == ~0ull ? 64 : __ffsll(static_cast<long long>(~m)) - 1;
      still += ones;
      run = ones == 64;
    }
  }
  if (t.n == 0) return kept;
  const int32_t* row = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  for (int32_t p = t.base / a.page_size; p <= (t.len - 1) / a.page_size; ++p) {
    const int32_t pg = __ldg(row + p);
    if (pg < 0 || pg >= a.num_pages) return -1;
    const bool written = kept > still && p >= (t.base + still) / a.page_size && p <= (t.base + kept - 1) / a.page_size;
    if (written && a.page_refs != nullptr && __ldg(a.page_refs + pg) > 1) return -1;
  }
  return kept;
}

// CTA (sequence, kv row set): the kept rows of one (K or V, head) move to the front of the drafted tokens, a
// round of rows at a time, all loads of a round before its stores.  A kept row only ever moves towards the
// front, and the rows are taken in order, so a round never overwrites a row that a later round still reads.
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(CompactArgs a) {
  __shared__ int16_t s_from[64 * kMaxMaskWords];  // drafted number of the k-th kept token
  __shared__ int32_t s_kept;
  const int32_t b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  if (b == a.batch) {  // one CTA more reports the sequences that are left as they are
    if (h != 0) return;
    bool bad = false;
    for (int32_t j = tid; j < a.batch; j += kCompactThreads) bad |= kept_tokens(a, j, drafted(a, j)) < 0;
    bad = __syncthreads_or(bad);
    if (tid == 0) *a.status = bad ? kStatusBadPages : 0;
    return;
  }
  const Drafted t = drafted(a, b);
  if (tid == 0) s_kept = kept_tokens(a, b, t);
  for (int32_t j = tid; j < t.n; j += kCompactThreads) {
    int32_t before = 0;
    uint64_t m = 0;
    for (int32_t w = 0; w <= j / 64; ++w) {
      m = keep_word(a, b, w, t.n);
      before += w < j / 64 ? __popcll(m) : __popcll(m & ((1ull << (j & 63)) - 1ull));
    }
    if ((m >> (j & 63)) & 1ull) s_from[before] = static_cast<int16_t>(j);
  }
  __syncthreads();
  const int32_t kept = s_kept;
  if (h == 0 && tid == 0) a.new_lens[b] = kept < 0 ? t.len : t.base + kept;
  if (kept <= 0) return;
  const int32_t* row = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  const int32_t P = a.page_size, code_vecs = a.head_dim / 16, blocks = a.head_dim / 32;
  auto row_of = [&](int32_t pos) -> int64_t {  // row of this (K or V, head) in the pool
    return (static_cast<int64_t>(__ldg(row + pos / P)) * a.kv_rows + h) * P + pos % P;
  };
  const int32_t slice = min(code_vecs, 64);           // pieces of a row taken at once
  const int32_t rows = kCompactPieces / slice;        // rows of a round
  for (int32_t v0 = 0; v0 < code_vecs; v0 += slice) {
    const int32_t nv = min(slice, code_vecs - v0);
    for (int32_t k0 = 0; k0 < kept; k0 += rows) {
      const int32_t items = min(rows, kept - k0) * nv;
      uint4 r[kCompactVecs];
#pragma unroll
      for (int u = 0; u < kCompactVecs; ++u) {
        const int32_t it = u * kCompactThreads + tid;
        const int32_t k = k0 + it / nv;
        if (it < items && s_from[k] != k)
          r[u] = reinterpret_cast<const uint4*>(a.codes + row_of(t.base + s_from[k]) * a.head_dim)[v0 + it % nv];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kCompactVecs; ++u) {
        const int32_t it = u * kCompactThreads + tid;
        const int32_t k = k0 + it / nv;
        if (it < items && s_from[k] != k)
          reinterpret_cast<uint4*>(a.codes + row_of(t.base + k) * a.head_dim)[v0 + it % nv] = r[u];
      }
      __syncthreads();
    }
  }
  if (a.scales == nullptr) return;
  for (int32_t k0 = 0; k0 < kept * blocks; k0 += kCompactThreads) {  // the scales, 128 in flight, in the same order
    const int32_t it = k0 + tid, k = it / blocks;
    const bool live = it < kept * blocks && s_from[k] != k;
    uint16_t x = 0;
    if (live) x = a.scales[row_of(t.base + s_from[k]) * blocks + it % blocks];
    __syncthreads();
    if (live) a.scales[row_of(t.base + k) * blocks + it % blocks] = x;
    __syncthreads();
  }
}

kvq_status launched() { return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ECUDA; }

template <bool FORK>
kvq_status launch_pages(const PagesArgs& a, cudaStream_t stream) {
  const unsigned slices = static_cast<unsigned>((a.max_pages + kSliceCols - 1) / kSliceCols);
  plan_pages_kernel<FORK><<<dim3(static_cast<unsigned>(a.n + a.chunks), FORK ? slices : 1), kPlanThreads, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return KVQ_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n), slices);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(std::max<int32_t>(a.chunks, 1)) * sizeof(int32_t);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, apply_pages_kernel<FORK>, a);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? KVQ_OK : KVQ_ECUDA;
}

}  // namespace

kvq_status launch_copy_pages(void* codes, void* scales, const int32_t* src, const int32_t* dst, int32_t n,
                             int64_t num_pages, uint32_t code_vecs, uint32_t scale_vecs, cudaStream_t stream) {
  const int64_t per_cta = kCopyThreads * kCopyVecs;
  const int64_t grid = (static_cast<int64_t>(n) * (code_vecs + scale_vecs) + per_cta - 1) / per_cta;
  if (grid > 0x7fffffffLL) return KVQ_EUNSUPPORTED;
  copy_pages_kernel<<<static_cast<unsigned>(grid), kCopyThreads, 0, stream>>>(
      static_cast<uint4*>(codes), static_cast<uint4*>(scales), src, dst, n, num_pages, code_vecs, scale_vecs);
  return launched();
}

kvq_status launch_fork_pages(const PagesArgs& a, cudaStream_t stream) { return launch_pages<true>(a, stream); }

kvq_status launch_resize_pages(const PagesArgs& a, cudaStream_t stream) { return launch_pages<false>(a, stream); }

kvq_status launch_compact(const CompactArgs& a, cudaStream_t stream) {
  compact_kernel<<<dim3(static_cast<unsigned>(a.batch + 1), static_cast<unsigned>(a.kv_rows)), kCompactThreads, 0,
                   stream>>>(a);
  return launched();
}

}  // namespace kvq
