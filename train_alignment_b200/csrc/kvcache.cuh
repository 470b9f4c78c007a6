// What the kernels over the paged NVFP4 key/value cache share (internal).
#pragma once

#include "common.cuh"

namespace quads {

// The cache and the sequences in it as kernels get them.
struct CacheArgs {
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  const float* g_k;
  const float* g_v;
  const int32_t* table;     // [n_seqs][max_pages]
  int64_t n_pages;
  int page_size;
  int n_heads;
  int max_pages;
  int n_seqs;
  FastDiv page_div;
};

// Row (of 16-element blocks) of token `at` of a page for one head:
// codes at row * D / 2, scales at row * D / 16.
__device__ __forceinline__ int64_t cache_row(const CacheArgs& c, int page, int head, int at) {
  return (static_cast<int64_t>(page) * c.n_heads + head) * c.page_size + at;
}

// Page of position pos (>= 0) of sequence b, or -1 where the table has none:
// past its width, or an entry that names no page of the cache.
__device__ __forceinline__ int page_of(const CacheArgs& c, int b, int pos, int& at) {
  const int j = static_cast<int>(fast_div(static_cast<uint32_t>(pos), c.page_div));
  at = pos - j * c.page_size;
  if (j >= c.max_pages) return -1;
  const int p = __ldg(c.table + static_cast<int64_t>(b) * c.max_pages + j);
  return (p >= 0 && p < c.n_pages) ? p : -1;
}

// The last b in [0, n) with off[b] <= row, or -1: one whole warp, 32 probes a
// step (off ascending, n + 1 entries).
__device__ __forceinline__ int warp_find_seq(const int32_t* __restrict__ off, int n, int row, int lane) {
  int lo = 0, len = n;
  while (len > 0) {
    const int step = (len + 31) >> 5;
    const int i = lane * step;
    const bool le = i < len && __ldg(off + lo + i) <= row;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    if (cnt == 0) return -1;
    const int at = (cnt - 1) * step;
    if (step == 1) return lo + at;
    lo += at;
    len = min(step, len - at);
  }
  return -1;
}

// Host checks of a cache and its sequences.
int check_cache(const quads_kv_cache* cache);
int check_seqs(const int32_t* row_off, const int32_t* block_table, int n_seqs, int max_pages);
CacheArgs cache_args(const quads_kv_cache* cache, const int32_t* block_table, int n_seqs, int max_pages);

}  // namespace quads
