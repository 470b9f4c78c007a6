// Softmax attention of new tokens over the paged NVFP4 key/value cache.
//
//   out[r][h] = sum_j softmax_j(scale q[r][h] . k_j) v_j,  j <= p, j > p - window
//
// One warp per (row, query head): an online softmax over the positions in
// order, 32 positions' scores at a time.
#include <math_constants.h>

#include "kvcache.cuh"

namespace quads {
namespace {

struct AttnArgs {
  CacheArgs c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int32_t* off;
  const int32_t* kv_len;
  int64_t rows, ld_q;
  int hq, group, max_q, window;
  float scale;
};

template <int D>
__global__ void __launch_bounds__(128) attention_kernel(AttnArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t r = item / p.hq;
  if (r >= p.rows) return;
  const int h = static_cast<int>(item - r * p.hq), hk = h / p.group;
  const int b = warp_find_seq(p.off, p.c.n_seqs, static_cast<int>(r), lane);
  if (b < 0) return;
  const int r0 = p.off[b], r1 = p.off[b + 1];
  if (r >= r1 || r - r0 >= p.max_q) return;
  const int len = p.kv_len[b];
  const int64_t pos = static_cast<int64_t>(len) - (r1 - r0) + (r - r0);
  constexpr int kE = D / 32;                          // elements of a lane
  float q[kE], acc[kE], m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
  for (int i = 0; i < kE; ++i) {
    q[i] = bf16_bits_to_float(p.q[r * p.ld_q + h * D + lane * kE + i]);
    acc[i] = 0.0f;
  }
  const float gk = p.c.g_k[hk], gv = p.c.g_v[hk];
  const int64_t lo64 = p.window > 0 ? pos - p.window + 1 : 0;
  const int lo = static_cast<int>(lo64 > 0 ? lo64 : 0);
  for (int j = lo; j <= pos; ++j) {
    int at;
    const int page = page_of(p.c, b, j, at);
    if (page < 0) continue;
    const int64_t row = cache_row(p.c, page, hk, at);
    float s = 0.0f, v[kE];
    const float ks = e4m3_value(p.c.k_scales[row * (D / 16) + lane * kE / 16]) * gk;
    const float vs = e4m3_value(p.c.v_scales[row * (D / 16) + lane * kE / 16]) * gv;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const int e = lane * kE + i;
      s += q[i] * (e2m1_value((p.c.k_codes[row * (D / 2) + e / 2] >> (4 * (e & 1))) & 15u) * ks);
      v[i] = e2m1_value((p.c.v_codes[row * (D / 2) + e / 2] >> (4 * (e & 1))) & 15u) * vs;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale;
    const float mn = fmaxf(m, s), a = m == -CUDART_INF_F ? 0.0f : __expf(m - mn), w = __expf(s - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < kE; ++i) acc[i] = acc[i] * a + w * v[i];
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int i = 0; i < kE; ++i)
    p.out[(r * p.hq + h) * D + lane * kE + i] = static_cast<uint16_t>(float_to_bf16_bits(acc[i] * inv));
  if (p.lse != nullptr && lane == 0) p.lse[r * p.hq + h] = l > 0.0f ? m + logf(l) : -CUDART_INF_F;
}

}  // namespace
}  // namespace quads

using namespace quads;

extern "C" {

size_t quads_attention_paged_workspace_bytes(const quads_kv_cache* cache, int64_t rows, int heads_q, int n_seqs,
                                             int max_pages, int max_q_len) {
  (void)cache; (void)rows; (void)heads_q; (void)n_seqs; (void)max_pages; (void)max_q_len;
  return 0;
}

int quads_attention_paged(const uint16_t* q, int64_t rows, int64_t ld_q, int heads_q, const quads_kv_cache* cache,
                          const int32_t* row_off, const int32_t* kv_len, const int32_t* block_table, int n_seqs,
                          int max_pages, int max_q_len, float scale, int window, uint16_t* out, float* lse, void* ws,
                          size_t ws_bytes, quads_stream_t stream) {
  clear_error();
  QUADS_TRY(check_cache(cache));
  QUADS_TRY(check_seqs(row_off, block_table, n_seqs, max_pages));
  QUADS_REQUIRE(rows >= 0 && rows < (int64_t(1) << 31), QUADS_ERR_INVALID_ARG, "rows must be in [0, 2^31)");
  QUADS_REQUIRE(heads_q >= 1 && heads_q <= 4096 && heads_q % cache->n_heads == 0, QUADS_ERR_UNSUPPORTED_SHAPE,
                "heads_q (%d) must be a multiple of the cache's %d heads, at most 4096", heads_q, cache->n_heads);
  QUADS_REQUIRE(ld_q >= static_cast<int64_t>(heads_q) * cache->head_dim && ld_q % 8 == 0, QUADS_ERR_INVALID_ARG,
                "q's row stride must be a multiple of 8 of at least heads_q * head_dim");
  QUADS_REQUIRE(window >= 0 && max_q_len >= 0, QUADS_ERR_INVALID_ARG, "window and max_q_len must be >= 0");
  QUADS_REQUIRE(scale - scale == 0.0f, QUADS_ERR_INVALID_ARG, "the scale must be finite");
  if (rows == 0 || n_seqs == 0 || max_q_len == 0) return QUADS_OK;
  QUADS_REQUIRE(q && out && kv_len, QUADS_ERR_INVALID_ARG, "null pointer");
  QUADS_REQUIRE(aligned(q, 16) && aligned(out, 16), QUADS_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  (void)ws; (void)ws_bytes;
  AttnArgs p{};
  p.c = cache_args(cache, block_table, n_seqs, max_pages);
  p.q = q; p.out = out; p.lse = lse; p.off = row_off; p.kv_len = kv_len;
  p.rows = rows; p.ld_q = ld_q; p.hq = heads_q; p.group = heads_q / cache->n_heads;
  p.max_q = max_q_len; p.window = window; p.scale = scale;
  const unsigned grid = static_cast<unsigned>(ceil_div(rows * heads_q, int64_t(4)));
  if (cache->head_dim == 64)
    attention_kernel<64><<<grid, 128, 0, stream>>>(p);
  else
    attention_kernel<128><<<grid, 128, 0, stream>>>(p);
  count_launches(1);
  return check_launch("attention_kernel");
}

}  // extern "C"
