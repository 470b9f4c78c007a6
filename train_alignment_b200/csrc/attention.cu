// Softmax attention of new tokens over the paged NVFP4 key/value cache.
//
//   out[r][h] = sum_j softmax_j(scale q[r][h] . k_j) v_j,  j <= p, j > p - window
//
// One warp per (row, query head): an online softmax over the positions in
// order, 32 positions' scores at a time.
#include "attention.cuh"
#include "attention_decode.cuh"

namespace quads {
namespace {

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

// CTAs of the kernel for few rows: as many as are resident at once.
int dec_grid(int nt) {
  const int n = dec_ctas_per_sm(nt) * num_sms();
  return n < kMaxRuns ? n : kMaxRuns;
}
constexpr int kDecMinQuota = 4;      // tiles of a run: shorter ones cost more in joining than they save

size_t dec_workspace(int D, int nt) {
  return static_cast<size_t>(dec_grid(nt)) * (2 * (8 * nt) * (D * sizeof(float) + sizeof(float2)) + sizeof(int4));
}

template <int D, int NT>
int launch_decode(AttnArgs p, void* ws, int unit_rows, cudaStream_t stream) {
  const int grid = dec_grid(NT);
  const int64_t units = static_cast<int64_t>(p.c.n_seqs) * p.c.n_heads;
  p.cuts = static_cast<int4*>(ws);
  p.part_o = reinterpret_cast<float*>(p.cuts + grid);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(2) * grid * (8 * NT) * D);
  p.by_unit = units <= grid;
  attention_decode_kernel<D, NT><<<grid, kDecThreads, 0, stream>>>(p, kDecMinQuota);
  QUADS_TRY(check_launch("attention_decode_kernel"));
  // the joining kernel is resident before the last run ends and waits for it
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  // rows on blocks of their own where few units are cut into many runs
  cfg.gridDim = dim3(static_cast<unsigned>(p.by_unit ? units : grid), units * 8 <= grid ? unit_rows : 1);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attention_combine_kernel<D, NT>, p) != cudaSuccess)
    return check_launch("attention_combine_kernel");
  count_launches(2);
  return QUADS_OK;
}

}  // namespace
}  // namespace quads

using namespace quads;

extern "C" {

size_t quads_attention_paged_workspace_bytes(const quads_kv_cache* cache, int64_t rows, int heads_q, int n_seqs,
                                             int max_pages, int max_q_len) {
  if (cache == nullptr || cache->n_heads < 1 || heads_q < 1 || heads_q % cache->n_heads != 0) return 0;
  (void)rows; (void)n_seqs; (void)max_pages;
  const int64_t unit_rows = static_cast<int64_t>(max_q_len) * (heads_q / cache->n_heads);
  if (unit_rows <= 16) return dec_workspace(cache->head_dim, unit_rows <= 8 ? 1 : 2);
  return 0;
}

int quads_attention_paged(const uint16_t* q, int64_t rows, int64_t ld_q, int heads_q, const quads_kv_cache* cache,
                          const int32_t* row_off, const int32_t* kv_len, const int32_t* block_table, int n_seqs,
                          int max_pages, int max_q_len, float scale, int window, uint16_t* out, float* lse, void* ws,
                          size_t ws_bytes, quads_stream_t stream) {
  clear_error();
  QUADS_TRY(check_cache(cache));
  QUADS_TRY(check_seqs(row_off, block_table, n_seqs, max_pages));
  QUADS_REQUIRE(rows >= 0 && rows < (int64_t(1) << 30), QUADS_ERR_INVALID_ARG, "rows must be in [0, 2^30)");
  QUADS_REQUIRE(rows * cache->n_heads < (int64_t(1) << 31), QUADS_ERR_UNSUPPORTED_SHAPE,
                "rows * n_heads must be below 2^31");
  QUADS_REQUIRE(heads_q >= 1 && heads_q <= 4096 && heads_q % cache->n_heads == 0, QUADS_ERR_UNSUPPORTED_SHAPE,
                "heads_q (%d) must be a multiple of the cache's %d heads, at most 4096", heads_q, cache->n_heads);
  QUADS_REQUIRE(ld_q >= static_cast<int64_t>(heads_q) * cache->head_dim && ld_q % 8 == 0, QUADS_ERR_INVALID_ARG,
                "q's row stride must be a multiple of 8 of at least heads_q * head_dim");
  QUADS_REQUIRE(window >= 0 && max_q_len >= 0, QUADS_ERR_INVALID_ARG, "window and max_q_len must be >= 0");
  QUADS_REQUIRE(scale - scale == 0.0f, QUADS_ERR_INVALID_ARG, "the scale must be finite");
  if (rows == 0 || n_seqs == 0 || max_q_len == 0) return QUADS_OK;
  QUADS_REQUIRE(q && out && kv_len, QUADS_ERR_INVALID_ARG, "null pointer");
  QUADS_REQUIRE(aligned(q, 16) && aligned(out, 16), QUADS_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  const size_t need = quads_attention_paged_workspace_bytes(cache, rows, heads_q, n_seqs, max_pages, max_q_len);
  QUADS_REQUIRE(need == 0 || (ws != nullptr && ws_bytes >= need && aligned(ws, 16)), QUADS_ERR_INVALID_ARG,
                "a 16-byte aligned workspace of %zu bytes is required", need);
  AttnArgs p{};
  p.c = cache_args(cache, block_table, n_seqs, max_pages);
  p.q = q; p.out = out; p.lse = lse; p.off = row_off; p.kv_len = kv_len;
  p.rows = rows; p.ld_q = ld_q; p.hq = heads_q; p.group = heads_q / cache->n_heads;
  p.max_q = max_q_len; p.window = window < (1 << 30) ? window : (1 << 30); p.scale = scale;
  p.group_div = make_fastdiv(static_cast<uint32_t>(p.group));
  const int64_t unit_rows = static_cast<int64_t>(max_q_len) * p.group;
  if (unit_rows <= 16) {
    const int64_t tiles = static_cast<int64_t>(max_pages) * cache->page_size / kDecTile + 2;
    QUADS_REQUIRE(tiles < (int64_t(1) << 30) && tiles * n_seqs * cache->n_heads < (int64_t(1) << 30),
                  QUADS_ERR_UNSUPPORTED_SHAPE, "n_seqs * n_heads * max_pages * page_size must be below 2^36");
    const int n = static_cast<int>(unit_rows);
    if (cache->head_dim == 64)
      return n <= 8 ? launch_decode<64, 1>(p, ws, n, stream) : launch_decode<64, 2>(p, ws, n, stream);
    return n <= 8 ? launch_decode<128, 1>(p, ws, n, stream) : launch_decode<128, 2>(p, ws, n, stream);
  }
  const unsigned grid = static_cast<unsigned>(ceil_div(rows * heads_q, int64_t(4)));
  if (cache->head_dim == 64)
    attention_kernel<64><<<grid, 128, 0, stream>>>(p);
  else
    attention_kernel<128><<<grid, 128, 0, stream>>>(p);
  count_launches(1);
  return check_launch("attention_kernel");
}

}  // extern "C"
