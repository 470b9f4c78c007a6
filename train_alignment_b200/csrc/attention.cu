// Softmax attention of new tokens over the paged NVFP4 key/value cache.
//
//   out[r][h] = sum_j softmax_j(scale q[r][h] . k_j) v_j,  j <= p, j > p - window
//
// Two kernels: few rows per sequence and key head (attention_decode.cuh) are
// bound by the cache's bytes and their conversion, many (attention_chunk.cuh)
// by the tensor cores.
#include "attention_chunk.cuh"
#include "attention_decode.cuh"

namespace quads {

int attention_wait_status(unsigned int* v) {
  if (cudaMemcpyFromSymbol(v, g_attention_wait_status, sizeof(*v)) != cudaSuccess)
    return set_error(QUADS_ERR_CUDA, "cannot read the device status word");
  const unsigned int zero = 0;
  if (*v && cudaMemcpyToSymbol(g_attention_wait_status, &zero, sizeof(zero)) != cudaSuccess)
    return set_error(QUADS_ERR_CUDA, "cannot clear the device status word");
  return QUADS_OK;
}

namespace {

// One thread waits on a barrier that nothing completes, as the kernel for many
// rows waits; the wait gives up after limit_ns and records the timeout.
__global__ void attention_wait_selftest_kernel(uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(smem_addr(&bar), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    ch_wait(smem_addr(&bar), 0, &abort_flag, limit_ns);
  }
}

// Launches a kernel that may become resident before the one in front of it in
// the stream has ended, and waits for that itself.
template <typename... Params, typename... Args>
int launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream, const char* what, Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return check_launch(what);
  return QUADS_OK;
}

// CTAs of the kernel for few rows: as many as are resident at once.
int dec_grid(int nt) { return dec_ctas_per_sm(nt) * num_sms(); }
// Key tiles (of 128) of a split: shorter ones cost more in joining than they save.
constexpr int kChMinTiles = 4;
// Whether the kernel for few rows (of a sequence and key head) is taken: up to
// 48, and up to 64 where the sequences' key heads are no more than the SMs, so
// that the kernel for many, whose blocks take one each, leaves some idle or
// waits for the longest.  4 key heads of 128: 16 sequences of up to 8192 keys
// with 48 rows 35 us against 58, with 64 rows 41 against 58 (of up to 1024
// keys 15.0 against 16.2); 64 sequences of up to 512 with 64 rows 32 against
// 24, of up to 2048 60 against 54; 16 of up to 2048 with 96 rows 28 against 23.
bool few_rows(const quads_kv_cache* c, int n_seqs, int64_t unit_rows) {
  return unit_rows <= 48 || (unit_rows <= 64 && static_cast<int64_t>(n_seqs) * c->n_heads <= num_sms());
}
// Tiles of a run, at least: as few as leave a unit at most 192 parts to join
// (one key head's 65536 keys: 171 parts 12.0 us, 256 13.2, 128 12.4).  Four
// contexts of 2048: runs of 1 tile 9.6 us, of 4 11.8.
constexpr int kDecMaxParts = 192;
// What beginning and ending a unit costs, in tiles: runs are equal with it, so
// that one with two ends in it has fewer tiles.  A run's tile takes about
// 1.4 us (three share an SM), its look-ups, fill and join 2.4 or more: without
// it the runs of 64 contexts of up to 4096 ended at 18.2, 20.8 and 22.8 us by
// the units in them.  0, 1, 2, 3, 4: 27.1, 25.7, 26.1, 25.5, 26.9 us (whole
// tiles); 256 contexts of up to 2000 99, 92, 89, 86, 87.  Not where a run would
// have but a tile or two.
constexpr int kDecUnitCost = 3;

// The parts of units that runs share, and where a run can be long enough, what
// its warps take out of their accumulators.
size_t dec_workspace(int D, int nt, bool keep) {
  const size_t kept = keep ? kDecWarps * dec_kept_floats(D, nt) * sizeof(float) : 0;
  return static_cast<size_t>(dec_grid(nt)) * (2 * (8 * nt) * (D * sizeof(float) + sizeof(float2)) + sizeof(int4) + kept);
}

// Keys that a unit can see, at most.
int64_t dec_keys(const quads_kv_cache* c, int max_pages, int max_q_len, int window) {
  const int64_t all = static_cast<int64_t>(max_pages) * c->page_size, seen = static_cast<int64_t>(window) + max_q_len + 15;
  return window > 0 && seen < all ? seen : all;
}
// Whether a CTA takes whole units: contexts of at most 8 tiles.  64 contexts of
// up to 1024, 8 heads: 19.3 us in one launch, 23.9 cut and joined in two; one
// context of 700, 4 heads: 8.2 us on the GPU against 6.9, but called one by
// one 15.3 against 19.8, because the host's second launch and workspace cost
// more than that.
constexpr int kDecWhole = 8;
bool dec_whole(int64_t keys) { return keys <= kDecWhole * kDecTile; }
int dec_min_quota(int64_t tiles) { return static_cast<int>(ceil_div(tiles, int64_t(kDecMaxParts))); }
int64_t dec_units(const quads_kv_cache* c, int n_seqs, int64_t unit_rows, int nt) {
  return static_cast<int64_t>(n_seqs) * c->n_heads * ceil_div(unit_rows, int64_t(8) * nt);
}
// Whether a warp can have so many steps in a unit that its sums are begun anew.
bool dec_keeps(int64_t units, int64_t tiles, int nt) {
  const int64_t run = ceil_div(units * (tiles + kDecUnitCost), int64_t(dec_grid(nt))), least = dec_min_quota(tiles);
  return tiles > kDecKeep && (run > least ? run : least) >= kDecKeep;
}

template <int D, int NT>
int launch_decode(AttnArgs p, const quads_kv_cache* cache, void* ws, int unit_rows, int64_t keys, bool whole, cudaStream_t stream) {
  const int grid = dec_grid(NT);
  p.row_groups = (unit_rows + 8 * NT - 1) / (8 * NT);
  const int64_t units = dec_units(cache, p.c.n_seqs, unit_rows, NT);
  const int64_t tiles = ceil_div(keys, int64_t(kDecTile));
  if (whole) {
    attention_decode_kernel<D, NT, true, false><<<static_cast<unsigned>(units < grid ? units : grid), kDecThreads, 0, stream>>>(p, 0);
    count_launches(1);
    return check_launch("attention_decode_kernel");
  }
  p.cuts = static_cast<int4*>(ws);
  p.part_o = reinterpret_cast<float*>(p.cuts + grid);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(2) * grid * (8 * NT) * D);
  if (dec_keeps(units, tiles, NT)) p.kept = reinterpret_cast<float*>(p.part_ml + static_cast<size_t>(2) * grid * (8 * NT));
  p.by_unit = units <= grid;
  p.unit_cost = units * tiles >= 2 * grid ? kDecUnitCost : 0;
  if (p.kept != nullptr)
    attention_decode_kernel<D, NT, false, true><<<grid, kDecThreads, 0, stream>>>(p, dec_min_quota(tiles));
  else
    attention_decode_kernel<D, NT, false, false><<<grid, kDecThreads, 0, stream>>>(p, dec_min_quota(tiles));
  QUADS_TRY(check_launch("attention_decode_kernel"));
  // the join: rows on blocks of their own as far as there are SMs for them
  const int64_t x = p.by_unit ? units : grid, per = num_sms() / x;
  const int most = unit_rows < 8 * NT ? unit_rows : 8 * NT;
  const dim3 join(static_cast<unsigned>(x), static_cast<unsigned>(per < 1 ? 1 : per < most ? per : most));
  QUADS_TRY(launch_dependent(attention_combine_kernel<D, NT>, join, kJoinThreads * NT, stream, "attention_combine_kernel", p));
  count_launches(2);
  return QUADS_OK;
}

// The grid of the kernel for many rows: blocks of 256 rows (at most; some
// find no rows), and the splits of their keys that fill the SMs.
struct ChunkPlan {
  int64_t blocks;
  int n_split;
  bool keep;           // contexts can be so long that sums are begun anew
};
ChunkPlan chunk_plan(const quads_kv_cache* c, int64_t rows, int heads_q, int n_seqs, int max_pages, int max_q_len) {
  const int64_t group = heads_q / c->n_heads;
  const int64_t by_rows = rows * group / kChRows + n_seqs;
  const int64_t by_seqs = ceil_div(static_cast<int64_t>(max_q_len) * group, int64_t(kChRows)) * n_seqs;
  ChunkPlan p{by_rows < by_seqs ? by_rows : by_seqs, 1, false};
  const int64_t units = p.blocks * c->n_heads;
  const int64_t tiles = ceil_div(static_cast<int64_t>(max_pages) * c->page_size, int64_t(kChTile));
  p.keep = tiles > kChKeep;
  int64_t n = units > 0 ? num_sms() / units : 1;
  if (n > tiles / kChMinTiles) n = tiles / kChMinTiles;
  // no more than 256 MB of parts (a call with many rows of no sequence)
  const int64_t part = rows * heads_q * static_cast<int64_t>(c->head_dim * sizeof(float) + sizeof(float2));
  while (n > 1 && n * part > (int64_t(1) << 28)) --n;
  if (n > 1) p.n_split = static_cast<int>(n);
  return p;
}

size_t chunk_workspace(const quads_kv_cache* c, int64_t rows, int heads_q, const ChunkPlan& p) {
  if (p.n_split <= 1 && !p.keep) return 0;
  return static_cast<size_t>(p.n_split) * rows * heads_q * (c->head_dim * sizeof(float) + sizeof(float2));
}

// The softmax warpgroups wait for registers that the others give up, which adds
// up only if the kernel was compiled to 128 a thread.
template <int D, bool kKeep>
bool chunk_registers_add_up() {
  static const bool ok = [] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, attention_chunk_kernel<D, kKeep>) == cudaSuccess && a.numRegs == kChRegs;
  }();
  return ok;
}

template <int D, bool kKeep>
int launch_chunk(AttnArgs p, const ChunkPlan& plan, void* ws, cudaStream_t stream) {
  p.part_o = static_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(plan.n_split) * p.rows * p.hq * D);
  p.kept = p.part_o;
  QUADS_REQUIRE((chunk_registers_add_up<D, kKeep>()), QUADS_ERR_CUDA, "attention_chunk_kernel is not compiled to %d registers", kChRegs);
  const int smem = ch_smem_bytes(D);
  if (cudaFuncSetAttribute(attention_chunk_kernel<D, kKeep>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return check_launch("attention_chunk_kernel attributes");
  const dim3 grid(static_cast<unsigned>(plan.blocks * p.c.n_heads), plan.n_split);
  attention_chunk_kernel<D, kKeep><<<grid, kChThreads, smem, stream>>>(p, plan.n_split);
  count_launches(1);
  QUADS_TRY(check_launch("attention_chunk_kernel"));
  if (plan.n_split > 1) {
    const dim3 join(static_cast<unsigned>(ceil_div(p.rows * p.hq, int64_t(8))));
    QUADS_TRY(launch_dependent(attention_join_kernel<D>, join, 256, stream, "attention_join_kernel", p, plan.n_split));
    count_launches(1);
  }
  return QUADS_OK;
}

}  // namespace
}  // namespace quads

using namespace quads;

extern "C" {

int quads_selftest_attention_wait(uint64_t timeout_ns, quads_stream_t stream) {
  clear_error();
  QUADS_REQUIRE(timeout_ns > 0 && timeout_ns <= 10000000000ull, QUADS_ERR_INVALID_ARG, "timeout must be in (0, 10 s]");
  attention_wait_selftest_kernel<<<1, 32, 0, stream>>>(timeout_ns);
  count_launches(1);
  return check_launch("attention_wait_selftest_kernel");
}

size_t quads_attention_paged_workspace_bytes(const quads_kv_cache* cache, int64_t rows, int heads_q, int n_seqs,
                                             int max_pages, int max_q_len) {
  if (cache == nullptr || cache->n_heads < 1 || heads_q < 1 || heads_q % cache->n_heads != 0) return 0;
  if (rows <= 0 || n_seqs <= 0 || max_q_len <= 0 || max_pages < 0) return 0;
  const int64_t unit_rows = static_cast<int64_t>(max_q_len) * (heads_q / cache->n_heads);
  if (few_rows(cache, n_seqs, unit_rows)) {               // without a window, with which a call may need none
    const int64_t keys = dec_keys(cache, max_pages, max_q_len, 0);
    const int nt = unit_rows <= 8 ? 1 : 2;
    return dec_whole(keys) ? 0 : dec_workspace(cache->head_dim, nt, dec_keeps(dec_units(cache, n_seqs, unit_rows, nt), ceil_div(keys, int64_t(kDecTile)), nt));
  }
  return chunk_workspace(cache, rows, heads_q, chunk_plan(cache, rows, heads_q, n_seqs, max_pages, max_q_len));
}

int quads_attention_paged(const uint16_t* q, int64_t rows, int64_t ld_q, int heads_q, const quads_kv_cache* cache,
                          const int32_t* row_off, const int32_t* kv_len, const int32_t* block_table, int n_seqs,
                          int max_pages, int max_q_len, float scale, int window, uint16_t* out, float* lse, void* ws,
                          size_t ws_bytes, quads_stream_t stream) {
  clear_error();
  QUADS_TRY(check_cache(cache));
  QUADS_TRY(check_seqs(row_off, block_table, n_seqs, max_pages));
  QUADS_REQUIRE(rows >= 0 && rows < (int64_t(1) << 30), QUADS_ERR_INVALID_ARG, "rows must be in [0, 2^30)");
  QUADS_REQUIRE(rows * heads_q < (int64_t(1) << 31), QUADS_ERR_UNSUPPORTED_SHAPE, "rows * heads_q must be below 2^31");
  QUADS_REQUIRE(heads_q >= 1 && heads_q <= 4096 && heads_q % cache->n_heads == 0, QUADS_ERR_UNSUPPORTED_SHAPE,
                "heads_q (%d) must be a multiple of the cache's %d heads, at most 4096", heads_q, cache->n_heads);
  QUADS_REQUIRE(ld_q >= static_cast<int64_t>(heads_q) * cache->head_dim && ld_q % 8 == 0, QUADS_ERR_INVALID_ARG,
                "q's row stride must be a multiple of 8 of at least heads_q * head_dim");
  // positions of a tile's keys then fit 32 bits
  QUADS_REQUIRE(static_cast<int64_t>(max_pages) * cache->page_size <= (int64_t(1) << 31) - (1 << 16),
                QUADS_ERR_UNSUPPORTED_SHAPE, "max_pages * page_size must be at most 2^31 - 2^16");
  QUADS_REQUIRE(window >= 0 && max_q_len >= 0, QUADS_ERR_INVALID_ARG, "window and max_q_len must be >= 0");
  QUADS_REQUIRE(scale - scale == 0.0f, QUADS_ERR_INVALID_ARG, "the scale must be finite");
  if (rows == 0 || n_seqs == 0 || max_q_len == 0) return QUADS_OK;
  QUADS_REQUIRE(q && out && kv_len, QUADS_ERR_INVALID_ARG, "null pointer");
  QUADS_REQUIRE(aligned(q, 16) && aligned(out, 16), QUADS_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  const size_t need = quads_attention_paged_workspace_bytes(cache, rows, heads_q, n_seqs, max_pages, max_q_len);
  QUADS_REQUIRE(need == 0 || (ws != nullptr && ws_bytes >= need && aligned(ws, 16)), QUADS_ERR_INVALID_ARG,
                "a 16-byte aligned workspace of %zu bytes is required", need);
  const int64_t width = static_cast<int64_t>(heads_q) * cache->head_dim;
  QUADS_REQUIRE(out + rows * width <= q || q + (rows - 1) * ld_q + width <= out, QUADS_ERR_INVALID_ARG,
                "out must not overlap q");
  AttnArgs p{};
  p.c = cache_args(cache, block_table, n_seqs, max_pages);
  p.q = q; p.out = out; p.lse = lse; p.off = row_off; p.kv_len = kv_len;
  p.rows = rows; p.ld_q = ld_q; p.hq = heads_q; p.group = heads_q / cache->n_heads;
  p.max_q = max_q_len; p.window = window; p.scale = scale;
  p.group_div = make_fastdiv(static_cast<uint32_t>(p.group));
  const int64_t unit_rows = static_cast<int64_t>(max_q_len) * p.group;
  if (few_rows(cache, n_seqs, unit_rows)) {
    const int64_t tiles = (static_cast<int64_t>(max_pages) * cache->page_size / kDecTile + 2 + kDecUnitCost) * ceil_div(unit_rows, int64_t(8));
    QUADS_REQUIRE(tiles < (int64_t(1) << 30) && tiles * n_seqs * cache->n_heads < (int64_t(1) << 30),
                  QUADS_ERR_UNSUPPORTED_SHAPE, "too many key tiles: n_seqs * n_heads * (max_pages * page_size / %d + %d) must be below 2^27", kDecTile, 2 + kDecUnitCost);
    const int n = static_cast<int>(unit_rows);
    const int64_t keys = dec_keys(cache, max_pages, max_q_len, window);
    const bool whole = dec_whole(keys);
    if (cache->head_dim == 64)
      return n <= 8 ? launch_decode<64, 1>(p, cache, ws, n, keys, whole, stream) : launch_decode<64, 2>(p, cache, ws, n, keys, whole, stream);
    return n <= 8 ? launch_decode<128, 1>(p, cache, ws, n, keys, whole, stream) : launch_decode<128, 2>(p, cache, ws, n, keys, whole, stream);
  }
  const ChunkPlan plan = chunk_plan(cache, rows, heads_q, n_seqs, max_pages, max_q_len);
  QUADS_REQUIRE(plan.blocks * cache->n_heads < (int64_t(1) << 31) && ceil_div(rows * heads_q, int64_t(8)) < (int64_t(1) << 31),
                QUADS_ERR_UNSUPPORTED_SHAPE, "too many rows");
  if (plan.keep)
    return cache->head_dim == 64 ? launch_chunk<64, true>(p, plan, ws, stream) : launch_chunk<128, true>(p, plan, ws, stream);
  return cache->head_dim == 64 ? launch_chunk<64, false>(p, plan, ws, stream) : launch_chunk<128, false>(p, plan, ws, stream);
}

}  // extern "C"
