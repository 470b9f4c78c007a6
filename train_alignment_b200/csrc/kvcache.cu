// The paged NVFP4 key/value cache of the rollout: quantized as it is written,
// read back for the trainer; and the rotary positions of its keys and the
// queries.
//
// [TRACE] "Le problème", "Résultats": the rollout keeps weights, activations
// and the KV cache in FP4.  A cached value is e2m1 * e4m3 * g on the grid of
// every other NVFP4 tensor here (blocks of 16 elements of a head, one E4M3
// scale each), with one decode scale g per key/value head that the caller
// calibrates, so a token can be written without reading the others.
#include "kvcache.cuh"

namespace quads {

int check_cache(const quads_kv_cache* c) {
  QUADS_REQUIRE(c != nullptr, QUADS_ERR_INVALID_ARG, "null cache");
  QUADS_REQUIRE(c->n_pages >= 0 && c->n_pages < (int64_t(1) << 31), QUADS_ERR_INVALID_ARG,
                "n_pages must be in [0, 2^31)");
  QUADS_REQUIRE(c->n_heads >= 1 && c->n_heads <= 1024, QUADS_ERR_UNSUPPORTED_SHAPE, "n_heads must be in [1, 1024]");
  QUADS_REQUIRE(c->head_dim == 64 || c->head_dim == 128, QUADS_ERR_UNSUPPORTED_SHAPE,
                "head_dim (%d) must be 64 or 128", c->head_dim);
  QUADS_REQUIRE(c->page_size >= 16 && c->page_size <= 65536 && c->page_size % 16 == 0, QUADS_ERR_UNSUPPORTED_SHAPE,
                "page_size (%d) must be a multiple of 16 in [16, 65536]", c->page_size);
  QUADS_REQUIRE(c->n_pages * c->n_heads * c->page_size < (int64_t(1) << 32) - 1, QUADS_ERR_UNSUPPORTED_SHAPE,
                "n_pages * n_heads * page_size must be below 2^32 - 1");
  QUADS_REQUIRE(c->n_pages == 0 || (c->k_codes && c->k_scales && c->v_codes && c->v_scales), QUADS_ERR_INVALID_ARG,
                "null cache pointer");
  QUADS_REQUIRE(c->g_k && c->g_v, QUADS_ERR_INVALID_ARG, "null decode scales");
  QUADS_REQUIRE(aligned(c->k_codes, 16) && aligned(c->k_scales, 16) && aligned(c->v_codes, 16) &&
                    aligned(c->v_scales, 16),
                QUADS_ERR_INVALID_ARG, "cache pointers must be 16-byte aligned");
  return QUADS_OK;
}

int check_seqs(const int32_t* row_off, const int32_t* block_table, int n_seqs, int max_pages) {
  QUADS_REQUIRE(n_seqs >= 0 && max_pages >= 0, QUADS_ERR_INVALID_ARG, "n_seqs and max_pages must be >= 0");
  QUADS_REQUIRE(n_seqs <= 65535, QUADS_ERR_UNSUPPORTED_SHAPE, "n_seqs must be at most 65535");
  QUADS_REQUIRE(n_seqs == 0 || (row_off && (max_pages == 0 || block_table)), QUADS_ERR_INVALID_ARG, "null pointer");
  return QUADS_OK;
}

CacheArgs cache_args(const quads_kv_cache* c, const int32_t* block_table, int n_seqs, int max_pages) {
  CacheArgs a{};
  a.k_codes = c->k_codes;
  a.k_scales = c->k_scales;
  a.v_codes = c->v_codes;
  a.v_scales = c->v_scales;
  a.g_k = c->g_k;
  a.g_v = c->g_v;
  a.table = block_table;
  a.n_pages = c->n_pages;
  a.page_size = c->page_size;
  a.n_heads = c->n_heads;
  a.max_pages = max_pages;
  a.n_seqs = n_seqs;
  a.page_div = make_fastdiv(static_cast<uint32_t>(c->page_size));
  return a;
}

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 32;       // rows (tokens) of one CTA

// Rows [r0, r0 + n) of a call: the page and the place in it of each, found by
// the CTA's warps (row_s[i] = page or -1, at_s[i]).  first(b) is the position
// of the sequence's first row of this call.
template <typename First>
__device__ __forceinline__ void locate_rows(const CacheArgs& c, const int32_t* __restrict__ off, int64_t r0, int n,
                                            int* page_s, int* at_s, First first) {
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < n; i += kThreads / 32) {
    const int row = static_cast<int>(r0) + i;
    const int b = warp_find_seq(off, c.n_seqs, row, lane);
    int page = -1, at = 0;
    bool in = false;
    if (b >= 0 && row < __ldg(off + b + 1)) {
      in = true;
      const int64_t pos = first(b) + (row - __ldg(off + b));
      if (pos >= 0 && pos < (int64_t(1) << 31)) page = page_of(c, b, static_cast<int>(pos), at);
    }
    if (lane == 0) {
      page_s[i] = in ? page : -2;                    // -2: behind the last sequence
      at_s[i] = at;
    }
  }
  __syncthreads();
}

// 32-byte global accesses.
__device__ __forceinline__ void load_32b(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void store_32b(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The blocks of 16 elements of a row: sides (keys, values) x heads x D / 16.
struct BlockMap {
  FastDiv row_div;             // by the blocks of a row
  int per_side, nb_log2, nb_mask;
};
struct Block {
  int r, head, blk;
  bool second;                 // of the second side
};
__device__ __forceinline__ Block block_of(const BlockMap& m, int i) {
  Block b;
  b.r = static_cast<int>(fast_div(static_cast<uint32_t>(i), m.row_div));
  int j = i - b.r * static_cast<int>(m.row_div.d);
  b.second = j >= m.per_side;
  if (b.second) j -= m.per_side;
  b.head = j >> m.nb_log2;
  b.blk = j & m.nb_mask;
  return b;
}

// --------------------------------------------------------------- the write
// One thread per block of 16 elements: 32 bytes in (one access where the rows
// are 32-byte aligned), 8 + 1 bytes out.  Bound by HBM: 2 bytes read and
// 0.5625 written per element.  16493 tokens of 8 heads of 128 (87 MB): 19 us,
// three quarters of the issue slots taken.
template <bool kWide>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(CacheArgs c, const uint16_t* __restrict__ k,
                                                            const uint16_t* __restrict__ v, int64_t rows,
                                                            int64_t ld_k, int64_t ld_v, BlockMap map,
                                                            const int32_t* __restrict__ off,
                                                            const int32_t* __restrict__ kv_len, int per_cta) {
  __shared__ int page_s[kMaxRows], at_s[kMaxRows];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * per_cta;
  const int n = static_cast<int>(min(static_cast<int64_t>(per_cta), rows - r0));
  locate_rows(c, off, r0, n, page_s, at_s,
              [&](int b) { return static_cast<int64_t>(__ldg(kv_len + b)) - (__ldg(off + b + 1) - __ldg(off + b)); });
  const int nb = map.nb_mask + 1;
  for (int i = threadIdx.x; i < n * static_cast<int>(map.row_div.d); i += kThreads) {
    const Block x = block_of(map, i);
    const int page = page_s[x.r];
    if (page < 0) continue;
    const uint16_t* src = (x.second ? v + (r0 + x.r) * ld_v : k + (r0 + x.r) * ld_k) + (x.head * nb + x.blk) * 16;
    uint32_t w[8];
    if constexpr (kWide) load_32b(src, w);
    else load_bf16x16(src, w);
    const QCore q = quant_core(w, __ldg((x.second ? c.g_v : c.g_k) + x.head));
    const int64_t at = cache_row(c, page, x.head, at_s[x.r]) * nb + x.blk;
    *reinterpret_cast<uint2*>((x.second ? c.v_codes : c.k_codes) + at * 8) = make_uint2(q.lo, q.hi);
    (x.second ? c.v_scales : c.k_scales)[at] = static_cast<uint8_t>(q.scale);
  }
}

// ---------------------------------------------------------------- the read
// One thread per block of 16 elements, two blocks in flight: 8 + 1 bytes in,
// 32 (BF16) or 64 (FP32) out in 32-byte stores.  Bound by HBM: 0.5625 bytes
// read and 2 or 4 written per element.  Eight contexts of up to 8192 tokens, 8
// heads of 128, to BF16 (262 MB): 50 us, 5.2 TB/s (CTAs of twice the rows and
// four blocks in flight: 54).
constexpr int kReadUnroll = 2;

template <bool kF32>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(CacheArgs c, void* __restrict__ k_out,
                                                           void* __restrict__ v_out, int64_t rows, BlockMap map,
                                                           const int32_t* __restrict__ off,
                                                           const int32_t* __restrict__ start, int per_cta) {
  __shared__ int page_s[kMaxRows], at_s[kMaxRows];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * per_cta;
  const int n = static_cast<int>(min(static_cast<int64_t>(per_cta), rows - r0));
  locate_rows(c, off, r0, n, page_s, at_s, [&](int b) -> int64_t { return start != nullptr ? __ldg(start + b) : 0; });
  const int nb = map.nb_mask + 1, total = n * static_cast<int>(map.row_div.d);
  const bool one_side = k_out == nullptr;               // values alone: they are the first side
  for (int i0 = threadIdx.x; i0 < total; i0 += kReadUnroll * kThreads) {
    uint2 codes[kReadUnroll];
    uint32_t s[kReadUnroll];
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      const int i = i0 + u * kThreads;
      codes[u] = make_uint2(0, 0);
      s[u] = 0;
      if (i < total) {
        const Block x = block_of(map, i);
        const int page = page_s[x.r];
        if (page >= 0) {
          const int64_t at = cache_row(c, page, x.head, at_s[x.r]) * nb + x.blk;
          const bool is_v = one_side || x.second;
          codes[u] = __ldg(reinterpret_cast<const uint2*>((is_v ? c.v_codes : c.k_codes) + at * 8));
          s[u] = __ldg((is_v ? c.v_scales : c.k_scales) + at);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= total) break;
      const Block x = block_of(map, i);
      const int page = page_s[x.r];
      if (page == -2) continue;
      const bool is_v = one_side || x.second;
      const float gh = __ldg((is_v ? c.g_v : c.g_k) + x.head), sv = e4m3_value(s[u]);
      const float g = page < 0 ? 0.0f : gh;            // a scale that is NaN or infinite would make a zero code NaN
      const uint64_t sv2 = pack_f32x2(sv, sv), g2 = pack_f32x2(g, g);
      uint32_t h[2][4];
      e2m1x8_to_f16x2(codes[u].x, h[0]);
      e2m1x8_to_f16x2(codes[u].y, h[1]);
      uint64_t f[8];                                   // e2m1 * e4m3 is exact, one rounding with g
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = fmul2_rn(fmul2_rn(f16x2_to_f32x2(h[e >> 2][e & 3]), sv2), g2);
      const int64_t o = ((r0 + x.r) * c.n_heads + x.head) * (16 * nb) + x.blk * 16;
      void* const out = is_v ? v_out : k_out;
      if constexpr (kF32) {
        float* const d = static_cast<float*>(out) + o;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[2 * e] = static_cast<uint32_t>(f[4 * half + e]);
            w[2 * e + 1] = static_cast<uint32_t>(f[4 * half + e] >> 32);
          }
          store_32b(d + 8 * half, w);
        }
      } else {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = f32x2_to_bf16x2(f[e]);
        store_32b(static_cast<uint16_t*>(out) + o, w);
      }
    }
  }
}

// -------------------------------------------------------------------- rope
struct RopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  int64_t T, ld_q, ld_k, ld_qo, ld_ko;
  const int64_t* pos;
  const double* freq;
  int hq, hk, D, rot;
  float mscale, sign;
  FastDiv half_div, row_div, head_div;     // by rot / 2, and by the items of a row and of a head
};

__device__ __forceinline__ void rotate2(uint32_t a, uint32_t b, const float2 (&cs)[2], uint32_t& ra, uint32_t& rb) {
  const float a0 = bf16_bits_to_float(a & 0xFFFFu), a1 = bf16_bits_to_float(a >> 16);
  const float b0 = bf16_bits_to_float(b & 0xFFFFu), b1 = bf16_bits_to_float(b >> 16);
  ra = pack_bf16x2(a0 * cs[0].x - b0 * cs[0].y, a1 * cs[1].x - b1 * cs[1].y);
  rb = pack_bf16x2(b0 * cs[0].x + a0 * cs[0].y, b1 * cs[1].x + a1 * cs[1].y);
}

// kVec elements of each side of kVec pairs: 16- or 32-byte accesses.
template <int kVec>
__device__ __forceinline__ void rope_load(const uint16_t* p, uint32_t (&w)[kVec / 2]) {
  if constexpr (kVec == 16) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);              // plain loads: out may be in
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  }
}
template <int kVec>
__device__ __forceinline__ void rope_store(uint16_t* p, const uint32_t (&w)[kVec / 2]) {
  if constexpr (kVec == 16) store_32b(p, w);
  else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA turns `per_cta` tokens: it fills a table of {m cos, m sin} for its
// tokens (the angle pos * freq in turns, in 64 bits, reduced to [-1/2, 1/2]
// before it is rounded to 32), then each thread takes 2 kVec elements of a
// head: kVec pairs.  Bound by HBM: 4 bytes per element, in and out.  16384
// tokens of 40 heads of 128 (336 MB): 61 us, 5.5 TB/s (16-byte accesses: 63).
template <bool kInterleaved, int kVec>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs p, int per_cta) {
  extern __shared__ float2 cs_s[];                     // [per_cta][rot / 2]
  const int half = p.rot / 2;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * per_cta;
  const int n = static_cast<int>(min(static_cast<int64_t>(per_cta), p.T - t0));
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int t = static_cast<int>(fast_div(i, p.half_div)), f = i - t * half;
    double turns = static_cast<double>(__ldg(reinterpret_cast<const long long*>(p.pos) + t0 + t)) *
                   (__ldg(p.freq + f) * 0.15915494309189533577);
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * static_cast<float>(turns), &s, &c);
    cs_s[i] = make_float2(p.mscale * c, p.sign * (p.mscale * s));
  }
  __syncthreads();
  const int per_row = static_cast<int>(p.row_div.d), nv = static_cast<int>(p.head_div.d);
  for (int i = threadIdx.x; i < n * per_row; i += kThreads) {
    const int t = static_cast<int>(fast_div(i, p.row_div)), j = i - t * per_row;
    int head = static_cast<int>(fast_div(j, p.head_div));
    const int x = j - head * nv;
    const bool is_k = head >= p.hq;
    if (is_k) head -= p.hq;
    const uint16_t* src = (is_k ? p.k + (t0 + t) * p.ld_k : p.q + (t0 + t) * p.ld_q) + head * p.D;
    uint16_t* dst = (is_k ? p.k_out + (t0 + t) * p.ld_ko : p.q_out + (t0 + t) * p.ld_qo) + head * p.D;
    // the thread's two groups of kVec elements: both of its pairs' sides in the
    // half layout, 2 kVec neighbours in the interleaved one and past rot
    const bool turned = x < p.rot / (2 * kVec);
    const int e0 = (!kInterleaved && turned) ? kVec * x : 2 * kVec * x;
    const int e1 = (!kInterleaved && turned) ? half + kVec * x : 2 * kVec * x + kVec;
    uint32_t u[kVec / 2], w[kVec / 2];
    rope_load<kVec>(src + e0, u);
    rope_load<kVec>(src + e1, w);
    if (turned) {
      const float2* cs = cs_s + t * half + kVec * x;
#pragma unroll
      for (int e = 0; e < kVec / 2; ++e) {
        const float2 c2[2] = {cs[2 * e], cs[2 * e + 1]};
        if constexpr (kInterleaved) {                  // one pair per word
          uint32_t& a = e < kVec / 4 ? u[2 * e] : w[2 * e - kVec / 2];
          uint32_t& b = e < kVec / 4 ? u[2 * e + 1] : w[2 * e + 1 - kVec / 2];
          uint32_t ra, rb;
          rotate2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632), c2, ra, rb);
          a = __byte_perm(ra, rb, 0x5410);
          b = __byte_perm(ra, rb, 0x7632);
        } else {
          rotate2(u[e], w[e], c2, u[e], w[e]);
        }
      }
    }
    rope_store<kVec>(dst + e0, u);
    rope_store<kVec>(dst + e1, w);
  }
}

BlockMap block_map(const quads_kv_cache* c, int sides) {
  const int nb = c->head_dim / 16;                      // 4 or 8
  return BlockMap{make_fastdiv(static_cast<uint32_t>(sides * c->n_heads * nb)), c->n_heads * nb, nb == 4 ? 2 : 3, nb - 1};
}

// Rows of a CTA: as many as keep `want` items of work, fewer where the call
// is too small to give every SM four CTAs.
int rows_per_cta(int64_t rows, int per_row, int want) {
  int64_t n = want / (per_row > 0 ? per_row : 1);
  const int64_t spread = ceil_div(rows, int64_t(4) * num_sms());
  if (n > spread) n = spread;
  if (n > kMaxRows) n = kMaxRows;
  return static_cast<int>(n < 1 ? 1 : n);
}

}  // namespace
}  // namespace quads

using namespace quads;

extern "C" {

int quads_kv_cache_write(const quads_kv_cache* cache, const uint16_t* k, const uint16_t* v, int64_t rows, int64_t ld_k,
                         int64_t ld_v, const int32_t* row_off, const int32_t* kv_len, const int32_t* block_table,
                         int n_seqs, int max_pages, quads_stream_t stream) {
  clear_error();
  QUADS_TRY(check_cache(cache));
  QUADS_TRY(check_seqs(row_off, block_table, n_seqs, max_pages));
  const int64_t width = static_cast<int64_t>(cache->n_heads) * cache->head_dim;
  QUADS_REQUIRE(rows >= 0 && rows < (int64_t(1) << 31), QUADS_ERR_INVALID_ARG, "rows must be in [0, 2^31)");
  QUADS_REQUIRE(ld_k >= width && ld_v >= width && ld_k % 8 == 0 && ld_v % 8 == 0, QUADS_ERR_INVALID_ARG,
                "row strides must be multiples of 8 of at least n_heads * head_dim");
  if (rows == 0 || n_seqs == 0 || max_pages == 0 || cache->n_pages == 0) return QUADS_OK;
  QUADS_REQUIRE(k && v && kv_len, QUADS_ERR_INVALID_ARG, "null pointer");
  QUADS_REQUIRE(aligned(k, 16) && aligned(v, 16), QUADS_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  const CacheArgs c = cache_args(cache, block_table, n_seqs, max_pages);
  const BlockMap map = block_map(cache, 2);
  const int per = rows_per_cta(rows, static_cast<int>(map.row_div.d), 1024);
  const unsigned grid = static_cast<unsigned>(ceil_div(rows, int64_t(per)));
  if (aligned(k, 32) && aligned(v, 32) && ld_k % 16 == 0 && ld_v % 16 == 0)
    kv_write_kernel<true><<<grid, kThreads, 0, stream>>>(c, k, v, rows, ld_k, ld_v, map, row_off, kv_len, per);
  else
    kv_write_kernel<false><<<grid, kThreads, 0, stream>>>(c, k, v, rows, ld_k, ld_v, map, row_off, kv_len, per);
  count_launches(1);
  return check_launch("kv_write_kernel");
}

int quads_kv_cache_read(const quads_kv_cache* cache, const int32_t* row_off, const int32_t* start,
                        const int32_t* block_table, int n_seqs, int max_pages, int64_t rows, void* k_out, void* v_out,
                        int out_dtype, quads_stream_t stream) {
  clear_error();
  QUADS_TRY(check_cache(cache));
  QUADS_TRY(check_seqs(row_off, block_table, n_seqs, max_pages));
  QUADS_REQUIRE(rows >= 0 && rows < (int64_t(1) << 31), QUADS_ERR_INVALID_ARG, "rows must be in [0, 2^31)");
  QUADS_REQUIRE(out_dtype == QUADS_OUT_BF16 || out_dtype == QUADS_OUT_F32, QUADS_ERR_INVALID_ARG,
                "unknown output dtype %d", out_dtype);
  if (rows == 0 || n_seqs == 0) return QUADS_OK;
  QUADS_REQUIRE(k_out || v_out, QUADS_ERR_INVALID_ARG, "no output");
  QUADS_REQUIRE(aligned(k_out, 32) && aligned(v_out, 32), QUADS_ERR_INVALID_ARG, "outputs must be 32-byte aligned");
  const CacheArgs c = cache_args(cache, block_table, n_seqs, max_pages);
  const bool f32 = out_dtype == QUADS_OUT_F32;
  const BlockMap map = block_map(cache, (k_out != nullptr) + (v_out != nullptr));
  const int per = rows_per_cta(rows, static_cast<int>(map.row_div.d), 1024);
  const unsigned grid = static_cast<unsigned>(ceil_div(rows, int64_t(per)));
  if (f32)
    kv_read_kernel<true><<<grid, kThreads, 0, stream>>>(c, k_out, v_out, rows, map, row_off, start, per);
  else
    kv_read_kernel<false><<<grid, kThreads, 0, stream>>>(c, k_out, v_out, rows, map, row_off, start, per);
  count_launches(1);
  return check_launch("kv_read_kernel");
}

int quads_rope(const uint16_t* q, int64_t ld_q, int heads_q, const uint16_t* k, int64_t ld_k, int heads_k, int64_t T,
               int head_dim, const int64_t* positions, const double* freq, int rot_dim, int interleaved, float mscale,
               int inverse, uint16_t* q_out, int64_t ld_q_out, uint16_t* k_out, int64_t ld_k_out,
               quads_stream_t stream) {
  clear_error();
  QUADS_REQUIRE(T >= 0 && T < (int64_t(1) << 31), QUADS_ERR_INVALID_ARG, "T must be in [0, 2^31)");
  QUADS_REQUIRE(heads_q >= 0 && heads_k >= 0 && heads_q + heads_k >= 1 && heads_q <= 4096 && heads_k <= 4096,
                QUADS_ERR_INVALID_ARG, "1 to 4096 heads of each kind");
  QUADS_REQUIRE(head_dim >= 16 && head_dim <= 1024 && head_dim % 16 == 0, QUADS_ERR_UNSUPPORTED_SHAPE,
                "head_dim (%d) must be a multiple of 16 in [16, 1024]", head_dim);
  QUADS_REQUIRE(rot_dim >= 16 && rot_dim <= head_dim && rot_dim % 16 == 0, QUADS_ERR_UNSUPPORTED_SHAPE,
                "rot_dim (%d) must be a multiple of 16 in [16, head_dim]", rot_dim);
  const int64_t wq = static_cast<int64_t>(heads_q) * head_dim, wk = static_cast<int64_t>(heads_k) * head_dim;
  QUADS_REQUIRE(heads_q == 0 || (ld_q >= wq && ld_q_out >= wq && ld_q % 8 == 0 && ld_q_out % 8 == 0),
                QUADS_ERR_INVALID_ARG, "q's row strides must be multiples of 8 of at least heads_q * head_dim");
  QUADS_REQUIRE(heads_k == 0 || (ld_k >= wk && ld_k_out >= wk && ld_k % 8 == 0 && ld_k_out % 8 == 0),
                QUADS_ERR_INVALID_ARG, "k's row strides must be multiples of 8 of at least heads_k * head_dim");
  if (T == 0) return QUADS_OK;
  QUADS_REQUIRE((heads_q == 0 || (q && q_out)) && (heads_k == 0 || (k && k_out)) && positions && freq,
                QUADS_ERR_INVALID_ARG, "null pointer");
  QUADS_REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(q_out, 16) && aligned(k_out, 16) && aligned(positions, 8) &&
                    aligned(freq, 8),
                QUADS_ERR_INVALID_ARG, "q, k and the outputs must be 16-byte aligned");
  RopeArgs p{};
  p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
  p.T = T; p.ld_q = ld_q; p.ld_k = ld_k; p.ld_qo = ld_q_out; p.ld_ko = ld_k_out;
  p.pos = positions; p.freq = freq;
  p.hq = heads_q; p.hk = heads_k; p.D = head_dim; p.rot = rot_dim;
  p.mscale = mscale; p.sign = inverse ? -1.0f : 1.0f;
  auto wide = [](const void* a, int64_t ld) { return aligned(a, 32) && ld % 16 == 0; };
  const bool vec16 = rot_dim % 32 == 0 && head_dim % 32 == 0 && wide(q, ld_q) && wide(k, ld_k) && wide(q_out, ld_q_out) &&
                     wide(k_out, ld_k_out);
  const int nv = head_dim / (vec16 ? 32 : 16), per_row = (heads_q + heads_k) * nv;
  p.half_div = make_fastdiv(static_cast<uint32_t>(rot_dim / 2));
  p.row_div = make_fastdiv(static_cast<uint32_t>(per_row));
  p.head_div = make_fastdiv(static_cast<uint32_t>(nv));
  int per = rows_per_cta(T, per_row, 1024);
  per = per < 12288 / rot_dim ? per : 12288 / rot_dim;                               // table of at most 48 KB
  const size_t smem = static_cast<size_t>(per) * (rot_dim / 2) * sizeof(float2);
  const unsigned grid = static_cast<unsigned>(ceil_div(T, int64_t(per)));
  if (vec16) {
    if (interleaved) rope_kernel<true, 16><<<grid, kThreads, smem, stream>>>(p, per);
    else rope_kernel<false, 16><<<grid, kThreads, smem, stream>>>(p, per);
  } else {
    if (interleaved) rope_kernel<true, 8><<<grid, kThreads, smem, stream>>>(p, per);
    else rope_kernel<false, 8><<<grid, kThreads, smem, stream>>>(p, per);
  }
  count_launches(1);
  return check_launch("rope_kernel");
}

}  // extern "C"
