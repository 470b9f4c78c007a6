// Attention of many rows of a sequence and key head (chunks of prompts: more
// than 48, or than 64 where the sequences' key heads are few): bound by the
// tensor cores and by the exponentials.
//
// A CTA takes 256 rows (two tiles of 128) of one key head: row r of a
// sequence is query head r % group of its token r / group, so the rows share
// every key.  Keys come in tiles of 128:
//   warps 8..11   convert a tile's E2M1 codes and E4M3 scales to FP16 (exact:
//                 at most 6 significant bits) in shared memory, a token per
//                 thread, keys and values in the same 128-byte-swizzled rows;
//   warp 12       issues S = Q_i K^T and O_i += P_i V (tcgen05, FP16
//                 operands, FP32 accumulators in tensor memory; V is read as
//                 the matrix whose reduction runs over its rows);
//   warps 0..3, 4..7  own tile 0 and 1, a row per thread: S goes to registers
//                 at once, so that one S serves both tiles; then its maximum,
//                 and exp(S - m) as FP16 to P_i (the A operand of the second
//                 product), the row's sum in FP32.
// Q_i K^T of the next keys runs during the exponentials of these, and the
// products of one tile during the other's.  O_i is rescaled only when a row's
// maximum has grown by more than 2^kLag since the last time, and begun anew
// after kChKeep tiles, its sums so far added to those in memory (a workspace,
// where the table is wide enough for such contexts).
// Tensor memory: S at column 0, P_0 and P_1 at 128 and 192, O_0 and O_1 at 256
// and 384.
//
// Measured on chunks of 4096 and 3793 tokens that end contexts of 12000 and
// 9909, 32 query and 8 key heads of 128 (1.17 TFLOP): 0.87 ms alone, 1340
// TFLOP/s, 0.82 of the measured burst of a library product; back to back under
// the power cap 0.97 ms in a graph, 0.87 of its sustained rate (1.00 ms as
// called with changing inputs, 0.85).  The tensor pipe is active 64 % of the cycles and so is the unit of exponentials; leaving out the
// exponentials changes nothing, leaving out the conversion 12 %.  The products'
// issue was the limit before: from one lane in a divergent branch 1.31 ms.
//
// Where the rows give fewer CTAs than SMs the keys are split too, and
// attention_join_kernel joins the parts.  Every wait is bounded.
#pragma once

#include "attention.cuh"
#include "sm100.cuh"

namespace quads {

constexpr int kChTile = 128;                     // rows of a tile, keys of a tile
constexpr int kChRows = 2 * kChTile;
constexpr int kChSoftWarps = 8;
constexpr int kChConvWarp = 8, kChConvWarps = 4;
constexpr int kChMmaWarp = 12;
constexpr int kChThreads = 512;                  // four warpgroups of 128 registers a thread, which they share out:
constexpr int kChRegs = 128, kChSoftRegs = 192, kChConvRegs = 88, kChMmaRegs = 40;
static_assert(2 * kChSoftRegs + kChConvRegs + kChMmaRegs <= 4 * kChRegs, "registers of the four warpgroups");
constexpr int kChStages = 2;
constexpr int kChKeep = kMaxAdds / (kChTile / 16);      // key tiles after which O_i is begun anew
static_assert((kChKeep & (kChKeep - 1)) == 0, "a power of two");
constexpr uint32_t kChPCol = 128, kChOCol = 256;   // P_i at kChPCol + 64 i, O_i at kChOCol + 128 i
constexpr uint64_t kChTimeoutNs = 4000000000ull, kChDrainNs = 500000000ull;
__host__ __device__ constexpr int ch_tile_bytes(int D) { return kChTile * D * 2; }
__host__ __device__ constexpr int ch_smem_bytes(int D) { return 1024 + (2 + 2 * kChStages) * ch_tile_bytes(D) + 256; }

// kind::f16 with FP16 operands and FP32 accumulators; trans_b: B's rows run
// along the reduction.
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool trans_b) {
  return (1u << 4) | (trans_b ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kChTile >> 4) << 24);
}
// B operand whose rows run along the reduction: 128-byte swizzled rows of 64
// elements, 8-row groups 1024 bytes apart, the next 64 elements 16 KB on.
__device__ __forceinline__ uint64_t desc_rows_sw128(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((kChTile * 128) >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// Set by a wait that gave up; read and cleared by quads_device_status().
__device__ unsigned int g_attention_wait_status = 0u;

__device__ __forceinline__ bool ch_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                        uint64_t limit_ns = kChTimeoutNs) {
  if (mbar_test(bar, parity)) return true;
  const uint64_t t0 = global_timer();
  while (true) {
    if (mbar_test(bar, parity)) return true;
    if (abort_flag != nullptr && *abort_flag) return false;
    if (global_timer() - t0 > limit_ns) {
      if (abort_flag != nullptr) *abort_flag = 1;
      atomicOr(&g_attention_wait_status, 1u);
      return false;
    }
  }
}

// ch_wait by a whole warp that goes on together.
__device__ __forceinline__ bool ch_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, ch_wait(bar, parity, abort_flag));
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
template <int kRegs>
__device__ __forceinline__ void regs_grow() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_shrink() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
// 32 columns of this warp's lanes, without waiting for them.
template <int kAt, int kN>
__device__ __forceinline__ void tmem_load32_at(uint32_t taddr, float (&r)[kN]) {
  uint32_t x[32];
  tmem_load32(taddr, x);
#pragma unroll
  for (int i = 0; i < 32; ++i) r[kAt + i] = __uint_as_float(x[i]);
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Bits first .. last of 32 columns that start at column c (first <= last or none).
__device__ __forceinline__ uint32_t column_mask(int first, int last, int c) {
  const int a = max(first - c, 0), b = min(last - c, 31);
  if (a > b) return 0u;
  return (0xFFFFFFFFu << a) & (0xFFFFFFFFu >> (31 - b));
}

// Rows of one CTA and the keys that they see.
struct ChUnit {
  SeqInfo s;
  int head;
  int row0;          // first row (of the sequence's nq * group)
  int t0, t1;        // key tiles of the CTA: [s.lo + 128 t0, s.lo + 128 t1)
};

// Key tiles (counted from s.lo) that rows [row0, row0 + n) see: [a, b).
__device__ __forceinline__ void ch_range(const AttnArgs& p, const SeqInfo& s, int row0, int n, int& a, int& b) {
  const int last = min(row0 + n, s.nq * p.group) - 1;
  if (last < row0) { a = b = 0; return; }
  const int pos_a = s.pos0 + static_cast<int>(fast_div(row0, p.group_div));
  const int pos_b = s.pos0 + static_cast<int>(fast_div(last, p.group_div));
  const int hi = max(min(s.hi, pos_b + 1), s.lo);
  const int lo = min(max(first_seen(p, pos_a), s.lo), hi);
  a = (lo - s.lo) / kChTile;
  b = (hi - s.lo + kChTile - 1) / kChTile;
}

// kKeep: contexts can be longer than kChKeep tiles.  (An instance of its own:
// a long chunk takes 1.5 % longer with it, windowed ones did 4 %.)
template <int D, bool kKeep>
__global__ void __launch_bounds__(kChThreads, 1) attention_chunk_kernel(AttnArgs p, int n_split) {
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  constexpr int kTB = ch_tile_bytes(D);
  const uint32_t q_s = base, k_s = base + 2 * kTB, v_s = k_s + kChStages * kTB;
  const uint32_t bar0 = v_s + kChStages * kTB;
  const uint32_t q_full = bar0, drain = bar0 + 8;
  auto k_full = [&](int s) { return bar0 + 16 + 8u * s; };
  auto k_empty = [&](int s) { return bar0 + 32 + 8u * s; };
  auto v_full = [&](int s) { return bar0 + 48 + 8u * s; };
  auto v_empty = [&](int s) { return bar0 + 64 + 8u * s; };
  auto s_full = [&](int i) { return bar0 + 80 + 8u * i; };
  auto p_full = [&](int i) { return bar0 + 96 + 8u * i; };
  auto pv_done = [&](int i) { return bar0 + 112 + 8u * i; };
  const uint32_t s_free = bar0 + 128;
  uint8_t* const misc = base_ptr + (bar0 + 136 - base);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  volatile uint32_t* const gone_s = reinterpret_cast<volatile uint32_t*>(misc + 8);   // [8]: groups of 16 keys without a page
  int* const unit_s = reinterpret_cast<int*>(misc + 40);                             // {sequence, block}

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform
  // the block'th 256 rows, counted through the sequences
  const int block = static_cast<int>(blockIdx.x) / p.c.n_heads;
  if (warp == 0) {
    int run = 0, found = -1, at = 0;
    for (int c0 = 0; c0 < p.c.n_seqs && found < 0; c0 += 32) {
      int n = 0;
      if (c0 + lane < p.c.n_seqs) {
        const SeqInfo s = seq_info(p, c0 + lane);
        n = (s.nq * p.group + kChRows - 1) / kChRows;
      }
      int incl = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, block < run + incl);
      if (hit) {
        const int l = __ffs(hit) - 1;
        found = c0 + l;
        // later rows see more keys: the longest blocks of a sequence first
        at = run + __shfl_sync(0xffffffffu, incl, l) - 1 - block;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      unit_s[0] = found;
      unit_s[1] = at;
    }
  }
  if (threadIdx.x == 32) {
    mbar_init(q_full, kChSoftWarps);
    mbar_init(drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full(i), kChConvWarps);
      mbar_init(k_empty(i), 1);
      mbar_init(v_full(i), kChConvWarps);
      mbar_init(v_empty(i), 1);
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), kChSoftWarps / 2);
      mbar_init(pv_done(i), 1);
    }
    mbar_init(s_free, kChSoftWarps / 2);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kChMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  const int b = unit_s[0];
  if (b >= 0) {
    ChUnit u;
    u.s = seq_info(p, b);
    u.head = static_cast<int>(blockIdx.x) - block * p.c.n_heads;
    u.row0 = unit_s[1] * kChRows;
    // this split's key tiles, and those of each row tile among them
    int ta[2], tb[2];
    ch_range(p, u.s, u.row0, kChTile, ta[0], tb[0]);
    ch_range(p, u.s, u.row0 + kChTile, kChTile, ta[1], tb[1]);
    const bool two = u.row0 + kChTile < u.s.nq * p.group;
    u.t0 = two ? min(ta[0], ta[1]) : ta[0];
    u.t1 = two ? max(tb[0], tb[1]) : tb[0];
    if (n_split > 1) {
      const int per = (u.t1 - u.t0 + n_split - 1) / n_split;
      u.t0 = min(u.t1, u.t0 + per * static_cast<int>(blockIdx.y));
      u.t1 = min(u.t1, u.t0 + per);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ta[i] = max(ta[i], u.t0);
      tb[i] = max(min(tb[i], u.t1), ta[i]);
    }

    if (warp < kChSoftWarps) {
      // ------------------------------------------------- softmax, a row each
      regs_grow<kChSoftRegs>();
      const int i = warp >> 2, r = threadIdx.x & 127;
      const int row = u.row0 + i * kChTile + r;
      const bool valid = row < u.s.nq * p.group;
      const int tok = valid ? static_cast<int>(fast_div(row, p.group_div)) : 0;
      const int head_q = u.head * p.group + (valid ? row - tok * p.group : 0);
      float c2;
      {
        // the row's queries, scaled by a power of two, as FP16
        const uint4* src = reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(u.s.r0 + tok) * p.ld_q + head_q * D);
        uint4 x[D / 8];
        uint32_t mx = 0;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          x[j] = valid ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(x[j].x & 0x7FFF7FFFu, x[j].y & 0x7FFF7FFFu),
                                     __vmaxu2(x[j].z & 0x7FFF7FFFu, x[j].w & 0x7FFF7FFFu)));
        }
        const uint32_t e = row_exponent(max(mx & 0xFFFFu, mx >> 16));
        const float down = exp_field_down(e);
        // the factor of the row's scores (to powers of two), positive: its sign goes to the queries, and so
        // does a NaN, which would reach masked scores too
        c2 = p.scale * kLog2e * kScaleUnit * __ldg(p.c.g_k + u.head) * exp_field_up(e);
        const float sign = c2 < 0.0f ? -down : c2 == c2 ? down : c2;
        c2 = fmaxf(fabsf(c2), kLeastFactor);
        const uint32_t dst = q_s + i * kTB + r * 128;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          st_shared_v4(dst + (j >> 3) * (kChTile * 128) + (((j & 7) ^ (r & 7)) << 4), bf16x2_scaled_f16x2(x[j].x, sign),
                       bf16x2_scaled_f16x2(x[j].y, sign), bf16x2_scaled_f16x2(x[j].z, sign),
                       bf16x2_scaled_f16x2(x[j].w, sign));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);

      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t s_col = tmem + lane_base, p_col = s_col + kChPCol + 64 * i, o_col = s_col + kChOCol + kChTile * i;
      const int pos = u.s.pos0 + tok, from = first_seen(p, pos);
      float xm = kNoMax, up = -kNoMax, l = 0.0f;        // the largest product so far; what is added to scores
      bool ok = true, far = false;
      // the row's place among the parts: there too are the sums that were taken out of O_i, at a largest of xm
      const auto part_at = [&] { return (static_cast<int64_t>(blockIdx.y) * p.rows + u.s.r0 + tok) * p.hq + head_q; };
      for (int t = ta[i]; t < tb[i]; ++t) {
        ok = ch_wait_warp(s_full(i), (t - ta[i]) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const int j0 = u.s.lo + t * kChTile;
        // columns [first, last] of the tile are seen
        const int last = valid ? min(pos, u.s.hi - 1) - j0 : -1;
        const int first = from - j0;
        uint32_t gone = gone_s[(t - u.t0) & 7];        // two bits in each byte: eight groups of 16 keys
        gone = (gone & 3u) | ((gone >> 6) & 0xCu) | ((gone >> 12) & 0x30u) | ((gone >> 18) & 0xC0u);
        const bool masked = __any_sync(0xffffffffu, last < kChTile - 1 || first > 0 || gone != 0);
        float x[kChTile];
        tmem_load32_at<0>(s_col, x);
        tmem_load32_at<32>(s_col + 32, x);
        tmem_load32_at<64>(s_col + 64, x);
        tmem_load32_at<96>(s_col + 96, x);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
        if (masked) {
#pragma unroll
          for (int c = 0; c < kChTile / 32; ++c) {
            uint32_t see = column_mask(first, last, 32 * c);
            if ((gone >> (2 * c)) & 1u) see &= 0xFFFF0000u;
            if ((gone >> (2 * c)) & 2u) see &= 0x0000FFFFu;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((see >> k) & 1u)) x[32 * c + k] = -CUDART_INF_F;
          }
        }
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmax3(x[k], x[k + 4], x[k + 8]);
#pragma unroll
        for (int k = 12; k < 124; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = fmax3(mx[e], x[k + e], x[k + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[124 + e]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (far || __any_sync(0xffffffffu, (top - xm) * c2 > kLag)) {
          // a new maximum: the first tile's, or one that has grown by kLag
          const float xn = fmaxf(xm, top), a = row_shrink(xm, xn, c2);
          xm = xn;
          up = row_shift(xn, c2);
          far = __any_sync(0xffffffffu, is_far(up));
          if (far && is_far(up)) {                      // every tile then comes here
            const uint64_t xm2 = pack_f32x2(-xm, -xm);
#pragma unroll
            for (int k = 0; k < kChTile; k += 2) {
              const uint64_t z = fadd2(pack_f32x2(x[k], x[k + 1]), xm2);
              x[k] = lo_f32(z);
              x[k + 1] = hi_f32(z);
            }
            up = kShift;
          }
          l *= a;
          if (t > ta[i]) {
            ok = ch_wait_warp(pv_done(i), (t - 1 - ta[i]) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_load16(o_col + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
              tmem_store16(o_col + 16 * c, o);
            }
          }
        }
        const uint64_t c22 = pack_f32x2(c2, c2), up2 = pack_f32x2(up, up);
        uint64_t sum[2] = {0ull, 0ull};
        uint32_t w[kChTile / 32][16];
#pragma unroll
        for (int c = 0; c < kChTile / 32; ++c)
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint64_t y = ffma2(pack_f32x2(x[32 * c + 2 * k], x[32 * c + 2 * k + 1]), c22, up2);
            const float e0 = ex2(lo_f32(y)), e1 = ex2(hi_f32(y));
            sum[k & 1] = fadd2(sum[k & 1], pack_f32x2(e0, e1));
            w[c][k] = pack_f16x2(e0, e1);
          }
        if (t > ta[i]) {                                // P_i has been read
          ok = ch_wait_warp(pv_done(i), (t - 1 - ta[i]) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll
        for (int c = 0; c < kChTile / 32; ++c) tmem_store16(p_col + 16 * c, w[c]);
        sum[0] = fadd2(sum[0], sum[1]);
        l += lo_f32(sum[0]) + hi_f32(sum[0]);
        if (kKeep && t > ta[i] && ((t - ta[i]) & (kChKeep - 1)) == 0) {   // the next product begins O_i anew
          const int64_t at = part_at();
          const bool first = t - ta[i] == kChKeep;
          const float f = first || !valid ? 0.0f : row_shrink(p.part_ml[at].x, xm, c2);
          if (valid) p.part_ml[at].x = xm;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_load16(o_col + 16 * c, o);
            tmem_wait_ld();
            if (valid) {
              float* const dst = p.kept + at * D + 16 * c;
#pragma unroll
              for (int k = 0; k < 16; ++k)
                dst[k] = first ? __uint_as_float(o[k]) : __fmaf_rn(dst[k], f, __uint_as_float(o[k]));
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(i));
      }
      if (ok && tb[i] > ta[i]) ok = ch_wait_warp(pv_done(i), (tb[i] - 1 - ta[i]) & 1, abort_flag);
      if (ok && (i == 0 || two)) {
        tc_fence_after();
        const bool some = tb[i] > ta[i];
        const int64_t orow = static_cast<int64_t>(u.s.r0 + tok) * p.hq + head_q, at = part_at();
        const bool kept = kKeep && valid && tb[i] - ta[i] > kChKeep;
        const float f = kept ? row_shrink(p.part_ml[at].x, xm, c2) : 0.0f;
        const auto add_kept = [&](uint32_t (&x)[32], int c) {
          const float* const src = p.kept + at * D + 32 * c;
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__fmaf_rn(src[k], f, __uint_as_float(x[k])));
        };
        if (n_split > 1) {
          if (valid) p.part_ml[at] = make_float2(row_max(xm, c2), l);
          if (some)
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t x[32];
              tmem_load32(o_col + 32 * c, x);
              tmem_wait_ld();
              if (kept) add_kept(x, c);
              if (valid) {
                uint4* dst = reinterpret_cast<uint4*>(p.part_o + at * D + 32 * c);
#pragma unroll
                for (int k = 0; k < 8; ++k) dst[k] = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
              }
            }
        } else {
          if (valid) l = row_sum(p, u.s, b, tok, l);
          const float inv = row_factor(p, u.head, l);
          if (valid && p.lse != nullptr) p.lse[orow] = l != 0.0f ? (row_max(xm, c2) - kShift) * kLn2 + logf(l) : -CUDART_INF_F;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t x[32];
            if (some) {
              tmem_load32(o_col + 32 * c, x);
              tmem_wait_ld();
              if (kept) add_kept(x, c);
            }
            if (valid) {
              uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + 32 * c);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int y = 8 * k + 2 * e;
                  // rows without a key: zeros, whatever the accumulator holds
                  w[e] = l != 0.0f && some ? pack_bf16x2(__uint_as_float(x[y]) * inv, __uint_as_float(x[y + 1]) * inv) : 0u;
                }
                dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
      }
    } else if (warp < kChConvWarp + kChConvWarps) {
      // -------------------------------------------- conversion, a token each
      regs_shrink<kChConvRegs>();
      const int r = threadIdx.x - 32 * kChConvWarp;     // token of the tile
      const int n = u.t1 - u.t0;
      auto lookup = [&](int t) -> uint32_t {
        const int j = u.s.lo + (u.t0 + t) * kChTile + r;
        if (t >= n || j >= u.s.hi) return kNoRow;
        int at;
        const int page = page_of(p.c, b, j, at);
        return page >= 0 ? static_cast<uint32_t>(cache_row(p.c, page, u.head, at)) : kNoRow;
      };
      uint4 kc[D / 32], vc[D / 32];
      uint32_t ks[D / 64], vs[D / 64];
      auto load = [&](const uint8_t* codes, const uint8_t* scales, uint32_t row, uint4 (&c)[D / 32], uint32_t (&s)[D / 64]) {
        if (row == kNoRow) {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) c[j] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < D / 64; ++j) s[j] = 0;
          return;
        }
        const uint4* src = reinterpret_cast<const uint4*>(codes + static_cast<uint64_t>(row) * (D / 2));
#pragma unroll
        for (int j = 0; j < D / 32; ++j) c[j] = __ldg(src + j);
        const uint32_t* ss = reinterpret_cast<const uint32_t*>(scales + static_cast<uint64_t>(row) * (D / 16));
#pragma unroll
        for (int j = 0; j < D / 64; ++j) s[j] = __ldg(ss + j);
      };
      auto convert = [&](uint32_t tile, const uint4 (&c)[D / 32], const uint32_t (&s)[D / 64]) {
        const uint32_t dst = tile + r * 128;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {               // 8 elements, one 16-byte chunk
          const uint32_t word = (&c[j >> 2].x)[j & 3];
          const uint32_t sc = scale_f16x2((s[j >> 3] >> (8 * ((j >> 1) & 3))) & 0x7Fu);
          uint32_t h[4];
          e2m1x8_to_f16x2(word, h);
          st_shared_v4(dst + (j >> 3) * (kChTile * 128) + (((j & 7) ^ (r & 7)) << 4), hmul2_rn(h[0], sc), hmul2_rn(h[1], sc),
                       hmul2_rn(h[2], sc), hmul2_rn(h[3], sc));
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      uint32_t row = lookup(0), next = lookup(1);
      load(p.c.k_codes, p.c.k_scales, row, kc, ks);
      load(p.c.v_codes, p.c.v_scales, row, vc, vs);
      for (int t = 0; t < n; ++t) {
        const int st = t % kChStages;
        const uint32_t free_parity = ((t / kChStages) & 1) ^ 1u;
        if (!ch_wait_warp(k_empty(st), free_parity, abort_flag)) break;
        // groups of 16 keys without a page (those past the last key are masked by position)
        const unsigned no = __ballot_sync(0xffffffffu, row == kNoRow);
        if (lane == 0)
          reinterpret_cast<volatile uint8_t*>(gone_s + (t & 7))[warp - kChConvWarp] =
              static_cast<uint8_t>((no & 1u) | ((no >> 15) & 2u));
        convert(k_s + st * kTB, kc, ks);
        if (lane == 0) mbar_arrive(k_full(st));
        const uint32_t after = lookup(t + 2);
        load(p.c.k_codes, p.c.k_scales, next, kc, ks);
        if (!ch_wait_warp(v_empty(st), free_parity, abort_flag)) break;
        convert(v_s + st * kTB, vc, vs);
        if (lane == 0) mbar_arrive(v_full(st));
        load(p.c.v_codes, p.c.v_scales, next, vc, vs);
        row = next;
        next = after;
      }
    } else {
      // ----------------------------------------------------------------- MMA
      regs_shrink<kChMmaRegs>();
      if (warp == kChMmaWarp) {
        // The whole warp keeps step, and one elected lane issues: descriptors
        // then stay in uniform registers.  (One lane alone in a branch took
        // about 110 cycles for each product, which is more than its 64.)
        constexpr uint32_t kIdQK = idesc_f16(kChTile, false), kIdPV = idesc_f16(D, true);
        const int n = u.t1 - u.t0;
        bool ok = ch_wait_warp(q_full, 0, abort_flag);
        auto active = [&](int i, int t) { return u.t0 + t >= ta[i] && u.t0 + t < tb[i]; };
        int used = 0;                                   // how often S has been written
        auto scores = [&](int i, int t) {               // S = Q_i K^T of tile t, once the last S has been read
          if (!active(i, t)) return;
          if (used && !ch_wait_warp(s_free, (used - 1) & 1, abort_flag)) { ok = false; return; }
          ++used;
          tc_fence_after();
          const uint64_t qd = desc_kmajor_sw128(q_s + i * kTB), kd = desc_kmajor_sw128(k_s + (t % kChStages) * kTB);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t at = ((kk >> 2) * (kChTile * 128) + (kk & 3) * 32) >> 4;
              mma_bf16(tmem, qd + at, kd + at, kIdQK, kk != 0);
            }
            tc_commit(s_full(i));
          }
          __syncwarp();
        };
        auto values = [&](int i, int t) {               // O_i += P_i V of tile t
          if (!active(i, t)) return;
          if (!ch_wait_warp(p_full(i), (u.t0 + t - ta[i]) & 1, abort_flag)) { ok = false; return; }
          tc_fence_after();
          const uint64_t vd = desc_rows_sw128(v_s + (t % kChStages) * kTB);
          const uint32_t more = (kKeep ? ((u.t0 + t - ta[i]) & (kChKeep - 1)) != 0 : u.t0 + t > ta[i]) ? 1u : 0u;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kChTile / 16; ++kk)
              mma_bf16_tmem_a(tmem + kChOCol + i * kChTile, tmem + kChPCol + 64 * i + 8 * kk, vd + kk * (2048 >> 4), kIdPV,
                              kk != 0 ? 1u : more);
            tc_commit(pv_done(i));
          }
          __syncwarp();
        };
        auto release = [&](uint32_t bar) {
          if (elect_one()) tc_commit(bar);
          __syncwarp();
        };
        for (int t = 0; t <= n && ok; ++t) {            // scores of tile t, values of tile t - 1
          if (t < n) ok = ch_wait_warp(k_full(t % kChStages), (t / kChStages) & 1, abort_flag);
          if (ok && t < n) scores(0, t);
          if (ok && t > 0) ok = ch_wait_warp(v_full((t - 1) % kChStages), ((t - 1) / kChStages) & 1, abort_flag);
          if (ok && t > 0) values(0, t - 1);
          if (ok && t < n) {
            scores(1, t);
            release(k_empty(t % kChStages));
          }
          if (ok && t > 0) {
            values(1, t - 1);
            release(v_empty((t - 1) % kChStages));
          }
        }
        // what was issued completes before the tensor memory is given back
        release(drain);
        ch_wait(drain, 0, nullptr, kChDrainNs);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kChMmaWarp) tmem_dealloc(tmem, 512);
}

// Joins the parts of rows whose keys were split: one warp per (row, head), the
// parts' weights a lane each.
template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(AttnArgs p, int n_split) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t r = item / p.hq;
  const int h = static_cast<int>(item - r * p.hq);
  bool mine = false;
  int b = -1;
  SeqInfo s{};
  if (r < p.rows) {
    b = warp_find_seq(p.off, p.c.n_seqs, static_cast<int>(r), lane);
    if (b >= 0) {
      s = seq_info(p, b);
      mine = r < s.r0 + s.nq;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");    // every block, so that this kernel ends after the first
  if (!mine) return;
  constexpr int kE = D / 32;
  const int64_t at = r * p.hq + h, step = p.rows * p.hq;
  float m = kNoMax;
  for (int i = lane; i < n_split; i += 32) m = fmaxf(m, __ldcg(p.part_ml + at + i * step).x);
#pragma unroll
  for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  float l = 0.0f, o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = 0.0f;
  for (int i0 = 0; i0 < n_split; i0 += 32) {
    float f = 0.0f;
    if (i0 + lane < n_split) {
      const float2 ml = __ldcg(p.part_ml + at + (i0 + lane) * step);
      f = ml.y != 0.0f ? ex2(ml.x - m) : 0.0f;           // a part without keys has no sums
      l += ml.y * f;
    }
    const int n = min(32, n_split - i0);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float w = __shfl_sync(0xffffffffu, f, i);
      float y[kE];
      if constexpr (kE == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + (at + (i0 + i) * step) * D) + lane);
        y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(p.part_o + (at + (i0 + i) * step) * D) + lane);
        y[0] = v.x; y[1] = v.y;
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) o[e] = w != 0.0f ? __fmaf_rn(y[e], w, o[e]) : o[e];
    }
  }
#pragma unroll
  for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  l = row_sum(p, s, b, static_cast<int>(r) - s.r0, l);
  const float inv = row_factor(p, h / p.group, l);
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * D + lane * kE);
#pragma unroll
  for (int e = 0; e < kE / 2; ++e) dst[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[at] = l != 0.0f ? (m - kShift) * kLn2 + logf(l) : -CUDART_INF_F;
}

}  // namespace quads
