// Attention of few rows (at most 16 per key head and sequence): bound by the
// bytes of the cache.
//
// A unit is (sequence, key head); its keys are cut into tiles of 64, and the
// tiles of all units, end to end, into equal runs, one per CTA, so that
// sequences of any lengths load the SMs alike.  A unit that spans several
// CTAs leaves partial sums that attention_combine_kernel joins in order.
//
// A CTA's four warps take 16 keys each of a tile, straight from global memory
// into the registers of the matrix instructions (m16n8k16, keys as M: the
// rows of up to 8 (16) queries are its N, so a group of 8 query heads wastes
// nothing):
//   S^T = K Q^T: a lane's 32 (16) elements of key g, g + 8 are one load; the
//   order of the elements along the reduction is free as long as Q's is the
//   same, so Q's registers are loaded in the same order;
//   O^T += V^T P^T: P^T comes from S^T's registers through a transposed move;
//   a lane's block of 16 (8) elements of values 2t, 2t+1, 2t+8, 2t+9 gives
//   the pairs along the keys that V^T needs by interleaving their 4-bit codes
//   before they are converted.
// E2M1 times E4M3 has at most 6 significant bits, so keys and values are
// exact in FP16.
#pragma once

#include "attention.cuh"

namespace quads {

constexpr int kDecThreads = 128;
constexpr int kDecWarps = kDecThreads / 32;
constexpr int kDecTile = 16 * kDecWarps;

__device__ __forceinline__ int dec_tiles(const SeqInfo& s) {
  if (s.nq <= 0) return 0;
  return max(1, (s.hi - s.lo + kDecTile - 1) / kDecTile);
}

// Tiles of all units, and the sequence that holds tile w, found by a block of
// kN threads (every thread gets the answer).
template <int kN>
struct DecPlan {
  int warp_s[kN / 32];
  int b;
  long long base;      // first tile of the sequence's first unit
  long long sum;

  __device__ __forceinline__ long long total(const AttnArgs& p) {
    const int lane = threadIdx.x & 31;
    long long n = 0;
    for (int i = threadIdx.x; i < p.c.n_seqs; i += kN) n += dec_tiles(seq_info(p, i));
#pragma unroll
    for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
    if (threadIdx.x == 0) sum = 0;
    __syncthreads();
    if (lane == 0 && n) atomicAdd(reinterpret_cast<unsigned long long*>(&sum), static_cast<unsigned long long>(n));
    __syncthreads();
    return sum * p.c.n_heads;
  }
  // w < total()
  __device__ __forceinline__ void find(const AttnArgs& p, long long w) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long run = 0;                                   // tiles (per head) before this chunk
    for (int c0 = 0; c0 < p.c.n_seqs; c0 += kN) {
      const int i = c0 + threadIdx.x;
      const int n = i < p.c.n_seqs ? dec_tiles(seq_info(p, i)) : 0;
      int incl = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      if (lane == 31) warp_s[warp] = incl;
      __syncthreads();
      long long before = run;
      int all = 0;
#pragma unroll
      for (int k = 0; k < kN / 32; ++k) {
        if (k < warp) before += warp_s[k];
        all += warp_s[k];
      }
      const long long first = (before + incl - n) * p.c.n_heads, last = (before + incl) * p.c.n_heads;
      if (n > 0 && w >= first && w < last) {
        b = i;
        base = first;
      }
      run += all;
      __syncthreads();
      if (w < run * p.c.n_heads) return;                 // the same for every thread
    }
  }
};

__device__ __forceinline__ long long dec_quota(long long total, int n_cta, int min_quota) {
  const long long q = (total + n_cta - 1) / n_cta;
  return q > min_quota ? q : min_quota;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t move_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A lane's part of 16 keys and values as they lie in the cache.
template <int D>
struct DecRaw {
  uint32_t k[2][D / 32];       // keys g, g + 8: 8 codes a word
  uint32_t ks[2];              // their scales: D / 64 bytes
  uint32_t v[4][D / 64];       // values 2t, 2t + 1, 2t + 8, 2t + 9
  uint32_t vs[4];

  __device__ __forceinline__ void load(const CacheArgs& c, int64_t row, int g, int t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = row + g + 8 * i;
      if constexpr (D == 128) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(c.k_codes + r * 64) + t);
        k[i][0] = x.x; k[i][1] = x.y; k[i][2] = x.z; k[i][3] = x.w;
        ks[i] = __ldg(reinterpret_cast<const uint16_t*>(c.k_scales + r * 8) + t);
      } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(c.k_codes + r * 32) + t);
        k[i][0] = x.x; k[i][1] = x.y;
        ks[i] = __ldg(c.k_scales + r * 4 + t);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = row + 2 * t + (i & 1) + 8 * (i >> 1);
      if constexpr (D == 128) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(c.v_codes + r * 64) + g);
        v[i][0] = x.x; v[i][1] = x.y;
        vs[i] = __ldg(c.v_scales + r * 8 + g);
      } else {
        v[i][0] = __ldg(reinterpret_cast<const uint32_t*>(c.v_codes + r * 32) + g);
        vs[i] = __ldg(c.v_scales + r * 4 + (g >> 1));
      }
    }
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kDecThreads, NT == 1 ? 4 : 3) attention_decode_kernel(AttnArgs p, int min_quota) {
  constexpr int kRows = 8 * NT;
  constexpr int kMT = D / 16;                           // 16-element tiles of O^T
  __shared__ float o_s[kDecWarps][kRows][D];
  __shared__ float2 ml_s[kDecWarps][kRows];
  __shared__ float f_s[kDecWarps][kRows];               // weight of each warp's sums; then 1 / l in [0]
  __shared__ DecPlan<kDecThreads> plan;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const long long total = plan.total(p);
  const long long quota = dec_quota(total, gridDim.x, min_quota);
  const long long w0 = quota * blockIdx.x, w1 = min(total, w0 + quota);
  if (w0 >= total) return;
  plan.find(p, w0);
  int b = plan.b;
  long long base = plan.base;

  for (long long w = w0; w < w1;) {
    SeqInfo s = seq_info(p, b);
    int nt = dec_tiles(s);
    while (w >= base + static_cast<long long>(nt) * p.c.n_heads) {      // on to the next sequence with rows
      base += static_cast<long long>(nt) * p.c.n_heads;
      s = seq_info(p, ++b);
      nt = dec_tiles(s);
    }
    const int head = static_cast<int>((w - base) / nt);
    const int tile0 = static_cast<int>(w - base - static_cast<long long>(head) * nt);
    const int tile1 = static_cast<int>(min(static_cast<long long>(nt), tile0 + (w1 - w)));
    const int R = min(s.nq * p.group, kRows);

    // queries: lane (g, t) holds elements [t D / 4, (t + 1) D / 4) of row g of each group of 8
    uint32_t qf[NT][D / 8];
    float c2[NT][2];                                    // score factor (to powers of two) of rows 2t, 2t + 1
    {
      const float base_f = p.scale * kLog2e * kScaleUnit * __ldg(p.c.g_k + head);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = 8 * n + g;
        uint32_t mx = 0;
        if (r < R) {
          const int tok = static_cast<int>(fast_div(r, p.group_div));
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + (s.r0 + tok) * p.ld_q + (head * p.group + (r - tok * p.group)) * D + t * (D / 4));
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint4 x = __ldg(src + i);
            qf[n][4 * i] = x.x; qf[n][4 * i + 1] = x.y; qf[n][4 * i + 2] = x.z; qf[n][4 * i + 3] = x.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) qf[n][i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) mx = __vmaxu2(mx, qf[n][i] & 0x7FFF7FFFu);
        mx = max(mx & 0xFFFFu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const uint32_t e = row_exponent(mx);
        const float down = exp_field_down(e);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) qf[n][i] = bf16x2_scaled_f16x2(qf[n][i], down);
        const float f = base_f * exp_field_up(e);       // row g's factor; rows 2t, 2t + 1 are lanes 8t, 8t + 4
        c2[n][0] = __shfl_sync(0xffffffffu, f, 8 * t);
        c2[n][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
      }
    }
    int pos[NT][2];                                     // positions of rows 2t, 2t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) pos[n][i] = s.pos0 + static_cast<int>(fast_div(8 * n + 2 * t + i, p.group_div));

    float o[NT][kMT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < kMT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
      m[n][0] = m[n][1] = -CUDART_INF_F;
      l[n][0] = l[n][1] = 0.0f;
    }

    // the warp's steps of 16 keys, one per tile; a step's keys share a page
    const int pos_last = s.pos0 + s.nq - 1;
    auto key0 = [&](int tile) { return s.lo + tile * kDecTile + 16 * warp; };
    auto row_of = [&](int j, int64_t& row) {            // cache row of key j, false without a page
      if (j >= s.hi) return false;
      int at;
      const int page = page_of(p.c, b, j, at);
      row = page >= 0 ? cache_row(p.c, page, head, at) : 0;
      return page >= 0;
    };
    DecRaw<D> cur, nxt;
    int64_t row = 0, row2 = 0;
    bool have = row_of(key0(tile0), row);
    if (have) nxt.load(p.c, row, g, t);
    bool have2 = tile0 + 1 < tile1 && row_of(key0(tile0 + 1), row2);
    for (int tile = tile0; tile < tile1; ++tile) {
      const bool now = have;
      cur = nxt;
      have = have2;
      if (have) nxt.load(p.c, row2, g, t);
      have2 = tile + 2 < tile1 && row_of(key0(tile + 2), row2);
      if (!now) continue;
      const int j0 = key0(tile);

      // S^T = K Q^T
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        uint32_t a[4], bb[4];
        e2m1x8_to_f16x2(cur.k[0][j], a);
        e2m1x8_to_f16x2(cur.k[1][j], bb);
        const int sh = D == 128 ? 8 * (j >> 1) : 0;
        const uint32_t s0 = scale_f16x2(cur.ks[0] >> sh), s1 = scale_f16x2(cur.ks[1] >> sh);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = hmul2_rn(a[i], s0);
          bb[i] = hmul2_rn(bb[i], s1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(sc[n], a[0], bb[0], a[1], bb[1], qf[n][4 * j], qf[n][4 * j + 1]);
          mma_f16(sc[n], a[2], bb[2], a[3], bb[3], qf[n][4 * j + 2], qf[n][4 * j + 3]);
        }
      }
      // scores in powers of two; masked where a row does not see the key
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] *= c2[n][i & 1];
      if (j0 + 15 > s.pos0 || j0 + 16 > s.hi || (p.window > 0 && j0 <= pos_last - p.window)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + g + 8 * (i >> 1);
            const bool see = j <= pos[n][i & 1] && j < s.hi && (p.window <= 0 || j > pos[n][i & 1] - p.window);
            if (!see) sc[n][i] = -CUDART_INF_F;
          }
      }
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) over |= sc[n][i] > m[n][i & 1] + kLag;
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x = fmaxf(sc[n][i], sc[n][i + 2]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float mn = fmaxf(m[n][i], x);
            const float a = m[n][i] == -CUDART_INF_F ? 0.0f : ex2(m[n][i] - mn);
            m[n][i] = mn;
            l[n][i] *= a;
#pragma unroll
            for (int d = 0; d < kMT; ++d) {
              o[n][d][i] *= a;
              o[n][d][i + 2] *= a;
            }
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m0 = m[n][0] == -CUDART_INF_F ? 0.0f : m[n][0] - kShift;
        const float m1 = m[n][1] == -CUDART_INF_F ? 0.0f : m[n][1] - kShift;
        const float e0 = ex2(sc[n][0] - m0), e1 = ex2(sc[n][1] - m1), e2 = ex2(sc[n][2] - m0), e3 = ex2(sc[n][3] - m1);
        l[n][0] += e0 + e2;
        l[n][1] += e1 + e3;
        pb[n][0] = move_trans(pack_f16x2(e0, e1));
        pb[n][1] = move_trans(pack_f16x2(e2, e3));
      }
      // O^T += V^T P^T
      const uint32_t sa = scale_pair_f16x2(cur.vs[0], cur.vs[1]), sb = scale_pair_f16x2(cur.vs[2], cur.vs[3]);
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        // bytes {value 2t, value 2t + 1} of elements 0, 2, 4, 6 and 1, 3, 5, 7 of the word
        constexpr uint32_t kLow = 0x0F0F0F0Fu;
        uint32_t a0[4], a1[4], b0[4], b1[4];
        e2m1x8_to_f16x2((cur.v[0][j] & kLow) | ((cur.v[1][j] << 4) & ~kLow), a0);
        e2m1x8_to_f16x2(((cur.v[0][j] >> 4) & kLow) | (cur.v[1][j] & ~kLow), a1);
        e2m1x8_to_f16x2((cur.v[2][j] & kLow) | ((cur.v[3][j] << 4) & ~kLow), b0);
        e2m1x8_to_f16x2(((cur.v[2][j] >> 4) & kLow) | (cur.v[3][j] & ~kLow), b1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a0[i] = hmul2_rn(a0[i], sa);
          a1[i] = hmul2_rn(a1[i], sa);
          b0[i] = hmul2_rn(b0[i], sb);
          b1[i] = hmul2_rn(b1[i], sb);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * j + i], a0[i], a1[i], b0[i], b1[i], pb[n][0], pb[n][1]);
        }
      }
    }

    // join the four warps: rows 2t, 2t + 1 of each group, elements [g D / 8, (g + 1) D / 8)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[n][i];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const int r = 8 * n + 2 * t + i;
        if (g == 0) ml_s[warp][r] = make_float2(m[n][i], x);
        float4* dst = reinterpret_cast<float4*>(&o_s[warp][r][g * (D / 8)]);
#pragma unroll
        for (int d = 0; d < kMT / 2; ++d)
          dst[d] = make_float4(o[n][2 * d][i], o[n][2 * d][i + 2], o[n][2 * d + 1][i], o[n][2 * d + 1][i + 2]);
      }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == nt;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (w == w0 ? 0 : 1);
    if (threadIdx.x < R) {
      const int r = threadIdx.x;
      float mm = -CUDART_INF_F, ll = 0.0f;
#pragma unroll
      for (int i = 0; i < kDecWarps; ++i) mm = fmaxf(mm, ml_s[i][r].x);
#pragma unroll
      for (int i = 0; i < kDecWarps; ++i) {
        const float f = ml_s[i][r].x == -CUDART_INF_F ? 0.0f : ex2(ml_s[i][r].x - mm);
        f_s[i][r] = f;
        ll += ml_s[i][r].y * f;
      }
      if (whole) {
        const float inv = ll > 0.0f ? kScaleUnit * __ldg(p.c.g_v + head) / ll : 0.0f;
#pragma unroll
        for (int i = 0; i < kDecWarps; ++i) f_s[i][r] *= inv;
        if (p.lse != nullptr) {
          const int tok = static_cast<int>(fast_div(r, p.group_div));
          p.lse[static_cast<int64_t>(s.r0 + tok) * p.hq + head * p.group + (r - tok * p.group)] =
              ll > 0.0f ? (mm - kShift) * kLn2 + logf(ll) : -CUDART_INF_F;
        }
      } else {
        p.part_ml[slot * kRows + r] = make_float2(mm, ll);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < R * (D / 4); i += kDecThreads) {
      const int r = i / (D / 4), d = i - r * (D / 4);
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kDecWarps; ++k) {
        const float f = f_s[k][r];
        const float4 y = reinterpret_cast<const float4*>(o_s[k][r])[d];
        x.x += y.x * f; x.y += y.y * f; x.z += y.z * f; x.w += y.w * f;
      }
      if (whole) {
        const int tok = static_cast<int>(fast_div(r, p.group_div));
        const int64_t at = (static_cast<int64_t>(s.r0 + tok) * p.hq + head * p.group + (r - tok * p.group)) * D;
        reinterpret_cast<uint2*>(p.out + at)[d] = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
      } else {
        reinterpret_cast<float4*>(p.part_o + (slot * kRows + r) * D)[d] = x;
      }
    }
    __syncthreads();
    w += tile1 - tile0;
  }
}

// Joins the partial sums of the units that the runs of n_cta CTAs cut: block
// (c, y) takes rows y, y + gridDim.y, ... of the unit whose first cut is the
// start of run c + 1.  Four groups of D threads each take a quarter of the
// partials.
template <int D, int NT>
__global__ void __launch_bounds__(4 * D) attention_combine_kernel(AttnArgs p, int n_cta, int min_quota) {
  constexpr int kRows = 8 * NT;
  __shared__ DecPlan<4 * D> plan;
  __shared__ float o_s[4][D];
  __shared__ float2 ml_s[4];
  const long long total = plan.total(p);
  const long long quota = dec_quota(total, n_cta, min_quota);
  const long long cut = quota * (blockIdx.x + 1);
  if (cut < total) plan.find(p, cut);
  // every block waits for the sums, also one that has none to join, so that
  // this kernel's end comes after the first one's
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (cut >= total) return;
  const SeqInfo s = seq_info(p, plan.b);
  const int nt = dec_tiles(s);
  const int head = static_cast<int>((cut - plan.base) / nt);
  const long long first = plan.base + static_cast<long long>(head) * nt, last = first + nt;
  if (first == cut || cut - quota > first) return;
  const int c0 = blockIdx.x, c1 = static_cast<int>((last - 1) / quota);
  const int R = min(s.nq * p.group, kRows);
  const int grp = threadIdx.x / D, d = threadIdx.x - grp * D;
  for (int r = blockIdx.y; r < R; r += gridDim.y) {
    float m = -CUDART_INF_F, l = 0.0f, o = 0.0f;
#pragma unroll 4
    for (int c = c0 + grp; c <= c1; c += 4) {
      // the unit's first run ends with it (slot 1) unless it begins with it
      const int64_t slot = 2 * static_cast<int64_t>(c) + ((c == c0 && first != c0 * quota) ? 1 : 0);
      const float2 ml = __ldcg(p.part_ml + slot * kRows + r);
      const float y = __ldcg(p.part_o + (slot * kRows + r) * D + d);
      const float mn = fmaxf(m, ml.x);
      const float a = m == -CUDART_INF_F ? 0.0f : ex2(m - mn), f = ml.x == -CUDART_INF_F ? 0.0f : ex2(ml.x - mn);
      m = mn;
      l = l * a + ml.y * f;
      o = o * a + y * f;
    }
    o_s[grp][d] = o;
    if (d == 0) ml_s[grp] = make_float2(m, l);
    __syncthreads();
    if (grp == 0) {
      float mm = -CUDART_INF_F, ll = 0.0f, oo = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) mm = fmaxf(mm, ml_s[i].x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = ml_s[i].x == -CUDART_INF_F ? 0.0f : ex2(ml_s[i].x - mm);
        ll += ml_s[i].y * f;
        oo += o_s[i][d] * f;
      }
      const int tok = static_cast<int>(fast_div(r, p.group_div));
      const int64_t row = static_cast<int64_t>(s.r0 + tok) * p.hq + head * p.group + (r - tok * p.group);
      const float inv = ll > 0.0f ? kScaleUnit * __ldg(p.c.g_v + head) / ll : 0.0f;
      p.out[row * D + d] = static_cast<uint16_t>(float_to_bf16_bits(oo * inv));
      if (d == 0 && p.lse != nullptr) p.lse[row] = ll > 0.0f ? (mm - kShift) * kLn2 + logf(ll) : -CUDART_INF_F;
    }
    __syncthreads();
  }
}

}  // namespace quads
