// Attention of few rows: bound by the bytes of the cache and by the conversion
// of its codes.
//
// A unit is (sequence, key head, 8 NT of its rows); its keys are cut into
// tiles of 128, and the tiles of all units, end to end, into equal runs, one
// per CTA, so that sequences of any lengths load the SMs alike; a unit's tiles
// come after a few slots that stand for what beginning and ending it costs.  A
// unit that several CTAs share leaves partial sums that
// attention_combine_kernel joins in order.  Where contexts are short a CTA
// takes whole units and nothing is joined (one launch instead of two).
//
// A CTA's four warps take 32 keys each of a tile, from a ring in shared memory
// (cp.async, the next step's copies under this one's arithmetic) into the
// registers of the matrix instructions (m16n8k16, keys as M: the rows of up to
// 8 (16) queries are its N, so a group of 8 query heads wastes nothing):
//   S^T = K Q^T: a lane's 32 (16) elements of key g, g + 8 are one load; the
//   order of the elements along the reduction is free as long as Q's is the
//   same, so Q's registers are loaded in the same order;
//   O^T += V^T P^T: P^T comes from S^T's registers through a transposed move;
//   a lane's block of 16 (8) elements of values 2t, 2t+1, 2t+8, 2t+9 gives
//   the pairs along the keys that V^T needs by interleaving their 4-bit codes
//   before they are converted.
// E2M1 times E4M3 has at most 6 significant bits, so keys and values are
// exact in FP16.
//
// Why these instructions and not tcgen05 as in the kernel for many rows: of
// about 285 instructions for 16 keys, 128 convert codes and apply scales, which
// every layout needs; with keys in tensor memory the stores and the softmax on
// 128 lanes come to about 240, while a tile of 128 rows for 4 queries would
// wait on its own products.  Two groups of 16 keys at once hide each other's
// latency (one group, and four CTAs an SM instead of three: an eighth slower).
//
// Four contexts of up to 65536, 32 / 8 heads of 128 (170 MB): 38.4 us in a graph, 4.4 TB/s (41.0 as called).
// Of an earlier 43.9 the copies alone took 38.9, and conversion and scaling
// could hide but 2.8: what bounds it is the memory and a run's two ends.  Its
// first keys land 3.8 us after the launch, the join takes 2.5 (64 contexts of
// up to 4096, 87 MB: 25.1 us; 28.7 as called).  A deeper ring, the next unit's copies under this
// one's join, the values' products a step behind the scores' and unequal runs
// for the CTAs that share an SM changed nothing or cost 2 to 7 %.
#pragma once

#include "attention.cuh"

namespace quads {

constexpr int kDecThreads = 128;
constexpr int kDecWarps = kDecThreads / 32;
constexpr int kDecSub = 2;                            // groups of 16 keys of a warp's step
constexpr int kDecTile = 16 * kDecSub * kDecWarps;
// Resident CTAs of an SM: its registers hold 168 (255) a thread.  Four of 128
// (three of 168) are within 5 % at 8 rows and up to 40 % slower at 16.
__host__ __device__ constexpr int dec_ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }

// Key tiles of a sequence's units, and its units per head.
__device__ __forceinline__ int dec_tiles(const SeqInfo& s) {
  if (s.nq <= 0) return 0;
  return max(1, (s.hi - s.lo + kDecTile - 1) / kDecTile);
}
template <int kRows>
__device__ __forceinline__ int dec_groups(const AttnArgs& p, const SeqInfo& s) {
  return (max(s.nq, 0) * p.group + kRows - 1) / kRows;
}

// The run of this CTA: slots [w0, w1) of all units' (fewer than 2^30, checked
// on the host), and the sequence of the first with the first slot of its first
// unit.  Calls of up to kDecThreads sequences scan them once and keep them.
template <int kRows>
struct DecPlan {
  int warp_s[kDecWarps];
  int b, base;
  int quota, longer;       // slots of a run; the first so many runs have one more
  SeqInfo seq[kDecThreads];

  // slots (of one head's units) of sequences c0 .. c0 + kDecThreads - 1: this
  // thread's, those before it, and all
  __device__ __forceinline__ int scan(const AttnArgs& p, int c0, int& before, int& n) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = c0 + threadIdx.x;
    n = 0;
    if (i < p.c.n_seqs) {
      const SeqInfo s = seq_info(p, i);
      const int groups = dec_groups<kRows>(p, s);
      n = (dec_tiles(s) + p.unit_cost) * groups;
      seq[threadIdx.x] = s;
      if (p.by_unit && blockIdx.x == 0)                 // units that this sequence has not
        for (int h = 0; h < p.c.n_heads; ++h)
          for (int k = groups; k < p.row_groups; ++k)
            p.cuts[(i * p.c.n_heads + h) * p.row_groups + k] = make_int4(-1, 0, 0, 0);
    }
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) warp_s[warp] = incl;
    __syncthreads();
    before = incl - n;
    int all = 0;
#pragma unroll
    for (int k = 0; k < kDecWarps; ++k) {
      if (k < warp) before += warp_s[k];
      all += warp_s[k];
    }
    return all;
  }

  // false: nothing to do
  __device__ __forceinline__ bool run(const AttnArgs& p, int min_quota, int& w0, int& w1) {
    int before, n, all = 0;
    for (int c0 = 0; c0 < p.c.n_seqs; c0 += kDecThreads) {
      if (c0) __syncthreads();
      all += scan(p, c0, before, n);
    }
    const int total = all * p.c.n_heads;
    unsigned runs = static_cast<unsigned>(total);
    if (min_quota > 1) runs = (runs + min_quota - 1) / static_cast<unsigned>(min_quota);
    runs = min(runs, gridDim.x);
    if (blockIdx.x >= runs) return false;
    const int i = static_cast<int>(blockIdx.x), q = static_cast<int>(static_cast<unsigned>(total) / runs);
    const int more = total - q * static_cast<int>(runs);
    w0 = q * i + min(i, more);
    w1 = w0 + q + (i < more ? 1 : 0);
    if (threadIdx.x == 0) {
      quota = q;
      longer = more;
    }
    int run = 0;
    for (int c0 = 0;; c0 += kDecThreads) {
      if (p.c.n_seqs > kDecThreads) {
        __syncthreads();
        const int t = scan(p, c0, before, n);
        before += run;
        run += t;
      }
      if (n > 0 && w0 >= before * p.c.n_heads && w0 < (before + n) * p.c.n_heads) {
        b = c0 + threadIdx.x;
        base = before * p.c.n_heads;
      }
      if (p.c.n_seqs <= kDecThreads || w0 < run * p.c.n_heads) break;      // the same for every thread
    }
    __syncthreads();
    return true;
  }
  // the run of a slot
  __device__ __forceinline__ int run_of(int w) const {
    const int far = longer * (quota + 1);
    return w < far ? static_cast<int>(static_cast<unsigned>(w) / static_cast<unsigned>(quota + 1))
                   : longer + static_cast<int>(static_cast<unsigned>(w - far) / static_cast<unsigned>(quota));
  }
  __device__ __forceinline__ SeqInfo info(const AttnArgs& p, int i) const {
    return p.c.n_seqs <= kDecThreads ? seq[i] : seq_info(p, i);
  }
};

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

// A warp's ring of steps in shared memory: for each group of 16 keys their and
// their values' codes and scales as they lie in the cache, copied 16 bytes at
// a time.  Chunk c of a value's codes is at c ^ (key / 2 % 4) (D = 128), and
// key i of a matrix of eight is row i ^ (i / 2 % 2) of the group: both matrix
// operands are then read without bank conflicts.
constexpr int kDecStages = 2;
constexpr int kDecKeep = kMaxAdds / kDecSub;          // steps after which a warp's sums are begun anew
__host__ __device__ constexpr int dec_kept_floats(int D, int nt) { return 32 * (2 * nt + D / 4 * nt); }     // of a warp
__host__ __device__ constexpr int dec_stage_bytes(int D) { return 16 * (D + D / 8); }
__device__ __forceinline__ int dec_key(int i) { return i ^ ((i >> 1) & 1); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Where a lane copies its chunks of a group from (for row 0 of the cache) and
// to (for a place at 0).
template <int D>
struct DecCopy {
  static constexpr int kChunks = D / 32;                 // 16-byte chunks of a key's codes
  static constexpr int kScales = D / 16;                 // and of 16 keys' scales
  const uint8_t *k, *v, *s;
  uint32_t dst_v, dst_s;                                 // keys' codes: 16 * lane (+ 512)

  __device__ __forceinline__ DecCopy(const CacheArgs& c, int lane) {
    const int key = lane / kChunks, ch = lane % kChunks;
    const int sw = D == 128 ? ch ^ ((key >> 1) & 3) : ch;
    k = c.k_codes + 16 * lane;
    v = c.v_codes + 16 * lane;
    s = (lane < kScales ? c.k_scales : c.v_scales) + 16 * (lane % kScales);
    dst_v = 8 * D + key * (D / 2) + 16 * sw;
    dst_s = 16 * D + 16 * lane;
  }
  __device__ __forceinline__ void load(uint32_t row, uint32_t dst, int lane) const {
    const uint64_t at = static_cast<uint64_t>(row) * (D / 2);
#pragma unroll
    for (int i = 0; i < kChunks / 2; ++i) {              // key + 8: the same swizzle
      cp_async16(dst + 512 * i + 16 * lane, k + at + 512 * i);
      cp_async16(dst + 512 * i + dst_v, v + at + 512 * i);
    }
    if (lane < 2 * kScales) cp_async16(dst + dst_s, s + static_cast<uint64_t>(row) * (D / 16));
  }
};

// A lane's part of a group: keys g and g + 8, elements [t D / 4, (t + 1) D / 4);
// values 2t, 2t + 1, 2t + 8, 2t + 9, elements [g D / 8, (g + 1) D / 8).
template <int D>
struct DecRaw {
  uint32_t k[2][D / 32];       // 8 codes a word
  uint32_t ks[2];              // their scales: D / 64 bytes
  uint32_t v[4][D / 64];
  uint32_t vs[4];

  __device__ __forceinline__ void read_keys(const uint8_t* st, int g, int t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = dec_key(g) + 8 * i;
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(st + key * 64 + t * 16);
        k[i][0] = x.x; k[i][1] = x.y; k[i][2] = x.z; k[i][3] = x.w;
        ks[i] = *reinterpret_cast<const uint16_t*>(st + 16 * D + key * 8 + t * 2);
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(st + key * 32 + t * 8);
        k[i][0] = x.x; k[i][1] = x.y;
        ks[i] = st[16 * D + key * 4 + t];
      }
    }
  }
  __device__ __forceinline__ void read_values(const uint8_t* st, int g, int t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = dec_key(2 * t + (i & 1)) + 8 * (i >> 1);
      const uint8_t* const vp = st + 8 * D + key * (D / 2);
      if constexpr (D == 128) {
        const uint2 x = *reinterpret_cast<const uint2*>(vp + (((g >> 1) ^ ((key >> 1) & 3)) * 16) + (g & 1) * 8);
        v[i][0] = x.x; v[i][1] = x.y;
        vs[i] = st[16 * D + 128 + key * 8 + g];
      } else {
        v[i][0] = *reinterpret_cast<const uint32_t*>(vp + g * 4);
        vs[i] = st[16 * D + 64 + key * 4 + (g >> 1)];
      }
    }
  }
};

// kWhole: a CTA takes whole units.  kKeep: a run can have more than kDecKeep
// steps of a unit (an instance of its own: in the other it cost 1 %).
template <int D, int NT, bool kWhole, bool kKeep>
__global__ void __launch_bounds__(kDecThreads, dec_ctas_per_sm(NT)) attention_decode_kernel(AttnArgs p, int min_quota) {
  constexpr int kRows = 8 * NT;
  constexpr int kMT = D / 16;                           // 16-element tiles of O^T
  constexpr int kGroup = dec_stage_bytes(D), kStage = kDecSub * kGroup, kRing = kDecWarps * kDecStages * kStage;
  constexpr int kJoin = kDecWarps * kRows * D * 4;
  __shared__ __align__(128) uint8_t buf_s[kRing > kJoin ? kRing : kJoin];    // the warps' rings, then their sums
  float (*const o_s)[kRows][D] = reinterpret_cast<float (*)[kRows][D]>(buf_s);
  __shared__ float2 ml_s[kDecWarps][kRows];
  __shared__ float f_s[kDecWarps][kRows];               // weight of each warp's sums (of a whole unit: over the row's sum)
  __shared__ DecPlan<kRows> plan;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  // a run of slots [w0, w1), or (kWhole) units blockIdx.x, + gridDim.x, ...
  int w0 = blockIdx.x, w1 = p.c.n_seqs * p.c.n_heads * p.row_groups, b = 0, base = 0;
  bool told = false;                                    // thread 0: this run's cut is written
  if constexpr (!kWhole) {
    if (!plan.run(p, min_quota, w0, w1)) {
      if (!p.by_unit && threadIdx.x == 0) p.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
      return;
    }
    b = plan.b;
    base = plan.base;
  }

  for (int w = w0; w < w1;) {
    SeqInfo s;
    int nt, head, grp, tile0, tile1, next;              // grp: which 8 NT of the rows
    int left = 0;                                       // slots of the unit from w on
    if constexpr (kWhole) {
      const int bh = static_cast<int>(static_cast<unsigned>(w) / static_cast<unsigned>(p.row_groups));
      grp = w - bh * p.row_groups;
      b = static_cast<int>(static_cast<unsigned>(bh) / static_cast<unsigned>(p.c.n_heads));
      head = bh - b * p.c.n_heads;
      s = seq_info(p, b);
      nt = dec_tiles(s);
      tile0 = 0;
      tile1 = nt;
      next = w + static_cast<int>(gridDim.x);
      if (grp >= dec_groups<kRows>(p, s)) {
        w = next;
        continue;
      }
    } else {
      s = plan.info(p, b);
      nt = dec_tiles(s);
      int per_head = (nt + p.unit_cost) * dec_groups<kRows>(p, s);
      while (w >= base + per_head * p.c.n_heads) {      // on to the next sequence with rows
        base += per_head * p.c.n_heads;
        s = plan.info(p, ++b);
        nt = dec_tiles(s);
        per_head = (nt + p.unit_cost) * dec_groups<kRows>(p, s);
      }
      head = static_cast<int>(static_cast<unsigned>(w - base) / static_cast<unsigned>(per_head));
      const int rest = w - base - head * per_head;
      grp = static_cast<int>(static_cast<unsigned>(rest) / static_cast<unsigned>(nt + p.unit_cost));
      left = nt + p.unit_cost - (rest - grp * (nt + p.unit_cost));
      tile0 = max(nt - left, 0);
      tile1 = nt - max(left - (w1 - w), 0);
      next = w + min(left, w1 - w);
      if (tile1 <= 0) break;                            // the run ends before the unit's first tile
    }
    const int first_row = grp * kRows;
    const int R = min(s.nq * p.group - first_row, kRows);

    // The warp's steps of two groups of 16 keys, one step per tile.  A group's
    // keys share a page: lane i looks up the cache row of group i of 32, the
    // next 32 half way through these.  A group without a page reads row 0 and
    // masks it.
    const int from_last = first_seen(p, s.pos0 + s.nq - 1);             // the last row's first key
    const int j_first = s.lo + tile0 * kDecTile + 16 * kDecSub * warp;
    const int steps = min(tile1 - tile0, (s.hi - j_first + kDecTile - 1) / kDecTile);     // those with a key below hi
    auto lookup = [&](int group) -> uint32_t {
      const int j = j_first + (group / kDecSub) * kDecTile + 16 * (group % kDecSub);
      if (group >= kDecSub * steps || j >= s.hi) return 0u;
      int at;
      const int page = page_of(p.c, b, j, at);
      return page >= 0 ? static_cast<uint32_t>(cache_row(p.c, page, head, at)) : kNoRow;
    };
    uint32_t rows_now = lookup(lane), rows_next = 0u;
    uint32_t gone_now = __ballot_sync(0xffffffffu, rows_now == kNoRow), gone_next = 0u;   // bit i: group i has no page
    if (rows_now == kNoRow) rows_now = 0u;

    // one step being computed, the next on its way
    const uint8_t* const ring = buf_s + warp * (kDecStages * kStage);
    const uint32_t ring_a = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const DecCopy<D> copy(p.c, lane);
    auto fetch = [&](int step, int place) {
#pragma unroll
      for (int h = 0; h < kDecSub; ++h) {
        const uint32_t row = __shfl_sync(0xffffffffu, rows_now, (kDecSub * step + h) & 31);
        copy.load(row, ring_a + place * kStage + h * kGroup, lane);
      }
    };
    if (steps > 0) fetch(0, 0);
    cp_async_commit();

    // queries: lane (g, t) holds elements [t D / 4, (t + 1) D / 4) of row g of each group of 8
    uint32_t qf[NT][D / 8];
    float c2[NT][2];                                    // score factor (to powers of two) of rows 2t, 2t + 1
    {
      const float base_f = p.scale * kLog2e * kScaleUnit * __ldg(p.c.g_k + head);      // its sign, or that it is NaN, goes to the queries
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = 8 * n + g;
        uint32_t mx = 0;
        if (r < R) {
          const int tok = static_cast<int>(fast_div(first_row + r, p.group_div));
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + (s.r0 + tok) * p.ld_q + (head * p.group + (first_row + r - tok * p.group)) * D + t * (D / 4));
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
        const float down = base_f < 0.0f ? -exp_field_down(e) : base_f == base_f ? exp_field_down(e) : base_f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) qf[n][i] = bf16x2_scaled_f16x2(qf[n][i], down);
        const float f = fmaxf(fabsf(base_f) * exp_field_up(e), kLeastFactor);       // row g's factor; rows 2t, 2t + 1 are lanes 8t, 8t + 4
        c2[n][0] = __shfl_sync(0xffffffffu, f, 8 * t);
        c2[n][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
      }
    }
    // xm: a row's largest product so far
    float o[NT][kMT][4], xm[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < kMT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
      xm[n][0] = xm[n][1] = kNoMax;
      l[n][0] = l[n][1] = 0.0f;
    }

    auto attend = [&](const uint8_t* st, int j0, uint32_t gone) {
      DecRaw<D> x[kDecSub];
      // S^T = K Q^T
      float sc[kDecSub][NT][4];
#pragma unroll
      for (int h = 0; h < kDecSub; ++h) {
        x[h].read_keys(st + h * kGroup, g, t);
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[h][n][0] = sc[h][n][1] = sc[h][n][2] = sc[h][n][3] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int h = 0; h < kDecSub; ++h) {
          uint32_t a[4], bb[4];
          e2m1x8_to_f16x2(x[h].k[0][j], a);
          e2m1x8_to_f16x2(x[h].k[1][j], bb);
          const bool hi = D == 128 && j >= 2;
          const uint32_t s0 = scale_f16x2(hi ? x[h].ks[0] >> 8 : x[h].ks[0] & 0xFFu);
          const uint32_t s1 = scale_f16x2(hi ? x[h].ks[1] >> 8 : x[h].ks[1] & 0xFFu);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = hmul2_rn(a[i], s0);
            bb[i] = hmul2_rn(bb[i], s1);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(sc[h][n], a[0], bb[0], a[1], bb[1], qf[n][4 * j], qf[n][4 * j + 1]);
            mma_f16(sc[h][n], a[2], bb[2], a[3], bb[3], qf[n][4 * j + 2], qf[n][4 * j + 3]);
          }
        }
      // exponents of the weights; -inf where a row does not see the key
      float y[kDecSub][NT][4], top = -CUDART_INF_F;
#pragma unroll
      for (int h = 0; h < kDecSub; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) y[h][n][i] = __fmaf_rn(sc[h][n][i] - xm[n][i & 1], c2[n][i & 1], kShift);
      constexpr int kKeys = 16 * kDecSub;
      if (gone || j0 + kKeys - 1 > s.pos0 || j0 + kKeys > s.hi || j0 < from_last) {
#pragma unroll
        for (int h = 0; h < kDecSub; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + 16 * h + dec_key(g) + 8 * (i >> 1);
              const int pos = s.pos0 + static_cast<int>(fast_div(first_row + 8 * n + 2 * t + (i & 1), p.group_div));
              const bool see = !((gone >> h) & 1u) && j <= pos && j < s.hi && j >= first_seen(p, pos);
              if (!see) y[h][n][i] = -CUDART_INF_F;
            }
      }
      // the sums are rescaled only when a score is kLag above its row's
      // maximum so far
#pragma unroll
      for (int h = 0; h < kDecSub; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, y[h][n][i]);
      if (__any_sync(0xffffffffu, top > kShift + kLag)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float z = -CUDART_INF_F;
#pragma unroll
            for (int h = 0; h < kDecSub; ++h)
#pragma unroll
              for (int k = i; k < 4; k += 2)
                if (y[h][n][k] > -CUDART_INF_F) z = fmaxf(z, sc[h][n][k]);
            z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 4));
            z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 8));
            z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 16));
            const float xn = fmaxf(xm[n][i], z), a = row_shrink(xm[n][i], xn, c2[n][i]);
            xm[n][i] = xn;
            l[n][i] *= a;
#pragma unroll
            for (int d = 0; d < kMT; ++d) {
              o[n][d][i] *= a;
              o[n][d][i + 2] *= a;
            }
#pragma unroll
            for (int h = 0; h < kDecSub; ++h)
#pragma unroll
              for (int k = i; k < 4; k += 2)
                if (y[h][n][k] > -CUDART_INF_F) y[h][n][k] = __fmaf_rn(sc[h][n][k] - xn, c2[n][i], kShift);
          }
      }
      uint32_t pb[kDecSub][NT][2];
#pragma unroll
      for (int h = 0; h < kDecSub; ++h) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float e0 = ex2(y[h][n][0]), e1 = ex2(y[h][n][1]), e2 = ex2(y[h][n][2]), e3 = ex2(y[h][n][3]);
          l[n][0] += e0 + e2;
          l[n][1] += e1 + e3;
          pb[h][n][0] = move_trans(pack_f16x2(e0, e1));
          pb[h][n][1] = move_trans(pack_f16x2(e2, e3));
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int h = 0; h < kDecSub; ++h) {
        x[h].read_values(st + h * kGroup, g, t);
        const uint32_t sa = scale_pair_f16x2(x[h].vs[0], x[h].vs[1]), sb = scale_pair_f16x2(x[h].vs[2], x[h].vs[3]);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          // bytes {value 2t, value 2t + 1} of elements 0, 2, 4, 6 and 1, 3, 5, 7 of the word
          constexpr uint32_t kLow = 0x0F0F0F0Fu;
          uint32_t a0[4], a1[4], b0[4], b1[4];
          e2m1x8_to_f16x2((x[h].v[0][j] & kLow) | ((x[h].v[1][j] << 4) & ~kLow), a0);
          e2m1x8_to_f16x2(((x[h].v[0][j] >> 4) & kLow) | (x[h].v[1][j] & ~kLow), a1);
          e2m1x8_to_f16x2((x[h].v[2][j] & kLow) | ((x[h].v[3][j] << 4) & ~kLow), b0);
          e2m1x8_to_f16x2(((x[h].v[2][j] >> 4) & kLow) | (x[h].v[3][j] & ~kLow), b1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a0[i] = hmul2_rn(a0[i], sa);
            a1[i] = hmul2_rn(a1[i], sa);
            b0[i] = hmul2_rn(b0[i], sb);
            b1[i] = hmul2_rn(b1[i], sb);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * j + i], a0[i], a1[i], b0[i], b1[i], pb[h][n][0], pb[h][n][1]);
          }
        }
      }
    };

    // the sums of kDecKeep steps to those before, in memory (each lane its own):
    // rescaled from the maxima that they were kept at
    float* const kept = p.kept + (static_cast<size_t>(blockIdx.x) * kDecWarps + warp) * dec_kept_floats(D, NT) + lane;
    auto keep = [&](bool first, bool back) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float* const at = kept + 32 * (2 * n + i);
          const float f = first ? 0.0f : row_shrink(*at, xm[n][i], c2[n][i]);
          *at = xm[n][i];
#pragma unroll
          for (int d = 0; d < kMT; ++d)
#pragma unroll
            for (int k = i; k < 4; k += 2) {
              float* const x = kept + 32 * (2 * NT + (n * kMT + d) * 4 + k);
              const float sum = first ? o[n][d][k] : __fmaf_rn(*x, f, o[n][d][k]);
              if (!back) *x = sum;
              o[n][d][k] = back ? sum : 0.0f;
            }
        }
    };
    uint32_t gone_cur = gone_now;
    constexpr int kTurn = 32 / kDecSub;                 // steps of a look-up
    for (int step0 = 0; step0 < steps; step0 += kDecStages) {
      if (kKeep && step0 > 0 && step0 % kDecKeep == 0) keep(step0 == kDecKeep, false);
#pragma unroll
      for (int u = 0; u < kDecStages; ++u) {             // step0 + u lies in place u of the ring
        const int step = step0 + u;
        if (step >= steps) break;
        cp_async_wait<0>();
        __syncwarp();                                   // the step has landed, and the other place is free
        const int ahead = step + 1;
        if (u == 1) {                                   // ahead is even
          if (ahead % kTurn == kTurn / 2) {
            rows_next = lookup(kDecSub * (ahead + kTurn / 2) + lane);
            gone_next = __ballot_sync(0xffffffffu, rows_next == kNoRow);
            if (rows_next == kNoRow) rows_next = 0u;
          }
          if (ahead % kTurn == 0) {
            rows_now = rows_next;
            gone_now = gone_next;
          }
        }
        if (ahead < steps) fetch(ahead, 1 - u);
        cp_async_commit();
        if (u == 0 && step % kTurn == 0) gone_cur = gone_now;     // ahead has passed into this step's look-up
        attend(ring + u * kStage, j_first + step * kDecTile, (gone_cur >> (kDecSub * (step % kTurn))) & ((1u << kDecSub) - 1u));
      }
    }
    if (kKeep && steps > kDecKeep) keep(false, true);
    cp_async_wait<0>();
    __syncthreads();

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
        if (g == 0) ml_s[warp][r] = make_float2(row_max(xm[n][i], c2[n][i]), x);
        float4* dst = reinterpret_cast<float4*>(&o_s[warp][r][g * (D / 8)]);
#pragma unroll
        for (int d = 0; d < kMT / 2; ++d)
          dst[d] = make_float4(o[n][2 * d][i], o[n][2 * d][i + 2], o[n][2 * d + 1][i], o[n][2 * d + 1][i + 2]);
      }
    __syncthreads();
    const int slot = 2 * blockIdx.x + (w == w0 ? 0 : 1);
    const bool whole = kWhole || (tile0 == 0 && tile1 == nt);
    // the run that begins a unit says whether and where others go on with it
    if (!kWhole && tile0 == 0 && threadIdx.x == 0) {
      const int4 cut = make_int4(whole ? -1 : slot, plan.run_of(w + left - 1), s.r0 * p.c.n_heads + head, R | (first_row << 8));
      if (p.by_unit)
        p.cuts[(b * p.c.n_heads + head) * p.row_groups + grp] = cut;
      else if (!whole)
        p.cuts[blockIdx.x] = cut;
      told |= !whole;
    }
    if (threadIdx.x < R) {
      const int r = threadIdx.x;
      float mm = kNoMax, ll = 0.0f;
#pragma unroll
      for (int i = 0; i < kDecWarps; ++i) mm = fmaxf(mm, ml_s[i][r].x);
#pragma unroll
      for (int i = 0; i < kDecWarps; ++i) {
        const float f = ex2(ml_s[i][r].x - mm);
        f_s[i][r] = f;
        ll += ml_s[i][r].y * f;
      }
      if (whole) {
        const int tok = static_cast<int>(fast_div(first_row + r, p.group_div));
        ll = row_sum(p, s, b, tok, ll);
        const float inv = row_factor(p, head, ll);
#pragma unroll
        for (int i = 0; i < kDecWarps; ++i) f_s[i][r] *= inv;
        if (p.lse != nullptr) {
          p.lse[static_cast<int64_t>(s.r0 + tok) * p.hq + head * p.group + (first_row + r - tok * p.group)] =
              ll != 0.0f ? (mm - kShift) * kLn2 + logf(ll) : -CUDART_INF_F;
        }
      } else {
        p.part_ml[static_cast<int64_t>(slot) * kRows + r] = make_float2(mm, ll);
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
        const int tok = static_cast<int>(fast_div(first_row + r, p.group_div));
        const int64_t at = (static_cast<int64_t>(s.r0 + tok) * p.hq + head * p.group + (first_row + r - tok * p.group)) * D;
        reinterpret_cast<uint2*>(p.out + at)[d] = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
      } else {
        reinterpret_cast<float4*>(p.part_o + (static_cast<int64_t>(slot) * kRows + r) * D)[d] = x;
      }
    }
    __syncthreads();
    w = next;
  }
  if (!kWhole && !p.by_unit && threadIdx.x == 0 && !told) p.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
}

// Joins the partial sums of a unit that several runs share: block (x, y) takes
// rows y, y + gridDim.y, ... of the unit that cut x names.  Bound by latency: a
// group of D / 4 threads reads a row's part in one access each, eight parts in
// flight, and groups share a row where it has more parts than that.  (With D
// threads to a part, and its loads one by one: four contexts of up to 65536
// 42.2 us instead of 40.5, 16 of up to 8192 with 32 rows 34 instead of 26.5;
// twice the threads in a block 28.7 instead of 27.5 for 64 of up to 4096,
// because they find room only when the runs have ended.)
constexpr int kJoinThreads = 256;                        // for 8 rows

template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads * NT) attention_combine_kernel(AttnArgs p) {
  constexpr int kRows = 8 * NT, kLanes = D / 4, kThreads = kJoinThreads * NT, kGroups = kThreads / kLanes;
  static_assert(kGroups >= kRows, "a group for every row");
  __shared__ float4 o_s[kGroups][kLanes];
  __shared__ float2 ml_s[kGroups];
  // every block waits for the sums, also one that has none to join, so that
  // this kernel's end comes after the first one's
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 cut = __ldcg(p.cuts + blockIdx.x);          // slot of the first part, last run, place, rows
  if (cut.x < 0) return;
  const int c0 = cut.x >> 1, n = cut.y - c0 + 1, R = cut.w & 255, first_row = cut.w >> 8;
  const int rows = (R - static_cast<int>(blockIdx.y) + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
  if (rows <= 0) return;
  constexpr int kBatch = 8;                              // parts whose loads are in flight together
  const bool alone = n <= kBatch;                        // a group takes a row's parts alone
  int row_log2 = 0;                                      // rows of the block, rounded up to a power of two
  while ((1 << row_log2) < (alone ? kGroups : rows)) ++row_log2;
  const int splits = kGroups >> row_log2;
  const int r0 = cut.z / p.c.n_heads, head = cut.z - r0 * p.c.n_heads;
  const int grp = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int mine = grp & ((1 << row_log2) - 1);
  float m = kNoMax, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (mine < rows) {
    const int r = blockIdx.y + mine * gridDim.y;
    for (int i0 = grp >> row_log2; i0 < n; i0 += kBatch * splits) {
      float2 ml[kBatch];
      float4 y[kBatch];
      float mn = m;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * splits;                   // the unit's first part, then the first of each later run
        ml[u] = make_float2(kNoMax, 0.0f);
        y[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < n) {
          const int64_t at = static_cast<int64_t>(i == 0 ? cut.x : 2 * (c0 + i)) * kRows + r;
          ml[u] = __ldcg(p.part_ml + at);
          y[u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D) + lane);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) mn = fmaxf(mn, ml[u].x);
      const float a = ex2(m - mn);
      m = mn;
      l *= a;
      o.x *= a; o.y *= a; o.z *= a; o.w *= a;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float f = ex2(ml[u].x - mn);
        l += ml[u].y * f;
        o.x += y[u].x * f; o.y += y[u].y * f; o.z += y[u].z * f; o.w += y[u].w * f;
      }
    }
  }
  auto row_of = [&](int k) {
    const int r = first_row + blockIdx.y + k * gridDim.y, tok = static_cast<int>(fast_div(r, p.group_div));
    return static_cast<int64_t>(r0 + tok) * p.hq + head * p.group + (r - tok * p.group);
  };
  auto whole_sum = [&](int64_t row, float sum) {         // the sequence is looked for where it is needed
    if (sum != 0.0f) return sum;
    const int b = find_seq(p.off, p.c.n_seqs, r0);
    return row_sum(p, seq_info(p, b), b, static_cast<int>(row / p.hq) - r0, sum);
  };
  auto log_sum = [&](float max, float sum) { return sum != 0.0f ? (max - kShift) * kLn2 + logf(sum) : -CUDART_INF_F; };
  if (alone) {
    if (mine < rows) {
      const int64_t row = row_of(mine);
      l = whole_sum(row, l);
      const float inv = row_factor(p, head, l);
      reinterpret_cast<uint2*>(p.out + row * D)[lane] = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (lane == 0 && p.lse != nullptr) p.lse[row] = log_sum(m, l);
    }
    return;
  }
  o_s[grp][lane] = o;
  if (lane == 0) ml_s[grp] = make_float2(m, l);
  __syncthreads();
  for (int e = threadIdx.x; e < rows * D; e += kThreads) {
    const int k = e / D, d = e % D;
    float m = kNoMax, l = 0.0f, o = 0.0f;
    for (int i = 0; i < splits; ++i) m = fmaxf(m, ml_s[k + (i << row_log2)].x);
    for (int i = 0; i < splits; ++i) {
      const int g = k + (i << row_log2);
      const float2 ml = ml_s[g];
      const float f = ex2(ml.x - m);
      l += ml.y * f;
      o += reinterpret_cast<const float*>(o_s[g])[d] * f;
    }
    const int64_t row = row_of(k);
    l = whole_sum(row, l);
    p.out[row * D + d] = static_cast<uint16_t>(float_to_bf16_bits(o * row_factor(p, head, l)));
    if (d == 0 && p.lse != nullptr) p.lse[row] = log_sum(m, l);
  }
}

}  // namespace quads
