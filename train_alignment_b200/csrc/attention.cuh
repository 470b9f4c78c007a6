// What the attention kernels share (internal).
#pragma once

#include <math_constants.h>

#include "kvcache.cuh"

namespace quads {

struct AttnArgs {
  CacheArgs c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;               // nullable
  const int32_t* off;
  const int32_t* kv_len;
  int64_t rows, ld_q;
  int hq, group, max_q, window;
  float scale;
  FastDiv group_div;
  // partial results of units whose keys are split: per slot kRows rows of D
  // unnormalised sums, and {maximum, sum} of each row
  float* part_o;
  float2* part_ml;
  // sums taken out of the matrix instructions' accumulators (few rows: by CTA
  // and warp; many: in part_o), or null where no sum is long enough for that
  float* kept;
  // {slot of the first part or -1, CTA of the last, the sequence's first row *
  // n_heads + head, rows | first of them << 8} of each unit (by_unit), or of
  // the one that each CTA begins and does not end
  int4* cuts;
  int by_unit;
  int row_groups;           // units of a sequence and key head, at most
  int unit_cost;            // what beginning and ending a unit costs, in key tiles
};

// A matrix instruction adds the products of 16 keys to its FP32 sum and
// truncates: a sum of n additions comes out about n 2^-24 too small (measured
// with values of one sign: 2^16 additions 0.6 %, more than the rounding to
// BF16).  So after this many it is added to another in memory, rounded, and
// begun anew: 2^-11.4 at most.
constexpr int kMaxAdds = 4096;

// A sequence of a call: its rows, and the keys that they can see.
struct SeqInfo {
  int r0;      // first row
  int nq;      // rows that are computed
  int pos0;    // position of the first row (may be negative)
  int lo, hi;  // keys [lo, hi), lo a multiple of 16
};

// The first position that a row at pos sees: of a window, or 0.  (Rows before
// position 0 see none; pos - window stays within 32 bits for the others.)
__device__ __forceinline__ int first_seen(const AttnArgs& p, int pos) {
  return p.window > 0 ? max(max(pos, -1) - p.window + 1, 0) : 0;
}

__device__ __forceinline__ SeqInfo seq_info(const AttnArgs& p, int b) {
  const int rows = static_cast<int>(p.rows);
  const int off0 = __ldg(p.off + b), off1 = __ldg(p.off + b + 1);
  const int r0 = min(max(off0, 0), rows), r1 = min(max(off1, r0), rows);
  SeqInfo s;
  s.r0 = r0;
  s.nq = min(r1 - r0, p.max_q);
  // rows are fewer than 2^30: all are before position 0 if the first is that far
  const int64_t pos0 = max(static_cast<int64_t>(max(__ldg(p.kv_len + b), 0)) - (static_cast<int64_t>(off1) - off0), -(int64_t(1) << 30));
  s.pos0 = static_cast<int>(pos0);
  const int64_t cap = p.c.n_pages > 0 ? static_cast<int64_t>(p.c.max_pages) * p.c.page_size : 0;
  s.hi = static_cast<int>(max(int64_t(0), min(cap, pos0 + s.nq)));
  int64_t lo = p.window > 0 ? pos0 - p.window + 1 : 0;
  lo = min(max(lo, int64_t(0)), static_cast<int64_t>(s.hi));
  s.lo = static_cast<int>(lo) & ~15;
  return s;
}

// Queries are multiplied as 16-bit floats with 11 significant bits: a row is
// scaled by a power of two that brings its largest element to [2^14, 2^15), which
// keeps every BF16 element down to 2^-31 of the largest exact (smaller ones
// are off by 2^-39 of the largest).  The largest FP16 of a BF16 element is
// then 2^16 - 2^8 and a product of D with cached values at most 2^27, far from
// FP32's range.  Returns the row's exponent field, within what both factors hold.
constexpr uint32_t kQueryExp = 14;
__device__ __forceinline__ uint32_t row_exponent(uint32_t max_bf16_bits) {
  const uint32_t e = (max_bf16_bits >> 7) & 0xFFu;
  return min(max(e, kQueryExp + 1u), 253u);
}
__device__ __forceinline__ float exp_field_up(uint32_t e) { return __uint_as_float((e - kQueryExp) << 23); }           // 2^(e - 127 - 14)
__device__ __forceinline__ float exp_field_down(uint32_t e) { return __uint_as_float((254u + kQueryExp - e) << 23); }  // 2^(127 + 14 - e)

// Two BF16 (a word) times r -> two FP16.
__device__ __forceinline__ uint32_t bf16x2_scaled_f16x2(uint32_t w, float r) {
  uint32_t o;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(__uint_as_float(w & 0xFFFF0000u) * r), "f"(__uint_as_float(w << 16) * r));
  return o;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t o;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(hi), "f"(lo));
  return o;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// An E4M3 scale as {v, v} FP16 with v = val(s) * 2^-8: the code shifted into
// FP16's exponent and mantissa (bias 15 instead of 7; subnormals alike).
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t s) { return s * 0x00800080u; }
// Two such scales, without their sign bits: no code then gives a NaN or an
// infinity (0x7F gives 480 * 2^-8), so that bytes of places that nothing was
// written to cannot pass through a weight of zero.  (A score that is NaN is
// replaced where it is masked, so the keys' scales need no such care.)
__device__ __forceinline__ uint32_t scale_pair_f16x2(uint32_t s0, uint32_t s1) {
  return ((s0 + (s1 << 16)) & 0x007F007Fu) << 7;
}
constexpr float kScaleUnit = 256.0f;      // what the 2^-8 above is undone with

constexpr uint32_t kNoRow = 0xFFFFFFFFu;     // in place of a cache row: no page
constexpr float kNoMax = -3.402823466e38f;   // the running maximum before the first key: the lowest finite
                                             // number, so that no finite score is below it and
                                             // differences of maxima are never NaN

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's running maximum may fall this far (in powers of two) behind a new
// score before its sums are rescaled; weights are kept at 2^kShift times
// their value so that FP16 holds them from 2^-31 of the maximum's (2^-21 as a
// normal number) to 2^8.
constexpr float kLag = 8.0f;
constexpr float kShift = 7.0f;
// A weight is 2^(c (x - top) + kShift), x the matrix instructions' product, top
// the row's largest so far, c its factor.  c is positive; not zero, so that a
// first product is always above kNoMax and -inf times it is no NaN.
constexpr float kLeastFactor = 1e-37f;
// The kernel for many rows has it as one FMA, c x + shift.  The shift is
// rounded, alike for a row's weights, which does not matter up to kFar; at 2^27
// it is by more than what FP16 holds.  (The difference first, as the kernel for
// few rows has it for half a percent, costs a long chunk 2.5 %, windowed ones 5.)
constexpr float kFar = 16384.0f;
__device__ __forceinline__ float row_shift(float top, float c) { return top > kNoMax ? __fmaf_rn(-top, c, kShift) : -kNoMax; }
__device__ __forceinline__ bool is_far(float shift) { return fabsf(shift) > kFar && fabsf(shift) < -kNoMax; }
// What sums shrink by when the largest product grows.  (0 times an infinite c is
// NaN, which fminf drops.)
__device__ __forceinline__ float row_shrink(float top, float now, float c) { return ex2(fminf((top - now) * c, 0.0f)); }
// A row's largest score (to powers of two), as the joins compare it.
__device__ __forceinline__ float row_max(float top, float c) { return top > kNoMax ? top * c : kNoMax; }

// Whether a row at position pos of sequence b sees a key.  Asked where a row's
// sum of weights is zero: its visible scores, if there are any, are then all
// -inf (any finite one is a maximum at some point, and its weight not zero), and
// such a row has no softmax.
__device__ __forceinline__ bool sees_a_key(const AttnArgs& p, const SeqInfo& s, int b, int pos) {
  const int end = min(pos, s.hi - 1);
  for (int j = first_seen(p, pos); j <= end;) {
    int at;
    if (page_of(p.c, b, j, at) >= 0) return true;
    j += p.c.page_size - at;
  }
  return false;
}
// The last b with off[b] <= row (row >= off[0], off ascending, n + 1 entries), by one thread.
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ off, int n, int row) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(off + mid) <= row) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// A row's sum of weights: zero for a row that sees nothing, NaN for one without
// a softmax.
__device__ __forceinline__ float row_sum(const AttnArgs& p, const SeqInfo& s, int b, int tok, float l) {
  return l == 0.0f && sees_a_key(p, s, b, s.pos0 + tok) ? CUDART_NAN_F : l;
}
// What a row's sums are multiplied with.  Values are infinite or NaN (a code of
// zero) where their decode scale is infinite: NaNs then, as for a NaN.
__device__ __forceinline__ float row_factor(const AttnArgs& p, int head, float l) {
  const float g = __ldg(p.c.g_v + head);
  return l != 0.0f ? kScaleUnit * (g + (g - g)) / l : 0.0f;
}

}  // namespace quads
