// What both attention kernels do to a tile of scores, and how their partial results are kept and joined.
//
// Scores come as S^T = K Q^T, so a lane holds one row of the queries and its registers hold tokens; P^T
// then stands in the registers as the other product, O^T = V^T P^T, takes it.  K's codes go in as fp16
// (exactly), and 2^ek, the softmax's scale and log2 e are one factor of the score.  V's codes go in as
// fp16 too; their 2^ev is added to the exponent, which costs nothing:
//     w_u = exp2(x_u + ev - rr + kBias),   O' = sum w_u code_u,   O = O' 2^(rr - kBias) / (l 2^mm)
// rr follows the largest x_u + ev seen, so w stays in fp16's range whatever the exponents are, and the
// softmax's own sum takes the factor back once for a block:
//     l = sum_blocks 2^(rr - kBias - ev - mm) sum_u w_u,     mm near the largest x_u.
// Both references only move when a block passes rr by more than kSlack or mm by more than kLead, so most
// blocks rescale nothing; w is then at most 2^(kBias + kSlack) = 2^15.  (With slack 5 and bias 10, 32 rows of
// scores with a deviation of 3 found one that moves in every other tile: a prompt of 4096 took 335 us
// instead of 324.)  A block whose V is so small that its tokens with x_u = mm lie more than 2^kFar below the row's
// largest product is taken as 2^kFar below, so that its w, which l needs, cannot underflow.  In O it cannot show: with
// x_u <= mm + kLead its w is at most 2^(kBias + kLead - kFar) = 2^-35, which is zero in fp16.  w is rounded to fp16,
// half a step of 2^-11, or 2^-25 / 2^kBias = 2^-30 of the row's largest where that is more; everything else is fp32.
#pragma once

#include "kv_device.h"

namespace pik {

constexpr float kBias = 5.0f, kSlack = 10.0f, kLead = 20.0f, kFar = 60.0f;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
// 2^(a - b) where a <= b and a may be -inf (then 0, whatever b is).
__device__ __forceinline__ float ex2_diff(float a, float b) { return a == -INFINITY ? 0.0f : ex2(a - b); }

// One row's state: references, and (this lane's part of) the sum.
struct RowState {
  float rr, mm, l;
};

// The same while blocks come in, with what weigh() takes of the references worked out when they move.
struct RowRun : RowState {
  float c, g;   // rr - kBias and rr - kBias - mm; 0 and -inf before the first score
};
__device__ __forceinline__ RowRun row_run() { return RowRun{{-INFINITY, -INFINITY, 0.0f}, 0.0f, -INFINITY}; }

// The factor of a block's scores, in the range in which no infinity or zero comes from it alone.
__device__ __forceinline__ float score_factor(float row, int ek) {
  return fminf(fmaxf(row * pow2i(ek), 1.17549435e-38f), 1.7e38f);
}

// Does this lane's largest score of the block, `top` (already scaled), pass the references?
__device__ __forceinline__ bool passes(const RowState& s, float top, float ev) {
  return top + ev > s.rr + kSlack || top > s.mm + kLead;
}

// New references from the row's largest score of the block (the same in all of the row's lanes);
// returns what O' has to be multiplied with.
__device__ __forceinline__ float move_refs(RowRun& s, float top, float ev) {
  const float rr = fmaxf(s.rr, top + ev), mm = fmaxf(s.mm, top);
  const float f = ex2_diff(s.rr, rr);
  s.l *= ex2_diff(s.mm, mm);
  s.rr = rr;
  s.mm = mm;
  s.c = rr > -INFINITY ? rr - kBias : 0.0f;
  s.g = rr > -INFINITY ? rr - kBias - mm : -INFINITY;
  return f;
}

// Scores s[N] of one block (raw sums; -inf where masked) -> fp16 weights, N = 8 or 16, and the row's sum.
template <int N>
__device__ __forceinline__ void weigh(RowRun& st, const float* s, float mul, float ev, f16x8* w) {
  const float e = fmaxf(ev, st.g - (kFar - kBias)), d = e - st.c;
  float sum = 0.0f;
#pragma unroll
  for (int q = 0; q < N / 8; ++q) {
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = ex2(fmaf(s[8 * q + j], mul, d));
    sum += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    w[q] = f16x8{(f16)p[0], (f16)p[1], (f16)p[2], (f16)p[3], (f16)p[4], (f16)p[5], (f16)p[6], (f16)p[7]};
  }
  st.l = fmaf(sum, ex2(st.g - e), st.l);
}

// O' -> out: 2^(rr - kBias - mm) can be far below what exp2 returns, so it is applied in two halves.
__device__ __forceinline__ float out_half(const RowState& s) {
  return s.l > 0.0f ? ex2(0.5f * (s.rr - kBias - s.mm)) : 0.0f;
}
__device__ __forceinline__ float out_value(float o, float l, float half) { return l != 0.0f ? o / l * half * half : 0.0f; }
// A row's value as it is returned: within the type's finite range, as stored values are read (the codes of the largest
// values stand for the next power of two).  A NaN, which only a query can bring, stays.  Each type has the form in which
// k_kv_step's variants of 64 rows keep their registers: fp16 the step back from infinity (the other form spills two
// registers more, 48.1 against 47.3 us for 8 tokens of 8 heads on 16 x 4000), bf16 the clamp (59.0 against 53.4 us).
template <int ACT>
__device__ __forceinline__ typename ActT<ACT>::T rounded(float x) {
  if constexpr (ACT == ACT_F16) {
    const unsigned short y = __builtin_bit_cast(unsigned short, (f16)x);
    return __builtin_bit_cast(f16, (unsigned short)((y & 0x7FFF) == 0x7C00 ? y - 1 : y));
  } else {
    const float y = __builtin_amdgcn_fmed3f(x, -ActT<ACT>::kMax, ActT<ACT>::kMax);
    return (typename ActT<ACT>::T)(x == x ? y : x);
  }
}
__device__ __forceinline__ float row_lse(const RowState& s) {
  return s.l > 0.0f ? (s.mm + log2f(s.l)) * kLn2 : (s.l == s.l ? -INFINITY : s.l);
}

// Joining partial results of a row: the sums of a's references with b's.  Returns the factors of O'.
__device__ __forceinline__ void join(RowState& a, const RowState& b, float& fa, float& fb) {
  const float rr = fmaxf(a.rr, b.rr), mm = fmaxf(a.mm, b.mm);
  fa = ex2_diff(a.rr, rr);
  fb = ex2_diff(b.rr, rr);
  a.l = a.l * ex2_diff(a.mm, mm) + b.l * ex2_diff(b.mm, mm);
  a.rr = rr;
  a.mm = mm;
}

// A query row's 8 dims at p as fp16.  bf16 queries are scaled by a power of two for the row, which brings
// their largest to [2^14, 2^15): what is lost lies 2^-39 below it, under the sums' own rounding.
template <int ACT>
__device__ __forceinline__ f16x8 query8(const typename ActT<ACT>::V8& x, float mul) {
  if constexpr (ACT == ACT_F16) return x;
  f16x8 r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = (f16)((float)x[e] * mul);
  return r;
}
template <int ACT>
__device__ __forceinline__ float max8(const typename ActT<ACT>::V8& x) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf((float)x[e]));
  return m;
}
// The row's power of two (returned) and its inverse, from the largest magnitude.
__device__ __forceinline__ float query_scale(float amax, float& inverse) {
  const int x = min(max((int)(__builtin_bit_cast(unsigned, amax) >> 23) - 127, -112), 127);
  inverse = pow2i(x - 14);
  return pow2i(14 - x);
}

// Which blocks of 32 tokens the rows of a sequence see: `sink` blocks from 0, then those from `from` up
// to `end`; p0 and p1 are the first and last position of the rows in question.
struct Span {
  int sink, from, end;
  __device__ __forceinline__ int count() const { return sink + end - from; }
  __device__ __forceinline__ int block(int i) const { return i < sink ? i : from + (i - sink); }
};
__device__ __forceinline__ Span span_of(int p0, int p1, int window, int sinks) {
  Span s{0, 0, p1 < 0 ? 0 : p1 / kKvBlock + 1};
  if (window > 0 && p0 >= window) {
    s.from = min((p0 - window + 1) / kKvBlock, s.end);
    s.sink = min((int)(((long long)sinks + kKvBlock - 1) / kKvBlock), s.from);
  }
  return s;
}

__device__ __forceinline__ bool row_sees(int p, int u, int window, int sinks) {
  return u <= p && (window == 0 || u > p - window || u < sinks);
}

// Fp32 partials pass between compute units in write-through stores (buffer cache policy sc1), which need
// no flush of a whole L2.
constexpr int kKvCoherent = 16;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t partial_rsrc(float* p) {
  return __builtin_amdgcn_make_buffer_rsrc(p, 0, 0x7fffffff, 0x00020000);
}
__device__ __forceinline__ void put4(__amdgpu_buffer_rsrc_t r, int word, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, 4 * word, 0, kKvCoherent);
}
__device__ __forceinline__ f32x4 get4(__amdgpu_buffer_rsrc_t r, int word) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, 4 * word, 0, kKvCoherent));
}

}  // namespace pik
