// Norms of queries and keys for each head, and their rotation by position, in one pass.
//
//   n = x rsqrt(mean x^2 + eps) w          (a, b) -> gain (a cos t - b sin t, a sin t + b cos t)
//
// for the pairs (a, b) of the first `rot` dims, t = position times the pair's frequency.  Frequencies are whole
// numbers of 2^-64 turns, so that position times frequency, taken modulo one turn, is one exact integer product however
// far the position is; its upper 32 bits go to the sine and cosine, which this hardware takes in turns, as fp32: to 2^-26
// of a turn.
//
// A lane holds 8 dims of a head.  A wave takes one token and PER times as many heads as fit in it, so that their
// angles are worked out once.
//
// Bound by reading and writing q and k once, a step by its launch: 4096 tokens of 32 + 32 heads of 128 dims, bf16, 134 MB,
// 23.6 us (5.7 TB/s; a large copy runs at 4.88, and the last cache holds part of these); five pieces of prompts, 128 + 8
// heads of 64 dims with norms and 32 of them turned, 59 MB, 17.3 us; 64 tokens of 64 + 8 heads 5.2 us.
#include "kv_device.h"
#include "kv_rotate.h"

namespace pik {

namespace {

enum : int { ROPE_HALF = 0, ROPE_INTERLEAVED = 1 };
constexpr int kRotateWaves = 4;

// Position of a row, and whether any sequence has it.
__device__ __forceinline__ bool row_position(const KvRotateArgs& A, int row, int& pos) {
  const KvView& c = A.c;
  if (A.positions != nullptr) {
    pos = A.positions[row];
    return row < c.starts[c.n];
  }
  int local;
  const int i = slot_owner(c, row, 1, 1, 0, local);
  const KvSeq s = kv_seq(c, i);
  pos = s.len - s.rows + (row - s.row0);
  return row >= s.row0 && row < s.row0 + s.rows;
}

template <int ACT, int D, int LAYOUT, int PER>
__global__ __launch_bounds__(WAVE* kRotateWaves) void k_kv_rotate(const KvRotateArgs A, const int parts) {
  using T = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  constexpr int kLanes = D / 8, kHeads = WAVE / kLanes;   // lanes of a head, heads of a wave at a time
  const int lane = threadIdx.x & (WAVE - 1), chunk = lane % kLanes;
  const long long job = (long long)blockIdx.x * kRotateWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int row = (int)(job / parts), part = (int)(job % parts);
  if (row >= A.c.rows) return;
  const int total = A.heads + A.c.kv_heads, h0 = part * (kHeads * PER) + lane / kLanes;

  V8 raw[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int h = h0 + p * kHeads;
    raw[p] = V8{};
    if (h < A.heads)
      raw[p] = *reinterpret_cast<const V8*>(static_cast<const T*>(A.q.data) + (int64_t)row * A.q.token +
                                            (int64_t)h * A.q.head + 8 * chunk);
    else if (h < total)
      raw[p] = *reinterpret_cast<const V8*>(static_cast<const T*>(A.k.data) + (int64_t)row * A.k.token +
                                            (int64_t)(h - A.heads) * A.k.head + 8 * chunk);
  }
  int pos;
  if (!row_position(A, row, pos)) return;

  // ---- this lane's angles: pair of dim 8 chunk + e ------------------------------------------------------
  const int half = A.rot / 2;
  const bool turned = 8 * chunk < A.rot, upper = LAYOUT == ROPE_HALF && 8 * chunk >= half;
  constexpr int kPairs = LAYOUT == ROPE_HALF ? 8 : 4;
  float cosine[kPairs], sine[kPairs];
  const int pair0 = LAYOUT == ROPE_HALF ? 8 * chunk - (upper ? half : 0) : 4 * chunk;
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    const uint64_t f = A.turns[turned ? pair0 + e : 0];
    const int t = (int)(((uint64_t)(int64_t)pos * f) >> 32);          // modulo one turn, nearest to 0
    const float turn = (float)t * 0x1p-32f;
    cosine[e] = A.gain * __builtin_amdgcn_cosf(turn);
    sine[e] = A.gain * __builtin_amdgcn_sinf(turn);
  }
  const int partner = lane + (upper ? -(half / 8) : half / 8);

#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int h = h0 + p * kHeads;
    const bool key = h >= A.heads;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)raw[p][e];
    const T* norm = static_cast<const T*>(key ? A.k_norm : A.q_norm);
    if (A.q_norm != nullptr || A.k_norm != nullptr) {
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
      sum += dpp_shuffled<0xB1>(sum);                        // over the head's 8 or 16 lanes
      sum += dpp_shuffled<0x4E>(sum);
      sum += dpp_shuffled<0x141>(sum);
      if constexpr (kLanes == 16) sum += dpp_shuffled<0x140>(sum);
      if (norm != nullptr) {
        const V8 w = *reinterpret_cast<const V8*>(norm + 8 * chunk);
        const float scale = rsqrtf(sum * (1.0f / D) + A.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * scale * (float)w[e];
      }
    }
    float y[8];
    if constexpr (LAYOUT == ROPE_HALF) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = __shfl(x[e], partner);
        y[e] = fmaf(x[e], cosine[e], (upper ? other : -other) * sine[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = fmaf(x[2 * e], cosine[e], -x[2 * e + 1] * sine[e]);
        y[2 * e + 1] = fmaf(x[2 * e + 1], cosine[e], x[2 * e] * sine[e]);
      }
    }
    V8 out;
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = (T)(turned ? y[e] : x[e]);
    if (h < A.heads)
      *reinterpret_cast<V8*>(static_cast<T*>(A.q_out.data) + (int64_t)row * A.q_out.token + (int64_t)h * A.q_out.head +
                             8 * chunk) = out;
    else if (h < total)
      *reinterpret_cast<V8*>(static_cast<T*>(A.k_out.data) + (int64_t)row * A.k_out.token +
                             (int64_t)(h - A.heads) * A.k_out.head + 8 * chunk) = out;
  }
}

template <int ACT, int D, int LAYOUT, int PER>
hipError_t rotate_go(const KvRotateArgs& a, hipStream_t s) {
  constexpr int kHeads = WAVE / (D / 8) * PER;
  const int parts = (a.heads + a.c.kv_heads + kHeads - 1) / kHeads;
  const long long grid = ((long long)a.c.rows * parts + kRotateWaves - 1) / kRotateWaves;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_kv_rotate<ACT, D, LAYOUT, PER>), dim3((unsigned)grid), dim3(WAVE * kRotateWaves), 0, s, a, parts);
  return hipGetLastError();
}

// A wave's position and angles serve more heads where there are waves enough without: by one, two or four times its
// heads, 64 tokens of 64 + 8 heads of 128 dims (1152 waves) take 4.5, 4.6 and 5.4 us, 300 (5400) 7.3, 6.3 and 6.6, 800 (14400)
// 13.6, 10.6 and 9.8, and 2000 28.2, 21.7 and 21.0.
template <int ACT, int D, int LAYOUT>
hipError_t rotate_any(const KvRotateArgs& a, hipStream_t s) {
  constexpr int kHeads = WAVE / (D / 8), kSimds = 1024, kFull = 8 * kSimds;
  const long long waves = (long long)a.c.rows * ((a.heads + a.c.kv_heads + kHeads - 1) / kHeads);
  if (waves < 2 * kSimds) return rotate_go<ACT, D, LAYOUT, 1>(a, s);
  return waves < kFull ? rotate_go<ACT, D, LAYOUT, 2>(a, s) : rotate_go<ACT, D, LAYOUT, 4>(a, s);
}

template <int ACT, int D>
hipError_t rotate_layout(int layout, const KvRotateArgs& a, hipStream_t s) {
  return layout == ROPE_HALF ? rotate_any<ACT, D, ROPE_HALF>(a, s) : rotate_any<ACT, D, ROPE_INTERLEAVED>(a, s);
}

}  // namespace

hipError_t launch_kv_rotate(int act, int layout, const KvRotateArgs& a, hipStream_t s) {
  if (act == ACT_F16) return a.c.dim == 128 ? rotate_layout<ACT_F16, 128>(layout, a, s) : rotate_layout<ACT_F16, 64>(layout, a, s);
  return a.c.dim == 128 ? rotate_layout<ACT_BF16, 128>(layout, a, s) : rotate_layout<ACT_BF16, 64>(layout, a, s);
}

}  // namespace pik
