// Device-side building blocks of the attention cache's kernels: the 8-bit codes, the layout of a
// block, and the sequences of a call, with everything that only the device knows bounded here.
//
// A block is 32 tokens of one head: codes x * 2^-e rounded to nearest even, e the smallest integer with
// amax <= TOP * 2^e.  A power of two makes scaling exact, so a code is off by its own rounding alone:
// half a step of e4m3 (2^-4 of the value) or of a whole number (2^-8 of the block's largest).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "kv.h"

namespace pik {

typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16;
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum : int { ACT_F16 = 0, ACT_BF16 = 1 };
enum : int { CODE_E4M3 = 0, CODE_INT8 = 1 };

template <int ACT> struct ActT;
template <> struct ActT<ACT_F16> {
  using T = f16;
  using V8 = f16x8;
  static constexpr float kMax = 65504.0f;
};
template <> struct ActT<ACT_BF16> {
  using T = bf16;
  using V8 = bf16x8;
  static constexpr float kMax = 3.38953139e38f;   // (2 - 2^-7) 2^127
};

// 2^e for whole e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __builtin_bit_cast(float, (unsigned)(e + 127) << 23); }

// The smallest e with amax <= TOP * 2^e, kept in [-126, 127]; amax >= 0 and finite.  With
// amax = m * 2^x, m in [1, 2), and TOP = t * 2^y, t in [1, 2): e = x - y, one more where m > t.
template <int CODE>
__device__ __forceinline__ int block_exponent(float amax) {
  constexpr unsigned kTop = CODE == CODE_E4M3 ? 0x43E00000u : 0x42FE0000u;   // 448, 127
  const unsigned b = __builtin_bit_cast(unsigned, amax);
  const int e = (int)(b >> 23) - (int)(kTop >> 23) + ((b & 0x7FFFFFu) > (kTop & 0x7FFFFFu) ? 1 : 0);
  return b < 0x00800000u ? -126 : max(e, -126);
}

// Four codes in a word -> four fp16 values, exactly (e4m3: 4 significant bits from 2^-9 to 448; int8:
// whole numbers up to 127).  int8: the byte with its sign flipped, b = x + 128, in the mantissa of
// 1024.0 reads 1024 + b, and 1152 is taken off.
template <int CODE>
__device__ __forceinline__ void decode4(unsigned w, f16x2& lo, f16x2& hi) {
  if constexpr (CODE == CODE_E4M3) {
    lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
  } else {
    const unsigned u = w ^ 0x80808080u;
    const f16x2 bias = {(f16)1152.0f, (f16)1152.0f};
    lo = as_h2(__builtin_amdgcn_perm(0x64006400u, u, 0x07010700u)) - bias;
    hi = as_h2(__builtin_amdgcn_perm(0x64006400u, u, 0x07030702u)) - bias;
  }
}

// Eight codes (two words) as one operand of a matrix instruction.
template <int CODE>
__device__ __forceinline__ f16x8 decode8(unsigned a, unsigned b) {
  f16x2 h[4];
  decode4<CODE>(a, h[0], h[1]);
  decode4<CODE>(b, h[2], h[3]);
  return f16x8{h[0].x, h[0].y, h[1].x, h[1].y, h[2].x, h[2].y, h[3].x, h[3].y};
}

// Four values, scaled already, -> four codes in a word, to nearest even.  |x| <= TOP by the choice of e.
template <int CODE>
__device__ __forceinline__ unsigned encode4(float a, float b, float c, float d) {
  if constexpr (CODE == CODE_E4M3) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return (unsigned)w;
  } else {
    const int x = (int)rintf(a), y = (int)rintf(b), z = (int)rintf(c), t = (int)rintf(d);
    return (unsigned)(x & 0xFF) | (unsigned)(y & 0xFF) << 8 | (unsigned)(z & 0xFF) << 16 | (unsigned)(t & 0xFF) << 24;
  }
}

// Where token u (of 32) stands in a K block: half t and row r of the two 16-row tiles a 16x16x32
// product takes, so that a lane's eight scores are eight consecutive tokens.
__device__ __forceinline__ int k_half(int u) { return (u >> 2) & 1; }
__device__ __forceinline__ int k_row(int u) { return ((u >> 3) << 2) | (u & 3); }
__device__ __forceinline__ int k_token(int t, int r) { return ((r >> 2) << 3) | (t << 2) | (r & 3); }

// Byte of a page's block in a layer's codes; blocks are 32 * D bytes.
__device__ __forceinline__ size_t block_at(const KvView& c, int page, int head, int slot) {
  return ((size_t)page * c.kv_heads + head) * c.page_blocks + slot;
}

// One sequence of a call.
struct KvSeq {
  int seq;     // row of the table, -1 if out of range
  int len;     // tokens it holds; 0 if the length is out of range
  int row0;    // its first row
  int rows;    // its rows
};

__device__ __forceinline__ KvSeq kv_seq(const KvView& c, int i) {
  KvSeq s;
  const int r0 = min(max(c.starts[i], 0), c.rows), r1 = min(c.starts[i + 1], c.rows);
  const int q = c.seqs[i];
  s.seq = q >= 0 && q < c.max_seqs ? q : -1;
  // clamped before it is tested: with the test alone k_kv_step's widest variant for int8 and bf16 spilled 55 registers
  // more, 66.8 against 55.3 us for 8 tokens of 8 heads on 16 x 4000
  const int cap = c.max_pages * c.page_blocks * kKvBlock;
  s.len = s.seq >= 0 ? min(max(c.lens[q], 0), cap + 1) : 0;
  s.len = s.len > cap ? 0 : s.len;
  s.row0 = r0;
  s.rows = max(r1 - r0, 0);
  return s;
}

// Page of a sequence's block, -1 if there is none.
__device__ __forceinline__ int kv_page(const KvView& c, int seq, int block) {
  const int p = c.table[(size_t)seq * c.max_pages + block / c.page_blocks];
  return p >= 0 && p < c.pages ? p : -1;
}

// Work slots without a prefix sum: sequence i owns the slots from start_i * per / unit + i * extra
// (rounded down) up to the next sequence's; with `extra` 1 (or 2, where the rows begin anywhere in a
// unit) there is one for each unit its rows touch.  Returns the sequence that owns `slot`, found 64
// sequences at a time, and the slot's number within it.
__device__ __forceinline__ int slot_owner(const KvView& c, int slot, int per, int unit, int extra, int& local) {
  const int lane = threadIdx.x & (WAVE - 1);
  int owner = 0;
  local = slot;
  for (int base = 0; base < c.n; base += WAVE) {
    const int i = base + lane;
    const long long at = i < c.n ? (long long)min(max(c.starts[i], 0), c.rows) * per / unit + (long long)i * extra
                                 : 0x7fffffffffffll;
    const unsigned long long le = __ballot(at <= slot);
    if (le == 0) break;
    const int last = 63 - __builtin_clzll(le);
    owner = base + last;
    local = slot - (int)__builtin_amdgcn_readlane((int)at, last);
    if (le != ~0ull) break;
  }
  return __builtin_amdgcn_readfirstlane(owner);
}

}  // namespace pik
