// Products with 4-bit weights: y = W x + bias + add for one row or many.
//
// A code is u = q + 8.  Four bits put into the mantissa of 16.0 read 16 + u = 24 + q, in fp16 and in bf16, so two
// codes of a word become two operands of a matrix instruction with one `and` and one `or` (the word is rotated by
// four bits from pair to pair), and no conversion.  The 24 is taken off by the accumulator that the product
// begins with, c = -24 sum x over the group, itself a product of the same x with a constant: all of it in fp32, off
// by at most 2^-24 of 32 times the group's largest |x| a term.  Each group of 32 columns is one 16x16x32 product;
// its sum, times the scale, is added in fp32.
#include "kv_device.h"
#include "kv_linear.h"

namespace pik {

namespace {

template <int ACT> struct Code;
template <> struct Code<ACT_F16> {
  static constexpr unsigned kTurn = 6, kMask = 0x03C003C0u, kOne = 0x4C004C00u;   // 16.0, steps of 2^-6
  static constexpr unsigned kMinus = 0xCE00CE00u;                                  // -24.0
};
template <> struct Code<ACT_BF16> {
  static constexpr unsigned kTurn = 3, kMask = 0x00780078u, kOne = 0x41804180u;   // 16.0, steps of 2^-3
  static constexpr unsigned kMinus = 0xC1C0C1C0u;                                  // -24.0
};

template <int ACT>
__device__ __forceinline__ f32x4 product(const typename ActT<ACT>::V8& x, const typename ActT<ACT>::V8& w, f32x4 c) {
  if constexpr (ACT == ACT_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
}

// One word: eight columns of a row as 24 + q.
template <int ACT>
__device__ __forceinline__ typename ActT<ACT>::V8 operand(unsigned w) {
  using C = Code<ACT>;
  u32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    r[j] = (__builtin_amdgcn_alignbit(w, w, 4 * j) & C::kMask) | C::kOne;
  return __builtin_bit_cast(typename ActT<ACT>::V8, r);
}

// ---- laying out ----------------------------------------------------------------------------------------

// One wave a slab.
template <int ACT>
__global__ __launch_bounds__(256) void k_linear_pack(const uint8_t* __restrict__ w, const unsigned short* __restrict__ scales,
                                                     uint8_t* __restrict__ packed, int d_in, int d_out, int slabs,
                                                     long long count) {
  const long long at = (long long)blockIdx.x * (256 / WAVE) + threadIdx.x / WAVE;
  if (at >= count) return;
  const int lane = threadIdx.x & (WAVE - 1), slab = (int)(at % slabs);
  const long long row = at / slabs * kSlabRows + lane % 16;
  uint8_t* to = packed + (size_t)at * kSlabBytes;
#pragma unroll
  for (int piece = 0; piece < 2; ++piece) {
    u32x4 out;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = slab * kSlabCols + piece * 128 + 32 * j + 8 * (lane / 16);
      unsigned q = 0;
      if (row < d_out && col < d_in) q = *reinterpret_cast<const unsigned*>(w + (size_t)row * (d_in / 2) + col / 2);
      q ^= 0x88888888u;
      unsigned r = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r |= ((q >> (8 * i)) & 15u) << (4 * i) | ((q >> (8 * i + 4)) & 15u) << (16 + 4 * i);
      out[j] = r << Code<ACT>::kTurn | r >> (32 - Code<ACT>::kTurn);
    }
    *reinterpret_cast<u32x4*>(to + piece * 1024 + lane * 16) = out;
  }
  // two groups' scales a lane: lanes 4 r + p have those of row r, groups 2 p and 2 p + 1
  const long long srow = at / slabs * kSlabRows + lane / 4;
  unsigned s = 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int group = slab * 8 + 2 * (lane % 4) + e;
    if (srow < d_out && group < d_in / 32) s |= (unsigned)scales[(size_t)srow * (d_in / 32) + group] << (16 * e);
  }
  *reinterpret_cast<unsigned*>(to + 2048 + lane * 4) = s;
}

// ---- the product ---------------------------------------------------------------------------------------

constexpr int kLinearWaves = 8;

// A slab of one tile as a wave holds it.
struct Slab {
  u32x4 code[2];
  u32x4 scale;   // eight fp16: the groups of row lane % 16
};
__device__ __forceinline__ Slab load_slab(const uint8_t* p) {
  const int lane = threadIdx.x & (WAVE - 1);
  Slab s;
  s.code[0] = ld_stream(reinterpret_cast<const u32x4*>(p) + lane);
  s.code[1] = ld_stream(reinterpret_cast<const u32x4*>(p + 1024) + lane);
  s.scale = ld_stream(reinterpret_cast<const u32x4*>(p + 2048) + lane % 16);
  return s;
}

// A workgroup takes T tiles of 16 outputs and NB tiles of 16 rows; its waves take the slabs in turn.  Row t of a tile
// of rows stands in row 4 (t % 4) + t / 4 of the product, so that up to four rows leave one sum a lane (NI of 4
// registers hold rows).
template <int ACT, int NB, int NI, int T>
__global__ __launch_bounds__(WAVE* kLinearWaves) void k_linear(const LinearArgs A) {
  using E = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  extern __shared__ float s_part[];   // [waves][T][NB][NI][64]
  const int lane = threadIdx.x & (WAVE - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int waves = blockDim.x / WAVE;
  const int groups = (A.tiles + T - 1) / T;
  const int tile0 = (int)(blockIdx.x % groups) * T, row0 = (int)(blockIdx.x / groups) * (16 * NB);
  const int g = lane >> 4, slot = lane & 15;
  const E* xrow[NB];
  bool live[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int t = row0 + 16 * b + (slot >> 2) + 4 * (slot & 3);
    live[b] = t < A.rows;
    xrow[b] = static_cast<const E*>(A.x) + (int64_t)(live[b] ? t : 0) * A.x_stride;
  }
  const uint8_t* from[T];
#pragma unroll
  for (int j = 0; j < T; ++j) from[j] = A.packed + (size_t)min(tile0 + j, A.tiles - 1) * A.slabs * kSlabBytes;

  float acc[T][NB][NI];
#pragma unroll
  for (int j = 0; j < T; ++j)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[j][b][i] = 0.0f;
  const V8 minus = __builtin_bit_cast(V8, u32x4{Code<ACT>::kMinus, Code<ACT>::kMinus, Code<ACT>::kMinus, Code<ACT>::kMinus});

  Slab next[T];
  if (wave < A.slabs) {
#pragma unroll
    for (int j = 0; j < T; ++j) next[j] = load_slab(from[j] + (size_t)wave * kSlabBytes);
  }
  for (int s = wave; s < A.slabs; s += waves) {
    Slab cur[T];
#pragma unroll
    for (int j = 0; j < T; ++j) cur[j] = next[j];
    const int col = s * kSlabCols + 8 * g;
    if (s + waves < A.slabs) {
#pragma unroll
      for (int j = 0; j < T; ++j) next[j] = load_slab(from[j] + (size_t)(s + waves) * kSlabBytes);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // columns past the end have q = 0 and scale 0, whatever x they meet: the row's own last
      const int at = min(col + 32 * k, A.d_in - 8);
      V8 x[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        x[b] = V8{};
        if (live[b]) x[b] = *reinterpret_cast<const V8*>(xrow[b] + at);
      }
      f32x4 c[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) c[b] = product<ACT>(x[b], minus, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int j = 0; j < T; ++j) {
        const V8 w = operand<ACT>(cur[j].code[k / 4][k % 4]);
        const float scale = (float)as_h2(cur[j].scale[k / 2])[k % 2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const f32x4 p = product<ACT>(x[b], w, c[b]);
#pragma unroll
          for (int i = 0; i < NI; ++i) acc[j][b][i] = fmaf(p[i], scale, acc[j][b][i]);
        }
      }
    }
  }

  // ---- the waves' sums, in their order, and out ----------------------------------------------------------
  constexpr int kSums = T * NB * NI * WAVE;
#pragma unroll
  for (int j = 0; j < T; ++j)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < NI; ++i) s_part[wave * kSums + ((j * NB + b) * NI + i) * WAVE + lane] = acc[j][b][i];
  __syncthreads();
  for (int k = threadIdx.x; k < kSums; k += blockDim.x) {
    const int n16 = k % 16, q = k / 16 % 4, j = k / (WAVE * NI * NB), b = k / (WAVE * NI) % NB, i = k / WAVE % NI;
    const int t = row0 + 16 * b + q + 4 * i, n = (tile0 + j) * 16 + n16;
    if (t >= A.rows || n >= A.d_out) continue;
    float v = s_part[k];
    for (int w = 1; w < waves; ++w) v += s_part[w * kSums + k];
    if (A.bias != nullptr) v += A.bias[n];
    if (A.add != nullptr) v += (float)static_cast<const E*>(A.add)[(int64_t)t * A.add_stride + n];
    static_cast<E*>(A.y)[(int64_t)t * A.y_stride + n] = (E)v;
  }
}

template <int ACT, int NB, int NI, int T>
hipError_t linear_go(const LinearArgs& a, hipStream_t s) {
  const long long grid = (long long)((a.tiles + T - 1) / T) * ((a.rows + 16 * NB - 1) / (16 * NB));
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  const int waves = a.slabs < kLinearWaves ? a.slabs : kLinearWaves;
  hipLaunchKernelGGL((k_linear<ACT, NB, NI, T>), dim3((unsigned)grid), dim3(WAVE * waves),
                     (size_t)waves * T * NB * NI * WAVE * sizeof(float), s, a);
  return hipGetLastError();
}

template <int ACT>
hipError_t linear_any(const LinearArgs& a, hipStream_t s) {
  if (a.rows <= 4) return linear_go<ACT, 1, 1, 1>(a, s);
  if (a.rows <= 16) return linear_go<ACT, 1, 4, 2>(a, s);
  return linear_go<ACT, 2, 4, 2>(a, s);
}

}  // namespace

hipError_t launch_linear_pack(int act, const void* w, const void* scales, void* packed, int d_in, int d_out, hipStream_t s) {
  const int slabs = (d_in + kSlabCols - 1) / kSlabCols;
  const long long count = (long long)((d_out + kSlabRows - 1) / kSlabRows) * slabs, grid = (count + 3) / 4;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  if (act == ACT_F16)
    hipLaunchKernelGGL((k_linear_pack<ACT_F16>), dim3((unsigned)grid), dim3(256), 0, s, static_cast<const uint8_t*>(w),
                       static_cast<const unsigned short*>(scales), static_cast<uint8_t*>(packed), d_in, d_out, slabs, count);
  else
    hipLaunchKernelGGL((k_linear_pack<ACT_BF16>), dim3((unsigned)grid), dim3(256), 0, s, static_cast<const uint8_t*>(w),
                       static_cast<const unsigned short*>(scales), static_cast<uint8_t*>(packed), d_in, d_out, slabs, count);
  return hipGetLastError();
}

hipError_t launch_linear(int act, const LinearArgs& a, hipStream_t s) {
  return act == ACT_F16 ? linear_any<ACT_F16>(a, s) : linear_any<ACT_BF16>(a, s);
}

}  // namespace pik
