// Products with 4-bit weights: y = W x + bias + add for one row or many.
//
// A code is u = q + 8.  Four bits put into the mantissa of 16.0 read 16 + u = 24 + q, in fp16 and in bf16, so two
// codes of a word become two operands of a matrix instruction with one `and` and one `or` (the word is rotated by
// four bits from pair to pair), and no conversion.
//
// Up to 64 rows are bound by reading the codes and x, and nothing is rounded but sums in fp32: the 24 is taken
// off by the accumulator that a product begins with, c = -24 sum x over the group, itself a product of the same x
// with a constant; each group of 32 columns is one 16x16x32 product, and its sum, times the scale, is added in fp32.
// These sums round at the size of 24 x to 31 x, where q x has up to 8 x: up to 2600 * 2^-24 of a group's sum of |x|.
//
// More than 64 rows are bound by issue: on this hardware a vector ALU instruction runs beside a matrix instruction only in part
// (a 16x16x32 one and n others take 15.6 + 3.7 n cycles together, a 32x32x16 one, twice the work, 19 + 3.9 n), and an
// fp32 multiply-add for each output and group alone takes as many cycles as the product itself (2000 rows 4096 -> 12288:
// 328 us).  So there code times scale is an fp16 operand, rounded to half a step of 2^-11, no more than an fp16 y itself
// is, and the sums stay in 32x32x16 products.  bf16 rows are made fp16 for this, each by a power of two of its own, in the
// caller's scratch: what is lost lies 2^-39 below a row's largest.  On measured weights an fp16 y is off by 2.7e-4
// (relative, root mean square) where 64 rows' sums leave it at the 2.1e-4 of its own rounding, and a bf16 y by 1.7e-3 both ways.
//
// Measured (codes and scales read once at 6.99 TB/s; products at a library's 1166 to 1223 TFLOP/s): 1 row 8192 -> 10240 10.0 us
// (6.8); 16 rows 8192 -> 8192 11.3 to 12.4 (5.5); 64 rows 7168 -> 21504 45 to 47 (12.9; products 16.1), where each workgroup reads all of x
// from its L2, the vector ALU is busy 37 % of the time and the matrix instructions 20 %; 2000 rows 4096 -> 12288 232 (products 173;
// the library's own fp16 product of this size takes 187), the vector ALU busy 58 % and the matrix instructions 48 %.
#include "kv_linear.h"
#include "kv_softmax.h"

namespace pik {

namespace {

constexpr unsigned kTurn = 6;   // words are stored rotated left by as much, where fp16's operands have the first pair
template <int ACT> struct Code;
template <> struct Code<ACT_F16> {
  static constexpr unsigned kBack = 0, kMask = 0x03C003C0u, kOne = 0x4C004C00u;   // 16.0, steps of 2^-6
  static constexpr unsigned kMinus = 0xCE00CE00u;                                  // -24.0
};
template <> struct Code<ACT_BF16> {
  static constexpr unsigned kBack = 3, kMask = 0x00780078u, kOne = 0x41804180u;   // 16.0, steps of 2^-3
  static constexpr unsigned kMinus = 0xC1C0C1C0u;                                  // -24.0
};

template <int ACT>
__device__ __forceinline__ f32x4 product(const typename ActT<ACT>::V8& x, const typename ActT<ACT>::V8& w, f32x4 c) {
  if constexpr (ACT == ACT_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
}

// The exponent that makes operands of codes, in a register: an instruction that masks and joins takes one constant.
template <int ACT>
__device__ __forceinline__ unsigned sixteen() {
  unsigned one = Code<ACT>::kOne;
  asm volatile("" : "+v"(one));
  return one;
}

// One word: eight columns of a row as 24 + q.
template <int ACT>
__device__ __forceinline__ typename ActT<ACT>::V8 operand(unsigned w, unsigned one) {
  u32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = (__builtin_amdgcn_alignbit(w, w, 4 * j + Code<ACT>::kBack) & Code<ACT>::kMask) | one;
  return __builtin_bit_cast(typename ActT<ACT>::V8, r);
}

// ---- laying out ----------------------------------------------------------------------------------------

// One wave a row of scales: the power of two that they are divided by.  It brings a largest below 8 to [8, 16), so that most
// products of codes and scales are normal in fp16, and takes one of 2^13 and more below that, since -8 times it has to be
// finite (8 * 8188 = 65504).  Only the latter, by up to 8, can cost a scale bits: those below 2^-11 beside one of 2^13.  All
// others are multiples of fp16's smallest value after it as they were before, and so is code times scale where it is subnormal.
// (With every largest brought to [8, 16) a scale 2^-28 of it became 0, and was missing where x is 0 beside the large ones.)
__global__ __launch_bounds__(256) void k_linear_factor(const unsigned short* __restrict__ scales, float* __restrict__ factor,
                                                       int groups, int d_out, int padded) {
  const int row = blockIdx.x * (256 / WAVE) + threadIdx.x / WAVE, lane = threadIdx.x & (WAVE - 1);
  if (row >= padded) return;
  float top = 0.0f;
  if (row < d_out)
    for (int k = lane; k < groups; k += WAVE)
      top = fmaxf(top, fabsf((float)__builtin_bit_cast(f16, scales[(size_t)row * groups + k])));
#pragma unroll
  for (int m = 1; m < WAVE; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
  const int x = (int)(__builtin_bit_cast(unsigned, top) >> 23) - 127;   // top in [2^x, 2^(x + 1)), exact in fp32
  if (lane == 0) factor[row] = top > 0.0f && top <= 65504.0f ? pow2i(min(x - 3, max(x - 12, 0))) : 1.0f;
}

// One wave a slab.
__global__ __launch_bounds__(256) void k_linear_pack(const uint8_t* __restrict__ w, const unsigned short* __restrict__ scales,
                                                     uint8_t* __restrict__ packed, const float* __restrict__ factor, int d_in,
                                                     int d_out, int slabs, long long count) {
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
      out[j] = r << kTurn | r >> (32 - kTurn);
    }
    *reinterpret_cast<u32x4*>(to + piece * 1024 + lane * 16) = out;
  }
  // two groups' scales a lane: lanes 4 r + p have those of row r, groups 2 p and 2 p + 1
  const long long srow = at / slabs * kSlabRows + lane / 4;
  unsigned s = 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int group = slab * 8 + 2 * (lane % 4) + e;
    if (srow < d_out && group < d_in / 32) {
      const float scale = (float)__builtin_bit_cast(f16, scales[(size_t)srow * (d_in / 32) + group]);
      s |= (unsigned)__builtin_bit_cast(unsigned short, (f16)(scale / factor[srow])) << (16 * e);
    }
  }
  *reinterpret_cast<unsigned*>(to + 2048 + lane * 4) = s;
}

// ---- up to 64 rows -------------------------------------------------------------------------------------

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
__device__ __forceinline__ float scale_of(const Slab& s, int k) { return (float)as_h2(s.scale[k / 2])[k % 2]; }

template <int ACT>
__device__ __forceinline__ typename ActT<ACT>::V8 minus24() {
  constexpr unsigned m = Code<ACT>::kMinus;
  return __builtin_bit_cast(typename ActT<ACT>::V8, u32x4{m, m, m, m});
}

// Products of NB tiles that are still to be scaled and added: this is done beside the next ones, so that neither the
// matrix instructions nor the vector ALU wait for each other's results.
template <int NB> struct Late {
  f32x4 p[NB];
  float scale = 0.0f;
  __device__ __forceinline__ Late() {
#pragma unroll
    for (int b = 0; b < NB; ++b) p[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void set(const f32x4 (&now)[NB], float s) {
#pragma unroll
    for (int b = 0; b < NB; ++b) p[b] = now[b];
    asm volatile("" : "+v"(s));
    scale = s;
  }
  __device__ __forceinline__ void add(float (&acc)[NB][4]) const {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[b][i] = fmaf(p[b][i], scale, acc[b][i]);
  }
};
// One matrix instruction, then what the vector ALU does meanwhile.
template <int N>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int b = 0; b < N; ++b) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
  }
}

// The waves' sums [tile][rows' tile][i][lane], joined in the waves' order, and out.  Sum i of lane group q is row
// 4 q + i of its tile; with one sum a lane, row q.
template <int ACT, int NB, int NI, int T>
__device__ __forceinline__ void join_waves(const LinearArgs& A, float* s_part, const float (&acc)[T][NB][NI], int tile0,
                                           int row0, int wave, int waves) {
  using E = typename ActT<ACT>::T;
  constexpr int kSums = T * NB * NI * WAVE;
  const int lane = threadIdx.x & (WAVE - 1);
#pragma unroll
  for (int j = 0; j < T; ++j)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < NI; ++i) s_part[wave * kSums + ((j * NB + b) * NI + i) * WAVE + lane] = acc[j][b][i];
  __syncthreads();
  for (int k = threadIdx.x; k < kSums; k += blockDim.x) {
    // neighbouring threads have neighbouring outputs of a row
    const int n = (tile0 * 16) + k % (16 * T), r = k / (16 * T), i = r % NI, q = r / NI % 4, b = r / (4 * NI);
    const int t = row0 + 16 * b + NI * q + i;
    if (t >= A.rows || n >= A.d_out) continue;
    const int at = (((k % (16 * T) / 16) * NB + b) * NI + i) * WAVE + 16 * q + k % 16;
    float v = s_part[at];
    for (int w = 1; w < waves; ++w) v += s_part[w * kSums + at];
    v *= A.factor[n];
    if (A.bias != nullptr) v += A.bias[n];
    if (A.add != nullptr) v += (float)static_cast<const E*>(A.add)[(int64_t)t * A.add_stride + n];
    static_cast<E*>(A.y)[(int64_t)t * A.y_stride + n] = (E)v;
  }
}

// Up to four rows: bound by reading the codes.  A workgroup takes one tile, its waves the slabs in turn, two of them
// on their way while one is computed.  x goes through LDS, each wave's own slab of it, since as an operand each lane of
// 64 would load a row's 16 bytes again for all of a tile's 16 slots.
constexpr int kFewWaves = 8, kFewRows = 4;
template <int ACT, int B>
__global__ __launch_bounds__(WAVE* kFewWaves, 5) void k_linear_few(const LinearArgs A) {
  using E = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  typedef E E4 __attribute__((ext_vector_type(4)));
  __shared__ __align__(16) E s_x[kFewWaves][2][B][kSlabCols];
  __shared__ float s_part[kFewWaves * WAVE];
  const int lane = threadIdx.x & (WAVE - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int waves = blockDim.x / WAVE, tile = blockIdx.x, g = lane >> 4;
  const uint8_t* from = A.packed + (size_t)tile * A.slabs * kSlabBytes;
  const E* xrow[B];
#pragma unroll
  for (int b = 0; b < B; ++b) xrow[b] = static_cast<const E*>(A.x) + (int64_t)min(b, A.rows - 1) * A.x_stride;
  // this lane's four columns of a slab of each row, and the codes; past the last slab the last again, which nobody uses.
  // Columns past the end have q = 0 and scale 0, whatever x they meet: the row's own last.
  struct Stage {
    E4 x[B];
    Slab w;
  };
  auto load = [&](int s, Stage& to) {
    s = min(s, A.slabs - 1);
    const int col = min(s * kSlabCols + 4 * lane, A.d_in - 4);
#pragma unroll
    for (int b = 0; b < B; ++b) to.x[b] = *reinterpret_cast<const E4*>(xrow[b] + col);
    to.w = load_slab(from + (size_t)s * kSlabBytes);
  };
  float acc = 0.0f;
  const V8 minus = minus24<ACT>();
  const unsigned one = sixteen<ACT>();
  const int row = min((lane & 15) >> 2, B - 1);
  auto step = [&](int s, const Stage& cur, Stage& later, int buf) {
    load(s + 2 * waves, later);
#pragma unroll
    for (int b = 0; b < B; ++b) *reinterpret_cast<E4*>(&s_x[wave][buf][b][4 * lane]) = cur.x[b];
    __builtin_amdgcn_wave_barrier();   // a wave's LDS operations are done in their order
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const V8 v = *reinterpret_cast<const V8*>(&s_x[wave][buf][row][32 * k + 8 * g]);
      const f32x4 c = product<ACT>(v, minus, f32x4{0.f, 0.f, 0.f, 0.f});
      const f32x4 p = product<ACT>(v, operand<ACT>(cur.w.code[k / 4][k % 4], one), c);
      acc = fmaf(p[0], scale_of(cur.w, k), acc);
    }
    __builtin_amdgcn_wave_barrier();
  };
  Stage st[3];
  load(wave, st[0]);
  load(wave + waves, st[1]);
  for (int s = wave;; s += 6 * waves) {
#pragma unroll
    for (int e = 0; e < 6; ++e) {
      step(s + e * waves, st[e % 3], st[(e + 2) % 3], e % 2);
      if (s + (e + 1) * waves >= A.slabs) goto out;
    }
  }
out:
  const float sums[1][1][1] = {{{acc}}};
  join_waves<ACT, 1, 1, 1>(A, s_part, sums, tile, 0, wave, waves);
}

// x on its way to LDS: no registers, and in the order in which it lies in memory, 128 bytes of a row by eight lanes
// (as operands, lane after lane another row, an L1 takes 64 cycles for a load instead of 16).  A tile of 16 rows and 64
// columns is [16][8] units of 16 bytes; unit u of row r holds columns 8 (u ^ r % 8) .., which keeps the lanes of an
// operand on banks of their own.
constexpr int kStage = 64;                                   // columns
template <class V8> using XTile = V8[16][kStage / 8];
// Where lane l's part of a row of a stage begins, in bytes of the row: unit l % 8 of row l / 8 (of eight).  Columns past the
// end have q = 0 and scale 0, whatever x they meet: the row's own last.
__device__ __forceinline__ unsigned stage_byte(int col, int end) {
  const int lane = threadIdx.x & (WAVE - 1);
  return 2u * (unsigned)min(col + 8 * ((lane ^ (lane >> 3)) & 7), end - 8);
}
// 16 bytes a lane from base + at to LDS, lane after lane.  (To the compiler they are words: LDS is read as vectors, for which
// it does not wait.)
__device__ __forceinline__ void bring(const void* base, unsigned at, void* to) {
  const auto* from = reinterpret_cast<const __attribute__((address_space(1))) char*>(reinterpret_cast<uintptr_t>(base));
  __builtin_amdgcn_global_load_lds(reinterpret_cast<const __attribute__((address_space(1))) unsigned*>(from + at),
                                   (__attribute__((address_space(3))) unsigned*)to, 16, 0, 0);
}
// Operand of group k (0 or 1) of a tile.
template <class V8>
__device__ __forceinline__ V8 x_operand(const V8 (&x)[16][kStage / 8], int k) {
  const int lane = threadIdx.x & (WAVE - 1), r = lane & 15;
  return x[r][(4 * k + (lane >> 4)) ^ (r & 7)];
}
// At most N of this wave's loads are still on their way, and L of its LDS operations (15: any number).  (The builtin, since
// the compiler adds waits of its own where it does not know of one.)
template <int N, int L = 15>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0070 | L << 8);
  asm volatile("" ::: "memory");
}
template <int N> struct Count { static constexpr int value = N; };

// Up to 16 NB rows; T tiles a workgroup, whose waves take the slabs in turn.  Each wave brings the x of its own slabs to
// LDS, DEPTH - 1 stages of 64 columns ahead; codes come PRE slabs ahead.
template <int ACT, int NB, int T, int W, int DEPTH, int PRE>
__global__ __launch_bounds__(WAVE* W, 2) void k_linear_rows(const LinearArgs A) {
  using E = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  constexpr int kX = W * DEPTH * NB * 16 * kStage * 2, kPart = W * T * NB * 4 * WAVE * 4;
  __shared__ __align__(16) char s_mem[kX > kPart ? kX : kPart];
  const int lane = threadIdx.x & (WAVE - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int waves = blockDim.x / WAVE, tile0 = (int)blockIdx.x * T;
  XTile<V8>(*s_x)[NB] = reinterpret_cast<XTile<V8>(*)[NB]>(s_mem) + wave * DEPTH;
  unsigned xrow[2 * NB];
#pragma unroll
  for (int e = 0; e < 2 * NB; ++e)   // rows past the end are not stored
    xrow[e] = 2u * (unsigned)min(8 * e + (lane >> 3), A.rows - 1) * (unsigned)A.x_stride;
  const uint8_t* from[T];
#pragma unroll
  for (int j = 0; j < T; ++j) from[j] = A.packed + (size_t)min(tile0 + j, A.tiles - 1) * A.slabs * kSlabBytes;

  float acc[T][NB][4];
#pragma unroll
  for (int j = 0; j < T; ++j)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][b][i] = 0.0f;
  const V8 minus = minus24<ACT>();
  const unsigned one = sixteen<ACT>();
  // past a wave's last slab the matrix's last again, which nobody uses
  auto bring_stage = [&](int s, int q, int i) {   // stage q of slab s, the wave's i-th
    const unsigned at = stage_byte(min(s, A.slabs - 1) * kSlabCols + q * kStage, A.d_in);
#pragma unroll
    for (int e = 0; e < 2 * NB; ++e) bring(A.x, xrow[e] + at, &s_x[i % DEPTH][e / 2][8 * (e % 2)][0]);
  };
  auto load = [&](int s, Slab (&to)[T]) {
#pragma unroll
    for (int j = 0; j < T; ++j) to[j] = load_slab(from[j] + (size_t)min(s, A.slabs - 1) * kSlabBytes);
  };
  Late<NB> late;
  Slab w[PRE + 1][T];   // the slab at hand and the next ones
  // A stage is complete when all that was asked for before it is: behind it are the DEPTH - 2 stages after it, and a
  // slab's codes where they were asked for since.
  auto step = [&](int s, const Slab (&cur)[T], Slab (&later)[T]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      constexpr int kAfter = (DEPTH - 2) * 2 * NB;
      if (q > 0 && q < DEPTH)
        wait_loads<kAfter + 3 * T>();
      else
        wait_loads<kAfter>();
      bring_stage(s + (q + DEPTH - 1) / 4 * waves, (q + DEPTH - 1) % 4, q + DEPTH - 1);
      __builtin_amdgcn_sched_barrier(0);   // the counts above go by this order
      if (q == 0) load(s + PRE * waves, later);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        V8 v[NB];
        f32x4 c[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          v[b] = x_operand(s_x[q % DEPTH][b], k);
          c[b] = product<ACT>(v[b], minus, f32x4{0.f, 0.f, 0.f, 0.f});
        }
#pragma unroll
        for (int j = 0; j < T; ++j) {
          const V8 u = operand<ACT>(cur[j].code[q / 2][2 * (q % 2) + k], one);
          f32x4 now[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) now[b] = product<ACT>(v[b], u, c[b]);
          late.add(acc[(j + T - 1) % T]);
          late.set(now, scale_of(cur[j], 2 * q + k));
          interleave<NB>();
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(DEPTH == 2 || DEPTH == 4, "a slab's stages fill the ring a whole number of times");
#pragma unroll
  for (int e = 0; e < PRE; ++e) load(wave + e * waves, w[e]);
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) bring_stage(wave, i, i);
  for (int s = wave;; s += (PRE + 1) * waves) {
#pragma unroll
    for (int e = 0; e <= PRE; ++e) {
      step(s + e * waves, w[e], w[(e + PRE) % (PRE + 1)]);
      if (s + (e + 1) * waves >= A.slabs) goto out;
    }
  }
out:
  late.add(acc[T - 1]);
  wait_loads<0>();      // nothing is on its way to LDS any more
  __syncthreads();
  join_waves<ACT, NB, 4, T>(A, reinterpret_cast<float*>(s_mem), acc, tile0, 0, wave, waves);
}

// ---- more than 64 rows: fp16 operands --------------------------------------------------------------------------

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Rows of bf16 as fp16, each times a power of two that brings its largest to [2^14, 2^15), and that power's inverse.
__global__ __launch_bounds__(256) void k_linear_half(const bf16* __restrict__ x, int64_t stride, int d_in, f16* __restrict__ to,
                                                     float* __restrict__ factor) {
  __shared__ float s_top[4];
  const int tid = threadIdx.x, row = blockIdx.x;
  const bf16* from = x + (int64_t)row * stride;
  float top = 0.0f;
  for (int c = 8 * tid; c < d_in; c += 8 * 256) {
    const float m = max8<ACT_BF16>(*reinterpret_cast<const bf16x8*>(from + c));
    top = fmaxf(top, m);
  }
#pragma unroll
  for (int m = 1; m < WAVE; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
  if (tid % WAVE == 0) s_top[tid / WAVE] = top;
  __syncthreads();
  top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  float down;
  const float up = query_scale(top, down);
  for (int c = 8 * tid; c < d_in; c += 8 * 256)
    *reinterpret_cast<f16x8*>(to + (size_t)row * d_in + c) =
        query8<ACT_BF16>(*reinterpret_cast<const bf16x8*>(from + c), up);
  if (tid == 0) factor[row] = down;
}

// Eight columns of a row of W as fp16 operands: code times scale.
__device__ __forceinline__ f16x8 weights(unsigned word, f16 scale, unsigned one) {
  const f16x8 raw = operand<ACT_F16>(word, one);
  const f16x2 by = {scale, scale}, less = {(f16)24.0f, (f16)24.0f};
  f16x8 w;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const f16x2 y = (f16x2{raw[2 * e], raw[2 * e + 1]} - less) * by;   // the difference is exact
    w[2 * e] = y.x;
    w[2 * e + 1] = y.y;
  }
  return w;
}

// A 32x32x16 operand: row lane % 32, columns 8 (lane / 32) .. of the 16.  Operand m of group k of 32 rows in two tiles.
__device__ __forceinline__ f16x8 x_operand32(const XTile<f16x8>* x, int k, int m) {
  const int lane = threadIdx.x & (WAVE - 1);
  return x[(lane >> 4) & 1][lane & 15][(4 * k + 2 * m + (lane >> 5)) ^ (lane & 7)];
}
// Register e of a product is row 8 (e / 4) + 4 (lane / 32) + e % 4, column lane % 32.

// A workgroup takes 128 rows and 128 outputs, four waves of 64 x 64, over one of `splits` ranges of slabs.  x, codes and
// scales go to LDS without passing registers: x in stages of 64 columns, one and a half ahead of the one in use, codes
// three.  Two buffers and no more, so that three workgroups fit in a compute unit (two took 256 us where this takes 232).
template <int ACT>
__global__ __launch_bounds__(256, 3) void k_linear_tile(const LinearArgs A) {
  using E = typename ActT<ACT>::T;
  constexpr int WN = 2, MT = 2, NT = 2, kM = kTileM, kTiles = kTileTiles, kRows = 4;   // kRows: eights of rows a wave brings
  __shared__ __align__(16) char s_mem[2 * kM * kStage * 2 + 2 * kTiles * 1024 + 2 * kTiles * 256];
  XTile<f16x8>(*s_x)[kM / 16] = reinterpret_cast<XTile<f16x8>(*)[kM / 16]>(s_mem);
  u32x4(*s_code)[kTiles][WAVE] = reinterpret_cast<u32x4(*)[kTiles][WAVE]>(s_mem + 2 * kM * kStage * 2);
  u32x4(*s_scale)[kTiles][16] = reinterpret_cast<u32x4(*)[kTiles][16]>(s_mem + 2 * kM * kStage * 2 + 2 * kTiles * 1024);
  const int lane = threadIdx.x & (WAVE - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int wm = wave / WN, wn = wave % WN, c = lane & 31, part = lane >> 5;
  const int across = (A.tiles + kTiles - 1) / kTiles;
  const int tile0 = (int)(blockIdx.x % across) * kTiles, rest = (int)(blockIdx.x / across);
  const int split = rest % A.splits, row0 = rest / A.splits * kM;
  const int per = (A.slabs + A.splits - 1) / A.splits, first = split * per, end = min(first + per, A.slabs);
  const f16* x0 = static_cast<const f16*>(A.x) + (int64_t)row0 * A.x_stride;
  unsigned xrow[kRows];   // rows past the end are not stored
#pragma unroll
  for (int e = 0; e < kRows; ++e)
    xrow[e] = 2u * (unsigned)min(8 * (kRows * wave + e) + (lane >> 3), A.rows - 1 - row0) * (unsigned)A.x_stride;
  const size_t tile_bytes = (size_t)A.slabs * kSlabBytes;
  // this wave brings the codes of tiles 2 wave and 2 wave + 1
  const uint8_t* from[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) from[e] = A.packed + (size_t)min(tile0 + 2 * wave + e, A.tiles - 1) * tile_bytes;
  // past the end the last again, which nobody uses
  auto bring_x = [&](int stage, int slot) {
    const unsigned at = stage_byte(min(stage, 4 * end - 1) * kStage, A.d_in);
#pragma unroll
    for (int e = 0; e < kRows; ++e)
      bring(x0, xrow[e] + at, &s_x[slot][(kRows * wave + e) / 2][8 * ((kRows * wave + e) % 2)][0]);
  };
  auto bring_codes = [&](int piece, int slot) {   // of 128 columns
    const int p = min(piece, 2 * end - 1);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      bring(from[e] + (size_t)(p / 2) * kSlabBytes + 1024 * (p % 2), 16u * lane, &s_code[slot][2 * wave + e][0]);
  };
  const unsigned scale_at =   // four tiles a wave, and twice, so that every wave has asked for as many loads
      (unsigned)(min(tile0 + 4 * (wave & 1) + (lane >> 4), A.tiles - 1) - tile0) * (unsigned)tile_bytes + 2048u + 16u * (lane & 15);
  auto bring_scales = [&](int slab, int slot) {
    bring(A.packed + (size_t)tile0 * tile_bytes + (size_t)min(slab, end - 1) * kSlabBytes, scale_at,
          &s_scale[slot][4 * (wave & 1)][0]);
  };
  f32x16 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int b = 0; b < MT; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[j][b][e] = 0.0f;
  const unsigned one = sixteen<ACT_F16>();
  // operands 2 t + m: columns 16 m .. of a group of tile t
  u32x2 code[2][2 * NT];   // of the stage at hand and the next one: a word for each of its two groups
  f16x2 scale[2][NT];      // and scale
  f16x8 x[2][2 * MT];      // of the group at hand and the next one
  auto read_x = [&](int slot, int k, f16x8 (&to)[2 * MT]) {
#pragma unroll
    for (int b = 0; b < 2 * MT; ++b) to[b] = x_operand32(&s_x[slot][2 * MT * wm + 2 * (b / 2)], k, b % 2);
  };
  auto read_codes = [&](int slab, int q, u32x2 (&to)[2 * NT], f16x2 (&scales)[NT]) {
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const int tile = 2 * (NT * wn + j / 2) + (c >> 4);
      to[j] = *(reinterpret_cast<const u32x2*>(&s_code[q / 2][tile][16 * (2 * (j % 2) + part) + (c & 15)]) + q % 2);
      if (j % 2 == 0) scales[j / 2] = *(reinterpret_cast<const f16x2*>(&s_scale[slab & 1][tile][c & 15]) + q);
    }
  };
  auto group = [&](const f16x8 (&v)[2 * MT], const u32x2 (&codes)[2 * NT], const f16x2 (&scales)[NT], int k) {
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const f16x8 w = weights(codes[j][k], scales[j / 2][k], one);
#pragma unroll
      for (int b = 0; b < MT; ++b)
        acc[j / 2][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[2 * b + j % 2], w, acc[j / 2][b], 0, 0, 0);
#pragma unroll
      for (int b = 0; b < MT; ++b) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 16 / MT, 0);
      }
    }
  };
  // Wait until all but the last N loads are there, for every wave.  (Not __syncthreads(), which waits for all of them; the
  // operands read so far are there too.)
  auto meet = [&](auto n) {
    __builtin_amdgcn_sched_barrier(0);
    wait_loads<decltype(n)::value, 0>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  bring_x(4 * first, 0);
  bring_codes(2 * first, 0);
  bring_scales(first, first & 1);
  __builtin_amdgcn_sched_barrier(0);
  bring_x(4 * first + 1, 1);
  __builtin_amdgcn_sched_barrier(0);
  bring_codes(2 * first + 1, 1);
  meet(Count<kRows + 2>{});
  read_x(0, 0, x[0]);
  read_codes(first, 0, code[0], scale[0]);
  for (int slab = first; slab < end; ++slab) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int stage = 4 * slab + q;
      read_x(q % 2, 1, x[1]);
      group(x[0], code[q % 2], scale[q % 2], 0);
      // this stage has been read, and the next one is there, if not yet the codes that were asked for after it
      if (q == 0) meet(Count<2>{});
      else if (q == 2) meet(Count<3>{});
      else meet(Count<0>{});
      bring_x(stage + 2, q % 2);
      __builtin_amdgcn_sched_barrier(0);
      if (q % 2 == 1) bring_codes(2 * slab + (q + 3) / 2, ((q + 3) / 2) % 2);
      if (q == 1) bring_scales(slab + 1, (slab + 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
      read_x((q + 1) % 2, 0, x[0]);
      read_codes(slab + (q + 1) / 4, (q + 1) % 4, code[(q + 1) % 2], scale[(q + 1) % 2]);
      group(x[1], code[q % 2], scale[q % 2], 1);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  wait_loads<0>();   // nothing is on its way to LDS when the workgroup ends

  // ---- out: this wave's rows from r0 on ------------------------------------------------------------------
  const int r0 = row0 + 32 * MT * wm, left = A.rows - r0;
  const E* add0 = static_cast<const E*>(A.add) + (int64_t)r0 * A.add_stride;
  E* y0 = static_cast<E*>(A.y) + (int64_t)r0 * A.y_stride;
  float* part0 = A.partial + ((size_t)split * A.rows + r0) * A.d_out;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = (tile0 + 2 * (NT * wn + j)) * 16 + c, at = min(n, A.d_out - 1);
    const float factor = A.factor[at], bias = A.bias != nullptr ? A.bias[at] : 0.0f;
#pragma unroll
    for (int b = 0; b < MT; ++b)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int r = 32 * b + 8 * a + 4 * part;
        const E* add = add0 + (int64_t)r * A.add_stride + n;
        E* y = y0 + (int64_t)r * A.y_stride + n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (r + i >= left || n >= A.d_out) continue;
          const float sum = acc[j][b][4 * a + i];
          if (A.splits > 1) {
            part0[(size_t)(r + i) * A.d_out + n] = sum;
            continue;
          }
          float v = fmaf(sum, A.row_factor != nullptr ? factor * A.row_factor[r0 + r + i] : factor, bias);
          if (A.add != nullptr) v += (float)add[i * A.add_stride];
          y[i * A.y_stride] = (E)v;
        }
      }
  }
}

// The ranges' sums, in their order, and out.
template <int ACT>
__global__ __launch_bounds__(256) void k_linear_join(const LinearArgs A) {
  using E = typename ActT<ACT>::T;
  const int blocks = (A.d_out + 255) / 256, t = (int)(blockIdx.x / blocks), n = (int)(blockIdx.x % blocks) * 256 + threadIdx.x;
  if (n >= A.d_out) return;
  const size_t step = (size_t)A.rows * A.d_out;
  const float* from = A.partial + (size_t)t * A.d_out + n;
  float v[kMostSplits], sum = 0.0f;
#pragma unroll
  for (int s = 0; s < kMostSplits; ++s) v[s] = from[min(s, A.splits - 1) * step];
#pragma unroll
  for (int s = 0; s < kMostSplits; ++s) sum += s < A.splits ? v[s] : 0.0f;
  sum *= A.factor[n];
  if (A.row_factor != nullptr) sum *= A.row_factor[t];
  if (A.bias != nullptr) sum += A.bias[n];
  if (A.add != nullptr) sum += (float)static_cast<const E*>(A.add)[(int64_t)t * A.add_stride + n];
  static_cast<E*>(A.y)[(int64_t)t * A.y_stride + n] = (E)sum;
}

template <int ACT, int B>
hipError_t few_go(const LinearArgs& a, hipStream_t s) {
  const int most = a.tiles <= 512 ? kFewWaves : kFewWaves / 2, waves = a.slabs < most ? a.slabs : most;
  hipLaunchKernelGGL((k_linear_few<ACT, B>), dim3((unsigned)a.tiles), dim3(WAVE * waves), 0, s, a);
  return hipGetLastError();
}

template <int ACT, int NB, int T, int W, int DEPTH, int PRE>
hipError_t rows_go(const LinearArgs& a, hipStream_t s) {
  const int waves = a.slabs < W ? a.slabs : W;
  hipLaunchKernelGGL((k_linear_rows<ACT, NB, T, W, DEPTH, PRE>), dim3((unsigned)((a.tiles + T - 1) / T)), dim3(WAVE * waves), 0,
                     s, a);
  return hipGetLastError();
}

template <int ACT>
hipError_t linear_any(const LinearArgs& a, hipStream_t s) {
  if (a.rows == 1) return few_go<ACT, 1>(a, s);
  if (a.rows <= kFewRows) return few_go<ACT, kFewRows>(a, s);
  if (a.rows <= 16) return rows_go<ACT, 1, 2, 8, 4, 2>(a, s);
  if (a.rows <= 32) return rows_go<ACT, 2, 2, 8, 2, 1>(a, s);
  if (a.rows <= kExactRows) {
    // the registers and LDS of eight waves fill a compute unit: 256 workgroups of eight waves, or 512 of four, are at work
    // at once.  64 rows, us by two tiles and eight waves, two and four, three and four: 8192 columns, 512 tiles 24.0, 25.0,
    // 30.0; 640 tiles 41.2, 37.8, 30.6; 768 tiles 41.8, 38.4, 32.2; 1024 tiles 46, 42.0, 49.2; 1792 tiles 85, 74.8, 75.0;
    // 7168 columns, 1280 tiles 57.5, 51.6, 46.2; 1344 tiles 57.9, 51.8, 46.4; 1536 tiles 61, 55.0, 49.2.  (Up to 768 tiles
    // three would be a workgroup for each compute unit.)
    if (a.tiles <= 512) return rows_go<ACT, 4, 2, 8, 2, 1>(a, s);
    return a.tiles <= 1024 ? rows_go<ACT, 4, 2, 4, 2, 1>(a, s) : rows_go<ACT, 4, 3, 4, 2, 1>(a, s);
  }
  LinearArgs b = a;
  const LinearScratch layout = linear_scratch(ACT, a.rows, a.d_in, a.d_out, a.scratch_bytes);
  char* scratch = static_cast<char*>(a.scratch);
  b.splits = layout.splits;
  b.partial = reinterpret_cast<float*>(scratch + layout.partial);
  if constexpr (ACT == ACT_BF16) {
    f16* x = reinterpret_cast<f16*>(scratch + layout.x);
    float* factor = reinterpret_cast<float*>(scratch + layout.factor);
    hipLaunchKernelGGL(k_linear_half, dim3((unsigned)a.rows), dim3(256), 0, s, static_cast<const bf16*>(a.x), a.x_stride, a.d_in,
                       x, factor);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    b.x = x;
    b.x_stride = a.d_in;
    b.row_factor = factor;
  }
  const long long grid = (long long)((a.tiles + kTileTiles - 1) / kTileTiles) * b.splits * ((a.rows + kTileM - 1) / kTileM);
  const long long join = (long long)((a.d_out + 255) / 256) * a.rows;
  if (grid > 0x7fffffff || (b.splits > 1 && join > 0x7fffffff)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_linear_tile<ACT>), dim3((unsigned)grid), dim3(256), 0, s, b);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || b.splits == 1) return e;
  hipLaunchKernelGGL((k_linear_join<ACT>), dim3((unsigned)join), dim3(256), 0, s, b);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_pack(const void* w, const void* scales, void* packed, float* factor, int d_in, int d_out,
                              hipStream_t s) {
  const int slabs = (d_in + kSlabCols - 1) / kSlabCols, tiles = (d_out + kSlabRows - 1) / kSlabRows;
  const long long count = (long long)tiles * slabs, grid = (count + 3) / 4;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  const auto* codes = static_cast<const uint8_t*>(w);
  const auto* halves = static_cast<const unsigned short*>(scales);
  auto* to = static_cast<uint8_t*>(packed);
  hipLaunchKernelGGL(k_linear_factor, dim3((unsigned)(tiles * kSlabRows + 3) / 4), dim3(256), 0, s, halves, factor, d_in / 32,
                     d_out, tiles * kSlabRows);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_linear_pack, dim3((unsigned)grid), dim3(256), 0, s, codes, halves, to, factor, d_in, d_out, slabs,
                     count);
  return hipGetLastError();
}

hipError_t launch_linear(int act, const LinearArgs& a, hipStream_t s) {
  return act == ACT_F16 ? linear_any<ACT_F16>(a, s) : linear_any<ACT_BF16>(a, s);
}

}  // namespace pik
