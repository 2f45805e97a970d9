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
  for (int j = 0; j < 4; ++j) r[j] = (__builtin_amdgcn_alignbit(w, w, 4 * j) & Code<ACT>::kMask) | one;
  return __builtin_bit_cast(typename ActT<ACT>::V8, r);
}

// ---- laying out ----------------------------------------------------------------------------------------

// One wave a row of scales: the power of two that brings the largest to [8, 16).  So products of codes and scales stay in
// fp16's normal range whatever the row's size is.
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
  if (lane == 0) factor[row] = top > 0.0f && top <= 65504.0f ? pow2i(x - 3) : 1.0f;
}

// One wave a slab.
template <int ACT>
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
    if (srow < d_out && group < d_in / 32) {
      const float scale = (float)__builtin_bit_cast(f16, scales[(size_t)srow * (d_in / 32) + group]);
      s |= (unsigned)__builtin_bit_cast(unsigned short, (f16)(scale / factor[srow])) << (16 * e);
    }
  }
  *reinterpret_cast<unsigned*>(to + 2048 + lane * 4) = s;
}

// ---- one to 64 rows ------------------------------------------------------------------------------------

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

// ---- more than 64 rows ---------------------------------------------------------------------------------

// Bound by issue: on this hardware a wave's vector ALU instruction runs beside a matrix instruction only in part (a
// 16x16x32 one and n others take 15.6 + 3.7 n cycles together, a 32x32x16 one, twice the work, 19 + 3.9 n).  With an fp32
// multiply-add for each output and group, as many cycles as the product itself, 2000 rows 4096 -> 12288 took 328 us.  So
// with fp16 activations code times scale is an fp16 operand, rounded to half a step of 2^-11 (as much as y itself), and the
// sums stay in the matrix instructions.  There is no packed arithmetic in bf16, whose operands stay whole numbers.
// A workgroup takes 128 rows and 128 outputs, four waves of 64 x 64.  x, codes and scales go to LDS
// without passing registers: x in stages of 64 columns, one and a half ahead of the one in use, codes three.  Two buffers
// and no more, so that three workgroups fit in a compute unit.
constexpr int kTileM = 128, kTileN = 128;
template <int ACT>
__global__ __launch_bounds__(256, 2) void k_linear_tile(const LinearArgs A) {
  using E = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  constexpr int kTiles = kTileN / 16, kRing = 2;
  __shared__ __align__(16) char s_mem[kRing * kTileM * kStage * 2 + 2 * kTiles * 1024 + 2 * kTiles * 256];
  XTile<V8>(*s_x)[kTileM / 16] = reinterpret_cast<XTile<V8>(*)[kTileM / 16]>(s_mem);
  u32x4(*s_code)[kTiles][WAVE] = reinterpret_cast<u32x4(*)[kTiles][WAVE]>(s_mem + kRing * kTileM * kStage * 2);
  u32x4(*s_scale)[kTiles][16] = reinterpret_cast<u32x4(*)[kTiles][16]>(s_mem + kRing * kTileM * kStage * 2 + 2 * kTiles * 1024);
  const int lane = threadIdx.x & (WAVE - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int wm = wave >> 1, wn = wave & 1;
  const int across = (A.tiles + kTiles - 1) / kTiles;
  const int row0 = (int)(blockIdx.x / across) * kTileM, tile0 = (int)(blockIdx.x % across) * kTiles;
  const E* x0 = static_cast<const E*>(A.x) + (int64_t)row0 * A.x_stride;
  unsigned xrow[4];   // this wave brings rows 32 wave .. of a stage; rows past the end are not stored
#pragma unroll
  for (int e = 0; e < 4; ++e)
    xrow[e] = 2u * (unsigned)min(32 * wave + 8 * e + (lane >> 3), A.rows - 1 - row0) * (unsigned)A.x_stride;
  const size_t tile_bytes = (size_t)A.slabs * kSlabBytes;
  // and the codes of tiles 2 wave and 2 wave + 1
  const uint8_t* from[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) from[e] = A.packed + (size_t)min(tile0 + 2 * wave + e, A.tiles - 1) * tile_bytes;
  const int stages = A.slabs * (kSlabCols / kStage);
  // past the end the last again, which nobody uses
  auto bring_x = [&](int stage, int slot) {
    const unsigned at = stage_byte(min(stage, stages - 1) * kStage, A.d_in);
#pragma unroll
    for (int e = 0; e < 4; ++e) bring(x0, xrow[e] + at, &s_x[slot][2 * wave + e / 2][8 * (e % 2)][0]);
  };
  auto bring_codes = [&](int piece, int slot) {   // of 128 columns
    const int p = min(piece, 2 * A.slabs - 1);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      bring(from[e] + (size_t)(p / 2) * kSlabBytes + 1024 * (p % 2), 16u * lane, &s_code[slot][2 * wave + e][0]);
  };
  const unsigned scale_at =   // four tiles a wave, and twice, so that every wave has asked for as many loads
      (unsigned)(min(tile0 + 4 * (wave & 1) + (lane >> 4), A.tiles - 1) - tile0) * (unsigned)tile_bytes + 2048u + 16u * (lane & 15);
  auto bring_scales = [&](int slab, int slot) {
    bring(A.packed + (size_t)tile0 * tile_bytes + (size_t)min(slab, A.slabs - 1) * kSlabBytes, scale_at,
          &s_scale[slot][4 * (wave & 1)][0]);
  };
  // kFold: 2 x 2 tiles of 32 x 32, operands 2 t + m for columns 16 m .. of a group of tile t; else 4 x 4 of 16 x 16
  constexpr bool kFold = ACT == ACT_F16;
  const int c = kFold ? lane & 31 : lane & 15, part = kFold ? lane >> 5 : lane >> 4;   // this lane's row of x or W, and columns
  typedef float f32x16 __attribute__((ext_vector_type(16)));
  f32x16 sum[2][2];
  float acc[4][4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[j][b][i] = 0.0f;
        sum[j / 2][b / 2][8 * (j % 2) + 4 * (b % 2) + i] = 0.0f;
      }
  const V8 minus = minus24<ACT>();
  const unsigned one = sixteen<ACT>();
  Late<4> late;
  u32x2 code[2][4];      // of the stage at hand and the next one: a word for each of its two groups
  f16x2 scale[2][4];     // and scale
  V8 v[2][4];            // of the group at hand and the next one
  auto read_x = [&](int slot, int k, V8 (&to)[4]) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int tile = kFold ? 4 * wm + 2 * (b / 2) + (c >> 4) : 4 * wm + b, chunk = kFold ? 2 * (b % 2) + part : part;
      to[b] = s_x[slot][tile][c & 15][(4 * k + chunk) ^ (c & 7)];
    }
  };
  auto read_codes = [&](int slab, int q, u32x2 (&to)[4], f16x2 (&scales)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int tile = kFold ? 4 * wn + 2 * (j / 2) + (c >> 4) : 4 * wn + j, chunk = kFold ? 2 * (j % 2) + part : part;
      to[j] = *(reinterpret_cast<const u32x2*>(&s_code[q / 2][tile][16 * chunk + (c & 15)]) + q % 2);
      if (!kFold || j % 2 == 0)
        scales[j] = *(reinterpret_cast<const f16x2*>(&s_scale[slab & 1][tile][c & 15]) + q);
    }
  };
  auto group = [&](const V8 (&x)[4], const u32x2 (&code)[4], const f16x2 (&scale)[4], int k) {
    if constexpr (kFold) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f16x2 by = {scale[j & ~1][k], scale[j & ~1][k]}, less = {(f16)24.0f, (f16)24.0f};
        const V8 raw = operand<ACT>(code[j][k], one);
        V8 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f16x2 y = (f16x2{raw[2 * e], raw[2 * e + 1]} - less) * by;   // the difference is exact
          w[2 * e] = y.x;
          w[2 * e + 1] = y.y;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) sum[j / 2][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[2 * b + j % 2], w, sum[j / 2][b], 0, 0, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
      }
    } else {
      f32x4 c[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) c[b] = product<ACT>(x[b], minus, f32x4{0.f, 0.f, 0.f, 0.f});
      late.add(acc[3]);
      interleave<4>();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const V8 w = operand<ACT>(code[j][k], one);
        f32x4 now[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) now[b] = product<ACT>(x[b], w, c[b]);
        if (j > 0) late.add(acc[j - 1]);
        late.set(now, (float)scale[j][k]);
        interleave<4>();
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
  bring_x(0, 0);
  bring_codes(0, 0);
  bring_scales(0, 0);
  __builtin_amdgcn_sched_barrier(0);
  bring_x(1, 1);
  __builtin_amdgcn_sched_barrier(0);
  bring_codes(1, 1);
  meet(Count<6>{});
  read_x(0, 0, v[0]);
  read_codes(0, 0, code[0], scale[0]);
  for (int slab = 0; slab < A.slabs; ++slab) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int stage = 4 * slab + q;
      read_x(q % 2, 1, v[1]);
      group(v[0], code[q % 2], scale[q % 2], 0);
      // this stage has been read, and the next one is there, if not yet the codes that were asked for after it
      if (q == 0) meet(Count<2>{});
      else if (q == 2) meet(Count<3>{});
      else meet(Count<0>{});
      bring_x(stage + 2, q % 2);
      __builtin_amdgcn_sched_barrier(0);
      if (q % 2 == 1) bring_codes(2 * slab + (q + 3) / 2, ((q + 3) / 2) % 2);
      if (q == 1) bring_scales(slab + 1, (slab + 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
      read_x((q + 1) % 2, 0, v[0]);
      read_codes(slab + (q + 1) / 4, (q + 1) % 4, code[(q + 1) % 2], scale[(q + 1) % 2]);
      group(v[1], code[q % 2], scale[q % 2], 1);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (!kFold) late.add(acc[3]);
  wait_loads<0>();   // nothing is on its way to LDS when the workgroup ends
  // Four rows of an output: rows r .. r + 3 of this wave's 64.
  const int left = A.rows - row0 - 64 * wm;
  const E* add0 = static_cast<const E*>(A.add) + (int64_t)(row0 + 64 * wm) * A.add_stride;
  E* y0 = static_cast<E*>(A.y) + (int64_t)(row0 + 64 * wm) * A.y_stride;
  auto store4 = [&](int r, int n, float factor, float bias, const float (&sums)[4]) {
    const E* add = add0 + (int64_t)r * A.add_stride + n;
    E* y = y0 + (int64_t)r * A.y_stride + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (r + i >= left || n >= A.d_out) continue;
      float v = fmaf(sums[i], factor, bias);
      if (A.add != nullptr) v += (float)add[i * A.add_stride];
      y[i * A.y_stride] = (E)v;
    }
  };
  constexpr int kWide = kFold ? 32 : 16, kEach = 64 / kWide;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int n = (tile0 + 4 * wn) * 16 + j * kWide + c, at = min(n, A.d_out - 1);
    const float factor = A.factor[at], bias = A.bias != nullptr ? A.bias[at] : 0.0f;
#pragma unroll
    for (int b = 0; b < kEach; ++b) {
      if constexpr (kFold) {
#pragma unroll
        for (int a = 0; a < 4; ++a)
          store4(32 * b + 8 * a + 4 * part, n, factor, bias,
                 {sum[j][b][4 * a], sum[j][b][4 * a + 1], sum[j][b][4 * a + 2], sum[j][b][4 * a + 3]});
      } else {
        store4(16 * b + 4 * part, n, factor, bias, {acc[j][b][0], acc[j][b][1], acc[j][b][2], acc[j][b][3]});
      }
    }
  }
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
  if (a.rows <= 64) return rows_go<ACT, 4, 3, 4, 2, 1>(a, s);
  const long long grid = (long long)((a.tiles + kTileN / 16 - 1) / (kTileN / 16)) * ((a.rows + kTileM - 1) / kTileM);
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_linear_tile<ACT>), dim3((unsigned)grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_pack(int act, const void* w, const void* scales, void* packed, float* factor, int d_in, int d_out,
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
  if (act == ACT_F16)
    hipLaunchKernelGGL((k_linear_pack<ACT_F16>), dim3((unsigned)grid), dim3(256), 0, s, codes, halves, to, factor, d_in, d_out,
                       slabs, count);
  else
    hipLaunchKernelGGL((k_linear_pack<ACT_BF16>), dim3((unsigned)grid), dim3(256), 0, s, codes, halves, to, factor, d_in, d_out,
                       slabs, count);
  return hipGetLastError();
}

hipError_t launch_linear(int act, const LinearArgs& a, hipStream_t s) {
  return act == ACT_F16 ? linear_any<ACT_F16>(a, s) : linear_any<ACT_BF16>(a, s);
}

}  // namespace pik
