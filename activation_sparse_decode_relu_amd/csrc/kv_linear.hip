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
// 16 bytes a lane from base + at to LDS, lane after lane.
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
// At most N of this wave's loads are still on their way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0f70);
  asm volatile("" ::: "memory");
}

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

// Bound by the vector ALU (an fp32 multiply-add for each output and group, as long as the product itself) and the matrix
// instructions.  A workgroup takes 128 rows and 128 outputs, four waves of 64 x 64.  x, codes and scales go to LDS
// without passing registers: x in stages of 64 columns, two ahead of the one in use, codes two stages ahead too.
constexpr int kTileM = 128, kTileN = 128;
template <int ACT>
__global__ __launch_bounds__(256, 2) void k_linear_tile(const LinearArgs A) {
  using E = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  constexpr int kTiles = kTileN / 16, kRing = 3;
  __shared__ __align__(16) char s_mem[kRing * kTileM * kStage * 2 + 2 * kTiles * 1024 + 2 * 4 * 1024];
  XTile<V8>(*s_x)[kTileM / 16] = reinterpret_cast<XTile<V8>(*)[kTileM / 16]>(s_mem);
  u32x4(*s_code)[kTiles][WAVE] = reinterpret_cast<u32x4(*)[kTiles][WAVE]>(s_mem + kRing * kTileM * kStage * 2);
  u32x4(*s_scale)[4][WAVE] = reinterpret_cast<u32x4(*)[4][WAVE]>(s_mem + kRing * kTileM * kStage * 2 + 2 * kTiles * 1024);
  const int lane = threadIdx.x & (WAVE - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int g = lane >> 4, wm = wave >> 1, wn = wave & 1;
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
  auto bring_scales = [&](int slab, int slot) {   // rows lane % 16 of the two tiles, twice
    const uint8_t* p = from[0] + (size_t)min(slab, A.slabs - 1) * kSlabBytes + 2048;
    bring(p, 16u * (lane & 15) + (lane & 16 ? (unsigned)(from[1] - from[0]) : 0u), &s_scale[slot][wave][0]);
  };
  float acc[4][4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][b][i] = 0.0f;
  const V8 minus = minus24<ACT>();
  const unsigned one = sixteen<ACT>();
  Late<4> late;
  u32x4 code[4], scale[4];
  bring_x(0, 0);
  bring_codes(0, 0);
  bring_scales(0, 0);
  bring_x(1, 1);
  int slot = 0;   // stage % kRing
  for (int slab = 0; slab < A.slabs; ++slab) {
#pragma unroll
    for (int q = 0; q < kSlabCols / kStage; ++q) {
      const int stage = slab * (kSlabCols / kStage) + q;
      // what was asked for two stages ago is there; behind it is what the last stage asked for
      if (q == 1) wait_loads<6>();
      else if (q == 3) wait_loads<7>();
      else wait_loads<4>();
      // (not __syncthreads(), which waits for all that is on its way; every operand read so far has been used)
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      const int ahead = slot >= 1 ? slot - 1 : kRing - 1;
      bring_x(stage + 2, ahead);
      if (q % 2 == 0) bring_codes(2 * slab + q / 2 + 1, (q / 2 + 1) % 2);
      if (q == 2) bring_scales(slab + 1, (slab + 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
      if (q == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) scale[j] = s_scale[slab & 1][2 * wn + j / 2][16 * (j % 2) + (lane & 15)];
      }
      if (q % 2 == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) code[j] = s_code[q / 2][4 * wn + j][lane];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        V8 v[4];
        f32x4 c[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          v[b] = x_operand(s_x[slot][4 * wm + b], k);
          c[b] = product<ACT>(v[b], minus, f32x4{0.f, 0.f, 0.f, 0.f});
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const V8 w = operand<ACT>(code[j][2 * (q % 2) + k], one);
          const int group = 2 * q + k;
          f32x4 now[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) now[b] = product<ACT>(v[b], w, c[b]);
          late.add(acc[(j + 3) % 4]);
          late.set(now, (float)as_h2(scale[j][group / 2])[group % 2]);
          interleave<4>();
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      slot = slot == kRing - 1 ? 0 : slot + 1;
    }
  }
  late.add(acc[3]);
  wait_loads<0>();   // nothing is on its way to LDS when the workgroup ends
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = (tile0 + 4 * wn + j) * 16 + (lane & 15);
    if (n >= A.d_out) continue;
    const float bias = A.bias != nullptr ? A.bias[n] : 0.0f;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = row0 + 64 * wm + 16 * b + 4 * g + i;
        if (t >= A.rows) continue;
        float y = acc[j][b][i] + bias;
        if (A.add != nullptr) y += (float)static_cast<const E*>(A.add)[(int64_t)t * A.add_stride + n];
        static_cast<E*>(A.y)[(int64_t)t * A.y_stride + n] = (E)y;
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
