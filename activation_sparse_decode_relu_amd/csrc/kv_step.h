// Attention of few rows: single tokens and a handful (up to 64 rows of a cached head), over long caches.
//
// Bound by reading the codes.  An item is a sequence and cached head with its blocks of 32 tokens; items are cut
// into pieces of up to S blocks, one workgroup each, so that the card is filled once: S is the smallest of five sizes
// from (blocks of the call) / step_shares to twice that which gives no more than step_pieces.  Every workgroup
// works this out by itself from the lengths (they are on the device).  Starting a piece costs as much as some 8
// blocks (its lengths, pages and codes are loads that wait for each other), so whole items are better than equal
// stretches of the call's blocks: 64 sequences of 1000 tokens, 8 heads, took 36.4 us with equal stretches and
// take 27.1.
//
// The four waves of a workgroup take the blocks of a piece in turn, each with its own online softmax,
// straight from memory to the matrix instructions' operands: a block's bytes are stored in their order, so
// each load is one contiguous KB and nothing passes through LDS.  One 16x16x32 tile holds up to 16 rows:
// all query heads of a cached head, for all its new tokens.
//
// An item of one piece is finished by its workgroup; otherwise each workgroup leaves its state (fp32) in the
// workspace and the last of them, by a ticket, joins the parts in their order, so the result does not depend
// on who was last.
//
// Measured: long caches stream at 6.1 TB/s (64 x 4000 tokens, 526 MB in 86.6 us) and some 9 us go to the start
// and the end, in which nothing streams.
#pragma once

#include "kv_items.h"

namespace pik {

namespace {

// What one sequence brings to the call, as a lane holds it.
struct StepSeq {
  int seq, len, row0, rows;   // rows: those computed, at most max_new
  int p0;                     // position of its first row
  int blocks;                 // visible blocks, at least 1 where there are rows
  int shared;                 // ATTEND_OWN: tokens that others have attended over
};

template <int MODE>
__device__ __forceinline__ StepSeq step_seq(const AttendArgs<MODE>& A, int i) {
  StepSeq r{-1, 0, 0, 0, 0, 0, 0};
  if (i >= items_of<MODE>(A)) return r;
  const KvSeq s = item_seq<MODE>(A, i);
  r.seq = s.seq;
  r.len = s.len;
  r.row0 = s.row0;
  r.rows = min(s.rows, A.max_new);
  r.p0 = item_first<MODE>(s);
  if constexpr (MODE == ATTEND_OWN) r.shared = shared_of(A, A.n_groups + i);
  if (r.rows > 0) r.blocks = max(item_span<MODE>(A, s.len, r.shared, r.p0, r.p0 + r.rows - 1).count(), 1);
  return r;
}

__device__ __forceinline__ int lane_of(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Inclusive sums over the wave's lanes, and all of them (both of the vector ALU alone).
__device__ __forceinline__ int wave_inclusive(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8: within 16 lanes
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast 15: rows 1 and 3 take the row before
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast 31: the upper half takes the lower
  return v;
}
__device__ __forceinline__ int wave_total(int v) { return lane_of(wave_inclusive(v), WAVE - 1); }

// Into how many pieces of about S blocks an item of `blocks` falls.
__device__ __forceinline__ int pieces_of(int blocks, int S) { return (int)((unsigned)(blocks + S - 1) / (unsigned)S); }

// The codes of one block of K or V, as a wave loads them: 16 bytes a lane in each of D / 32 pieces.  A block
// that is not there has 0 bytes: its loads read nothing and return 0, with no branch around them.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t codes_rsrc(const uint8_t* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, bytes, 0x00020000);
}
constexpr int kKvStream = 2;   // buffer cache policy nt: codes are read once
__device__ __forceinline__ u32x4 codes_piece(__amdgpu_buffer_rsrc_t r, int piece) {
  const int lane = threadIdx.x & (WAVE - 1);
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, 16 * lane + 1024 * piece, 0, kKvStream));
}

// Where the parts of a sequence and head lie that is spread over several workgroups, and what is joined there.
// More than kFan parts are joined in two levels, by groups of about the square root of their number: one workgroup
// joining 64 parts of 64 rows took 60 of 101 us.
constexpr int kFan = 8;
__device__ __forceinline__ int fan_of(int parts) { return parts <= kFan ? parts : (int)ceilf(sqrtf((float)parts)); }

// The joined state of `n` parts (slots from, from + step, ... of the workspace) of R rows; sink(r, d, v, state)
// gets four dims of a row's O' and its state.
template <int D, int kRows, int kWaves, class Sink>
__device__ __forceinline__ void join_parts(__amdgpu_buffer_rsrc_t prs, float* lds, int from, int step, int n, int R,
                                           Sink&& sink) {
  constexpr int kRow = D + 4;
  f32x4* state = reinterpret_cast<f32x4*>(lds);          // [n + 1][kRows]: the last is the joined one
  auto word = [&](int i, int r) { return ((from + i * step) * kRows + r) * kRow; };
  // every load of a batch of parts is on its way before the first is used, the first batch before the states
  constexpr int kThreads = WAVE * kWaves, kMine = kRows * (D / 4) / kThreads, kBatch = (kRows == 64 ? 32 : 16) / kMine;
  f32x4 y[kMine][kBatch], v[kMine];
  auto batch = [&](int i0) {
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int k = q * kThreads + threadIdx.x, r = min(k / (D / 4), R - 1), d = 4 * (k % (D / 4));
#pragma unroll
      for (int e = 0; e < kBatch; ++e) y[q][e] = get4(prs, word(min(i0 + e, n - 1), r) + d);
    }
  };
  batch(0);
  for (int k = threadIdx.x; k < n * kRows; k += kThreads) {
    const int i = k / kRows, r = k % kRows;
    if (r < R) state[k] = get4(prs, word(i, r) + D);
  }
  __syncthreads();
  if ((int)threadIdx.x < R) {
    const int r = threadIdx.x;
    RowState a{-INFINITY, -INFINITY, 0.0f};
    for (int i = 0; i < n; ++i) {
      a.rr = fmaxf(a.rr, state[i * kRows + r].x);
      a.mm = fmaxf(a.mm, state[i * kRows + r].y);
    }
    for (int i = 0; i < n; ++i) {
      const f32x4 b = state[i * kRows + r];
      a.l += b.z * ex2_diff(b.y, a.mm);
      state[i * kRows + r].x = ex2_diff(b.x, a.rr);
    }
    state[n * kRows + r] = f32x4{a.rr, a.mm, a.l, 0.f};
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kMine; ++q) v[q] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    if (i0 > 0) batch(i0);
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int r = min((int)(q * kThreads + threadIdx.x) / (D / 4), R - 1);
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        if (i0 + e < n) v[q] += y[q][e] * state[(i0 + e) * kRows + r].x;
    }
  }
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    const int k = q * kThreads + threadIdx.x, r = k / (D / 4), d = 4 * (k % (D / 4));
    if (r >= R) continue;
    const f32x4 s = state[n * kRows + r];
    sink(r, d, v[q], RowState{s.x, s.y, s.z});
  }
}

// Counts this workgroup in; true in the last of `n`, which also clears the ticket.  The workgroup's partial
// stores are complete in every wave before the ticket is drawn.
__device__ __forceinline__ bool last_of(unsigned* ticket, int n, int* s_last) {
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last =
        __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(n - 1);
    if (last) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_last = last;
  }
  __syncthreads();
  return *s_last != 0;
}

template <int MODE, int ACT, int CODE, int D, int NT>
__global__ __launch_bounds__(WAVE* step_waves(NT, D), step_groups(NT, D) * step_waves(NT, D) / 1024) void k_kv_step(
    const AttendArgs<MODE> A) {
  using T = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  constexpr int kWaves = step_waves(NT, D), kRows = 16 * NT, kRow = D + 4;   // rows of a tile; floats of a row's part
  __shared__ float s_part[kWaves][kRows][kRow];       // O', then rr, mm, l
  __shared__ int s_last;
  const KvView& c = A.c;
  const int items = items_of<MODE>(A);
  const int lane = threadIdx.x & (WAVE - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int g = lane >> 4, col = lane & 15;
  const __amdgpu_buffer_rsrc_t prs = partial_rsrc(A.partial);

  // ---- the pieces: see the top of the file --------------------------------------------------------
  constexpr int G = step_shares(NT, D), kTries = 5;
  StepSeq mine = step_seq<MODE>(A, lane);
  int sum = mine.blocks;
  for (int base = WAVE; base < items; base += WAVE) sum += step_seq<MODE>(A, base + lane).blocks;
  const int total = wave_total(sum) * c.kv_heads;
  int S = 0;
  {
    int tries[kTries], got[kTries];
#pragma unroll
    for (int e = 0; e < kTries; ++e) {
      tries[e] = max((int)(((long long)total * (4 + e) + 4 * G - 1) / (4 * G)), MODE == ATTEND_OWN ? kOwnGrain : kStepGrain);
      got[e] = pieces_of(mine.blocks, tries[e]);
    }
    for (int base = WAVE; base < items; base += WAVE) {
      const int blocks = step_seq<MODE>(A, base + lane).blocks;
#pragma unroll
      for (int e = 0; e < kTries; ++e) got[e] += pieces_of(blocks, tries[e]);
    }
    const int most = step_pieces(NT, D, items * c.kv_heads);
#pragma unroll
    for (int e = kTries - 1; e >= 0; --e)
      if (e == kTries - 1 || wave_total(got[e]) * c.kv_heads <= most) S = tries[e];
  }
  int base = 0, before = 0, slots = 0;                // the 64 sequences in `mine`, the pieces and slots before them
  int pieces = pieces_of(mine.blocks, S);
  int incl = wave_inclusive(pieces) * c.kv_heads;
  int incl_slots = wave_inclusive(pieces > 1 ? pieces : 0) * c.kv_heads;

  for (int w = blockIdx.x;; w += gridDim.x) {
    while (before + lane_of(incl, WAVE - 1) <= w) {
      before += lane_of(incl, WAVE - 1);
      slots += lane_of(incl_slots, WAVE - 1);
      base += WAVE;
      if (base >= items) return;
      mine = step_seq<MODE>(A, base + lane);
      pieces = pieces_of(mine.blocks, S);
      incl = wave_inclusive(pieces) * c.kv_heads;
      incl_slots = wave_inclusive(pieces > 1 ? pieces : 0) * c.kv_heads;
    }
    const int at = __builtin_ctzll(__ballot(before + incl > w));   // lane of the piece's sequence
    const int seq = lane_of(mine.seq, at), len = lane_of(mine.len, at), row0 = lane_of(mine.row0, at);
    const int nrows = lane_of(mine.rows, at), p0 = lane_of(mine.p0, at), blocks = lane_of(mine.blocks, at);
    const int parts = lane_of(pieces, at), local = w - (before + lane_of(incl, at) - parts * c.kv_heads);
    const int head = local / parts, part = local - head * parts;
    const int first = slots + lane_of(incl_slots, at) - (c.kv_heads - head) * parts;   // slot of part 0, if parts > 1
    const int per = (blocks + parts - 1) / parts, b0 = part * per, b1 = min(b0 + per, blocks);
    const int p1 = p0 + nrows - 1, R = nrows * A.group;
    const int shared = MODE == ATTEND_OWN ? lane_of(mine.shared, at) : 0;
    Span span = item_span<MODE>(A, len, shared, p0, p1);
    if (seq < 0) span = Span{0, 0, 0};
    const int inv_group = (65536 + A.group - 1) / A.group;   // r / group for r < 128: r * inv_group >> 16

    // ---- the rows: row 16 t + col of the tile, dims (4 (s / 2) + g) 16 + 8 (s % 2) .. + 8 in step s ----
    f16x8 q[NT][D / 32];
    float row_mul[NT];
    int pos[NT];
    RowRun st[NT];
    f32x4 o[NT][D / 16];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 16 * t + col;
      const int j = (r * inv_group) >> 16, hh = r - j * A.group;
      const bool live = r < R;
      pos[t] = live ? p0 + j : -1;
      const T* src = static_cast<const T*>(A.q.data) + (int64_t)(row0 + (live ? j : 0)) * A.q.token +
                     (int64_t)(head * A.group + (live ? hh : 0)) * A.q.head;
      V8 x[D / 32];
#pragma unroll
      for (int s = 0; s < D / 32; ++s) {
        x[s] = V8{};
        if (live) x[s] = *reinterpret_cast<const V8*>(src + (4 * (s / 2) + g) * 16 + 8 * (s % 2));
      }
      float up = 1.0f, down = 1.0f;
      if constexpr (ACT == ACT_BF16) {
        float m = 0.0f;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) m = fmaxf(m, max8<ACT>(x[s]));
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        up = query_scale(m, down);
      }
#pragma unroll
      for (int s = 0; s < D / 32; ++s) q[t][s] = query8<ACT>(x[s], up);
      row_mul[t] = A.scale * kLog2e * down;
      st[t] = row_run();
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // ---- this wave's blocks: b0 + wave, + kWaves, ... ------------------------------------------------
    const int count = b1 - b0 > wave ? (b1 - b0 - wave + kWaves - 1) / kWaves : 0;
    for (int k0 = 0; k0 < count; k0 += WAVE) {
      // where 64 of them lie: lane k holds block k0 + k
      const int m = min(count - k0, WAVE), bi = b0 + wave + (k0 + lane) * kWaves;
      const int blk = span.block(min(bi, max(span.count() - 1, 0)));
      const int slot = blk % c.page_blocks, there = kv_page(c, max(seq, 0), blk);
      const int page = lane < m && bi < span.count() ? there : -1;
      const size_t eat = block_at(c, max(page, 0), head, slot);
      const int exps = (int)c.k_exp[eat] | (int)c.v_exp[eat] << 8;
      // the block after this one is on its way while this one is computed: a piece's registers are loaded
      // again as soon as its codes are decoded
      u32x4 kc[D / 32], vc[D / 32];
      auto rsrc = [&](const uint8_t* base, int k) {
        const int pg = lane_of(page, k & (WAVE - 1));
        const size_t e = block_at(c, max(pg, 0), head, lane_of(slot, k & (WAVE - 1))) * (kKvBlock * D);
        return codes_rsrc(base + e, k < m && pg >= 0 ? kKvBlock * D : 0);
      };
      {
        const __amdgpu_buffer_rsrc_t rk = rsrc(c.k, 0), rv = rsrc(c.v, 0);
#pragma unroll
        for (int p = 0; p < D / 32; ++p) kc[p] = codes_piece(rk, p);
#pragma unroll
        for (int p = 0; p < D / 32; ++p) vc[p] = codes_piece(rv, p);
      }
      for (int k = 0; k < m; ++k) {
        const int t0 = lane_of(blk, k) * kKvBlock;
        const bool held = lane_of(page, k) >= 0;
        const __amdgpu_buffer_rsrc_t rk = rsrc(c.k, k + 1), rv = rsrc(c.v, k + 1);
        const int ex = lane_of(exps, k);
        const int ek = max((ex & 255) - 127, -126), ev = max((ex >> 8) - 127, -126);
        const float evf = (float)ev;
        // scores: register 4 t + i of the lane is token t0 + 8 g + 4 t + i
        float s[NT][8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          f16x8 a[D / 32];
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            const int p = t * (D / 64) + w;
            a[2 * w] = decode8<CODE>(kc[p].x, kc[p].y);
            a[2 * w + 1] = decode8<CODE>(kc[p].z, kc[p].w);
            kc[p] = codes_piece(rk, p);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < D / 32; ++w) acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[w], q[n][w], acc, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][4 * t + i] = acc[i];
          }
        }
        // every row sees the whole block unless it reaches past the first row or before a window
        if (!held || t0 + kKvBlock - 1 > p0 || (A.window > 0 && t0 <= p1 - A.window)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              s[n][j] = held && row_sees(pos[n], t0 + 8 * g + j, A.window, A.sinks) ? s[n][j] : -INFINITY;
          // codes past the end are whatever the memory held
          const int left = min(max(len - (t0 + 8 * g), 0), 8);
          const unsigned lo = left >= 4 ? ~0u : (1u << (8 * left)) - 1u;
          const unsigned hi = left >= 8 ? ~0u : (left > 4 ? (1u << (8 * (left - 4))) - 1u : 0u);
#pragma unroll
          for (int p = 0; p < D / 32; ++p) vc[p] &= u32x4{lo, hi, lo, hi};
        }
        float mul[NT], top[NT];
        bool move = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mul[n] = score_factor(row_mul[n], ek);
          top[n] = s[n][0];
#pragma unroll
          for (int j = 1; j < 8; ++j) top[n] = fmaxf(top[n], s[n][j]);
          top[n] *= mul[n];
          move |= passes(st[n], top[n], evf);
        }
        if (__any(move)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float x = fmaxf(top[n], __shfl_xor(top[n], 16));
            x = fmaxf(x, __shfl_xor(x, 32));
            const float f = move_refs(st[n], x, evf);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) o[n][d] *= f;
          }
        }
        f16x8 w[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) weigh<8>(st[n], s[n], mul[n], evf, &w[n]);
#pragma unroll
        for (int p = 0; p < D / 32; ++p) {
          const f16x8 a = decode8<CODE>(vc[p].x, vc[p].y), b = decode8<CODE>(vc[p].z, vc[p].w);
          vc[p] = codes_piece(rv, p);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[n][2 * p] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, w[n], o[n][2 * p], 0, 0, 0);
            o[n][2 * p + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, w[n], o[n][2 * p + 1], 0, 0, 0);
          }
        }
      }
    }

    // ---- join the waves: the row's state and O' through LDS -------------------------------------------
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float l = st[n].l;
      l += __shfl_xor(l, 16);
      l += __shfl_xor(l, 32);
      float* to = s_part[wave][16 * n + col];
#pragma unroll
      for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f32x4*>(to + 16 * d + 4 * g) = o[n][d];
      if (g == 0) *reinterpret_cast<f32x4*>(to + D) = f32x4{st[n].rr, st[n].mm, l, 0.f};
    }
    __syncthreads();
    auto store_row = [&](int r, int d, const f32x4& u, const RowState& of) {
      const int j = (r * inv_group) >> 16, h = head * A.group + r - j * A.group;
      f32x4 v = u;
      RowState a = of;
      if constexpr (MODE == ATTEND_SHARED) {
        put_state<D>(A, 0, row0 + j, h, d, v, a);
        return;
      }
      if constexpr (MODE == ATTEND_OWN)
        if (shared > 0) join_state<D>(A, parts_of(A, shared), row0 + j, h, d, v, a);
      T* out = static_cast<T*>(A.out.data) + (int64_t)(row0 + j) * A.out.token + (int64_t)h * A.out.head + d;
      const float half = out_half(a);
      typedef T T4 __attribute__((ext_vector_type(4)));
      T4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = rounded<ACT>(out_value(v[e], a.l, half));
      *reinterpret_cast<T4*>(out) = y;
      if (d == 0 && A.lse != nullptr) A.lse[(size_t)(row0 + j) * A.heads + h] = row_lse(a);
    };
    auto store_part = [&](int at, int r, int d, const f32x4& v, const RowState& a) {
      const int to = (at * kRows + r) * kRow;
      put4(prs, to + d, v);
      if (d == 0) put4(prs, to + D, f32x4{a.rr, a.mm, a.l, 0.f});
    };
    // the rows' joined states and the waves' factors, once a row
    if ((int)threadIdx.x < R) {
      RowState a{-INFINITY, -INFINITY, 0.0f};
      f32x4 x[kWaves];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        x[w] = *reinterpret_cast<const f32x4*>(&s_part[w][threadIdx.x][D]);
        a.rr = fmaxf(a.rr, x[w].x);
        a.mm = fmaxf(a.mm, x[w].y);
      }
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        a.l += x[w].z * ex2_diff(x[w].y, a.mm);
        s_part[w][threadIdx.x][D + 3] = ex2_diff(x[w].x, a.rr);
      }
      *reinterpret_cast<f32x4*>(&s_part[0][threadIdx.x][D]) = f32x4{a.rr, a.mm, a.l, s_part[0][threadIdx.x][D + 3]};
    }
    __syncthreads();
    for (int k = threadIdx.x; k < R * (D / 4); k += WAVE * kWaves) {
      const int r = k / (D / 4), d = 4 * (k % (D / 4));
      const f32x4 x = *reinterpret_cast<const f32x4*>(&s_part[0][r][D]);
      f32x4 v = *reinterpret_cast<const f32x4*>(&s_part[0][r][d]) * x.w;
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += *reinterpret_cast<const f32x4*>(&s_part[w][r][d]) * s_part[w][r][D + 3];
      const RowState a{x.x, x.y, x.z};
      if (parts == 1)
        store_row(r, d, v, a);
      else
        store_part(first + part, r, d, v, a);
    }
    if (parts > 1) {
      // `fan` parts from w0 on are joined by the last of them, then these by the last of those
      const int fan = fan_of(parts), groups = (parts + fan - 1) / fan;
      const int w0 = first + part / fan * fan, m = min(fan, first + parts - w0);
      if (last_of(A.tickets + w0, m, &s_last)) {
        float* lds = &s_part[0][0][0];
        if (groups == 1) {
          join_parts<D, kRows, kWaves>(prs, lds, first, 1, m, R, store_row);
        } else {
          join_parts<D, kRows, kWaves>(prs, lds, w0, 1, m, R,
                               [&](int r, int d, const f32x4& v, const RowState& a) { store_part(w0, r, d, v, a); });
          if (last_of(A.tickets + kStepTickets / 2 + first, groups, &s_last))
            join_parts<D, kRows, kWaves>(prs, lds, first, fan, groups, R, store_row);
        }
      }
    }
    __syncthreads();   // s_part is free again
  }
}

template <int MODE, int ACT, int CODE, int D, int NT>
hipError_t step_go(const AttendArgs<MODE>& a, hipStream_t s) {
  hipLaunchKernelGGL((k_kv_step<MODE, ACT, CODE, D, NT>), dim3(step_launch(NT, D, items_of<MODE>(a) * a.c.kv_heads)),
                     dim3(WAVE * step_waves(NT, D)), 0, s, a);
  return hipGetLastError();
}

template <int MODE, int ACT, int CODE, int D>
hipError_t step_rows(const AttendArgs<MODE>& a, hipStream_t s) {
  const int rows = a.max_new * a.group;
  if (rows <= 16) return step_go<MODE, ACT, CODE, D, 1>(a, s);
  if (rows <= 32) return step_go<MODE, ACT, CODE, D, 2>(a, s);
  return step_go<MODE, ACT, CODE, D, 4>(a, s);
}

template <int MODE, int ACT>
hipError_t step_code(int code, const AttendArgs<MODE>& a, hipStream_t s) {
  if (code == CODE_E4M3)
    return a.c.dim == 128 ? step_rows<MODE, ACT, CODE_E4M3, 128>(a, s) : step_rows<MODE, ACT, CODE_E4M3, 64>(a, s);
  return a.c.dim == 128 ? step_rows<MODE, ACT, CODE_INT8, 128>(a, s) : step_rows<MODE, ACT, CODE_INT8, 64>(a, s);
}

template <int MODE>
hipError_t step_act(int act, int code, const AttendArgs<MODE>& a, hipStream_t s) {
  if (a.max_new < 1 || (long long)a.max_new * a.group > kStepRows) return hipErrorInvalidValue;
  return act == ACT_F16 ? step_code<MODE, ACT_F16>(code, a, s) : step_code<MODE, ACT_BF16>(code, a, s);
}

}  // namespace

}  // namespace pik
