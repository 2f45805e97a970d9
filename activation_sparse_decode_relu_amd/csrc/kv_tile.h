// Attention of many rows: prompts, and pieces of prompts over what earlier pieces left.
//
// Bound by the matrix instructions and, as much, by the vector ALU: a row and token costs 4 D operations of the one
// and, of the other, an exponential and about six more (scale, maximum, sum, rounding, its share of the decoding).
// A workgroup takes 128 rows (query heads of a cached head times tokens), four waves of 32, and passes over the
// tokens they see in tiles of two blocks.  The codes of a tile are decoded once, to fp16 operands in LDS that every
// wave reads in whole lines (the 32x32x16 fragments, lane after lane), into one of two buffers while the other is being
// used; the next tile's codes are on their way from memory meanwhile.  Scores, softmax and output never leave the
// registers (kv_softmax.h).  The scores of one block are computed beside the exponentials of the block before.  Only
// blocks at the diagonal or at a window's edge are masked.
//
// Workgroups that read the same cached head stand kv_heads apart, so with 8 heads or a multiple they share an L2,
// and the longest rows come first.  With few workgroups the tokens are split over several of them; their states
// (fp32) are joined by a second kernel.
//
// Measured, a prompt of 4096 with 64 query heads on 8: 306 to 337 us on different cards, 816 to 897 TFLOP/s (a library
// matrix product of 8192 runs at 1107 to 1167), the matrix instructions busy 38 % of the time and the vector ALU 50 %.
// One workgroup a compute unit instead of two took 440 us where this took 318; three, with blocks of 32 tokens in turn
// so that the registers suffice, 322.  Raising a wave's priority in its products, or interleaving these with the
// exponentials one by one, was 1 to 6 % slower.
#pragma once

#include "kv_items.h"

namespace pik {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileWaves = 4, kTileThreads = kTileWaves * WAVE;
static_assert(kTileRows == 32 * kTileWaves, "a wave takes 32 rows");

// One workgroup's rows, tokens and share of them.
struct TileJob {
  KvSeq s;
  int r0, R;            // first of its rows and how many the sequence has (tokens times group)
  int p0;               // position of the sequence's first row
  Span span;
  int begin, end;       // 64-token tiles of the span
  int splits;           // how many workgroups share the span
  int shared = 0;       // ATTEND_OWN: tokens that others have attended over
  __device__ __forceinline__ int pos(int r, int group) const { return p0 + r / group; }
};

// Up to 64 sequences: which of them owns `slot`, and its tile of rows, in the order in which the card is best
// kept busy to the end: the longest sequences first and each one's last rows first.
template <int MODE>
__device__ __forceinline__ int sorted_owner(const AttendArgs<MODE>& A, int slot, int& local) {
  const int items = items_of<MODE>(A), lane = threadIdx.x & (WAVE - 1), i = min(lane, items - 1);
  auto lane_of = [](int v, int k) { return __builtin_amdgcn_readlane(v, k); };
  auto at = [&](int k) {   // less k
    const long long r = (long long)item_start<MODE>(A, k) * A.group;
    if constexpr (MODE == ATTEND_SHARED) return (int)((r + (long long)k * (kTileRows - 1)) / kTileRows) - k;
    else return (int)(r / kTileRows);
  };
  const int count = max(at(i + 1) + 1 - at(i), 0), len = item_seq<MODE>(A, i).len;
  int before = 0;
  for (int k = 0; k < items; ++k) {
    const int other = lane_of(len, k);
    before += other > len || (other == len && k < lane) ? lane_of(count, k) : 0;
  }
  const unsigned long long mine = __ballot(lane < items && slot >= before && slot < before + count);
  if (mine == 0) return -1;
  const int owner = __builtin_ctzll(mine);
  local = lane_of(count, owner) - 1 - (slot - lane_of(before, owner));
  return owner;
}

template <int MODE>
__device__ __forceinline__ bool tile_job(const AttendArgs<MODE>& A, int slot, int split, TileJob& j) {
  int local;
  const int i = items_of<MODE>(A) <= WAVE ? sorted_owner<MODE>(A, slot, local)
                                          : item_owner<MODE>(A, A.slots - 1 - slot, kTileRows, local);
  if (i < 0) return false;
  j.s = item_seq<MODE>(A, i);
  if constexpr (MODE == ATTEND_OWN) j.shared = shared_of(A, A.n_groups + i);
  j.R = min(j.s.rows, A.max_new) * A.group;
  j.r0 = local * kTileRows;
  if (j.r0 >= j.R) return false;
  j.p0 = item_first<MODE>(j.s);
  j.span = item_span<MODE>(A, j.s.len, j.shared, j.pos(j.r0, A.group), j.pos(min(j.R, j.r0 + kTileRows) - 1, A.group));
  if (j.s.seq < 0) j.span = Span{0, 0, 0};
  const int tiles = (j.span.count() + 1) / 2;
  const int per = tiles_each(tiles, A.splits);
  j.splits = max((tiles + per - 1) / per, 1);
  j.begin = split * per;
  j.end = min(j.begin + per, tiles);
  return split < j.splits;
}

// The two blocks of a tile: first token and exponents (K's, V's << 8), the latter -1 where there is no page.
struct Tile {
  int ta, tb, xa, xb;
  size_t oa, ob;        // where the blocks' codes begin
};

template <int MODE, int ACT, int CODE, int D>
__global__ __launch_bounds__(kTileThreads, 2) void k_kv_tile(const AttendArgs<MODE> A) {
  using T = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  constexpr int kUnits = 2 * D;                            // 16-byte units of a block's codes
  constexpr int kMine = 4 * kUnits / kTileThreads;         // of a tile, K and V, a thread's share
  constexpr int kFrag = 32 * D / 8;                        // fp16 operands (16 bytes) of a block
  __shared__ f16x8 s_k[2][2][kFrag], s_v[2][2][kFrag];     // [buffer][block]
  const KvView& c = A.c;
  const int tid = threadIdx.x, lane = tid & (WAVE - 1), wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int col = lane & 31, h = lane >> 5;
  const int head = blockIdx.x % c.kv_heads, rest = blockIdx.x / c.kv_heads;
  const int split = rest % A.splits, slot = rest / A.splits;
  TileJob job;
  if (!tile_job<MODE>(A, slot, split, job)) return;

  // ---- the rows ---------------------------------------------------------------------------------------
  const int w0 = job.r0 + 32 * wave, r = w0 + col;
  const bool live = r < job.R, busy = w0 < job.R;
  const int j = live ? r / A.group : 0, hq = head * A.group + (live ? r - j * A.group : 0);
  const int pos = live ? job.p0 + j : -1;
  const int wp0 = job.pos(w0, A.group), wp1 = busy ? job.pos(min(w0 + 31, job.R - 1), A.group) : -1;
  f16x8 q[D / 16];
  float row_mul;
  {
    const T* src = static_cast<const T*>(A.q.data) + (int64_t)(job.s.row0 + j) * A.q.token + (int64_t)hq * A.q.head;
    V8 x[D / 16];
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      x[s] = V8{};
      if (live) x[s] = *reinterpret_cast<const V8*>(src + 16 * s + 8 * h);
    }
    float up = 1.0f, down = 1.0f;
    if constexpr (ACT == ACT_BF16) {
      float m = 0.0f;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) m = fmaxf(m, max8<ACT>(x[s]));
      up = query_scale(fmaxf(m, __shfl_xor(m, 32)), down);
    }
#pragma unroll
    for (int s = 0; s < D / 16; ++s) q[s] = query8<ACT>(x[s], up);
    row_mul = A.scale * kLog2e * down;
  }
  RowRun st = row_run();
  f32x16 o[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;

  // ---- tiles: memory -> registers -> LDS -----------------------------------------------------------------
  // A thread carries the same unit of every block: its place in memory and in LDS is worked out once.
  int vexps = -1, vblk = 0, window0 = 0, window1 = 0;   // lane k: block window0 + k of the span
  size_t voff = 0;
  u32x4 kc[kMine / 2], vc[kMine / 2];
  const int unit = tid % kUnits, side = kUnits < kTileThreads ? wave / (kTileWaves / 2) : 0;
  int k_to, v_to;
  {
    const int t = unit / D, chunk = (unit / 16) % (D / 16), rr = unit % 16;
    // K: the row where the token's scores shall come out
    k_to = 2 * chunk * 32 + 8 * (2 * (rr >> 3) + t) + 4 * ((rr >> 2) & 1) + (rr & 3);
    const int p = unit / 64, g = (unit / 16) % 4;
    v_to = ((((g >> 1) * (D / 32) + p) * 2) + (g & 1)) * 32 + unit % 16;
  }
  auto find = [&](int tile) {
    if (2 * tile >= window1) {
      window0 = 2 * tile;
      window1 = window0 + WAVE;
      const int bi = window0 + lane;
      vexps = -1;
      vblk = 0;
      voff = 0;
      if (bi < min(job.span.count(), 2 * job.end)) {
        vblk = job.span.block(bi);
        const int page = kv_page(c, job.s.seq, vblk);
        if (page >= 0) {
          const size_t e = block_at(c, page, head, vblk % c.page_blocks);
          vexps = (int)c.k_exp[e] | (int)c.v_exp[e] << 8;
          voff = e * (kKvBlock * D);
        }
      }
    }
    const int k = 2 * tile - window0;
    auto lane_of = [&](int v, int i) { return __builtin_amdgcn_readlane(v, i); };
    auto off = [&](int i) {
      return (size_t)(unsigned)lane_of((int)(unsigned)voff, i) | (size_t)(unsigned)lane_of((int)(voff >> 32), i) << 32;
    };
    return Tile{lane_of(vblk, k) * kKvBlock, lane_of(vblk, k + 1) * kKvBlock, lane_of(vexps, k), lane_of(vexps, k + 1),
                off(k), off(k + 1)};
  };
  // this thread's units of two blocks: on their way from memory, and, decoded, to their places
  auto fetch = [&](const uint8_t* base, size_t first, size_t second, u32x4* to) {
#pragma unroll
    for (int e = 0; e < kMine / 2; ++e) {
      const size_t at = kMine == 4 ? (e ? second : first) : side ? second : first;
      to[e] = *(reinterpret_cast<const u32x4*>(base + at) + unit);
    }
  };
  auto stage_k = [&](f16x8* first, f16x8* second) {
#pragma unroll
    for (int e = 0; e < kMine / 2; ++e) {
      f16x8* to = (kMine == 4 ? (e ? second : first) : side ? second : first) + k_to;
      to[0] = decode8<CODE>(kc[e].x, kc[e].y);
      to[32] = decode8<CODE>(kc[e].z, kc[e].w);
    }
  };
  auto stage_v = [&](int buf, const Tile& m) {
    // codes of tokens that are not there may be anything, and their weight of 0 is not enough
    if (m.xa < 0 || m.xb < 0 || max(m.ta, m.tb) + kKvBlock > job.s.len) {
#pragma unroll
      for (int e = 0; e < kMine / 2; ++e) {
        const bool b = kMine == 4 ? e != 0 : side != 0;
        const int first = (b ? m.tb : m.ta) + 8 * ((unit / 16) % 4);
        const int left = (b ? m.xb : m.xa) < 0 ? 0 : min(max(job.s.len - first, 0), 8);
        const unsigned lo = left >= 4 ? ~0u : (1u << (8 * left)) - 1u;
        const unsigned hi = left >= 8 ? ~0u : (left > 4 ? (1u << (8 * (left - 4))) - 1u : 0u);
        vc[e] &= u32x4{lo, hi, lo, hi};
      }
    }
#pragma unroll
    for (int e = 0; e < kMine / 2; ++e) {
      f16x8* to = &s_v[buf][kMine == 4 ? e : side][v_to];
      to[0] = decode8<CODE>(vc[e].x, vc[e].y);
      to[16] = decode8<CODE>(vc[e].z, vc[e].w);
    }
  };
  // scores of a block: register e of the lane is token t0 + 16 (e / 8) + 8 h + e % 8
  auto scores = [&](const f16x8* k) {
    f32x16 acc;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[64 * s + lane], q[s], acc, 0, 0, 0);
    return acc;
  };
  auto mask = [&](f32x16& s, int t0, int ex) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      s[e] = ex >= 0 && row_sees(pos, t0 + 16 * (e / 8) + 8 * h + e % 8, A.window, A.sinks) ? s[e] : -INFINITY;
  };
  auto top_of = [&](const f32x16& s) {
    float m = s[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) m = fmaxf(m, s[e]);
    return m;
  };
  auto values = [&](const f16x8* v, const f32x16& s, float mul, float ev) {
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = s[e];
    f16x8 w[2];
    weigh<16>(st, x, mul, ev, w);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[64 * (k * (D / 32) + d) + lane], w[k], o[d], 0, 0, 0);
  };
  // do all rows of this wave see all of the block
  auto whole = [&](int t0, int ex) {
    return ex >= 0 && t0 + kKvBlock - 1 <= wp0 && (A.window == 0 || t0 > wp1 - A.window);
  };
  // One block: its scores `s` are there already; those of the block after it are computed beside its exponentials,
  // so that the matrix instructions and the vector ALU work at the same time.
  auto step = [&](int t0, int ex, f32x16& s, const f16x8* v, f32x16& next, const f16x8* k) {
    if (!whole(t0, ex)) mask(s, t0, ex);
    const float mul = score_factor(row_mul, max((ex & 255) - 127, -126)), ev = (float)max(((ex >> 8) & 255) - 127, -126);
    const float top = top_of(s) * mul;
    if (__any(passes(st, top, ev))) {
      const float f = move_refs(st, fmaxf(top, __shfl_xor(top, 32)), ev);
#pragma unroll
      for (int d = 0; d < D / 32; ++d) o[d] *= f;
    }
    next = scores(k);
    values(v, s, mul, ev);
  };
  if (job.begin < job.end) {
    // tiles t, t + 1 and t + 2.  K is staged a block further ahead than V: the pair that is on its way is block b of one
    // tile and block a of the next.
    Tile cur = find(job.begin), nxt = find(job.begin + 1), far = find(job.begin + 2);
    fetch(c.k, cur.oa, cur.ob, kc);
    fetch(c.v, cur.oa, cur.ob, vc);
    stage_k(s_k[0][0], s_k[0][1]);
    fetch(c.k, nxt.oa, nxt.oa, kc);
    stage_k(s_k[1][0], s_k[1][0]);
    stage_v(0, cur);
    fetch(c.k, nxt.ob, far.oa, kc);
    fetch(c.v, nxt.oa, nxt.ob, vc);
    __syncthreads();
    f32x16 sa = scores(s_k[0][0]), sb;
    __syncthreads();                        // every wave is past them before tile 2 takes their place
    auto advance = [&](int t, int buf) {
      stage_k(s_k[buf ^ 1][1], s_k[buf][0]);
      stage_v(buf ^ 1, nxt);
      cur = nxt;
      nxt = far;
      if (t + 2 < job.end) {
        far = find(t + 3);
        fetch(c.k, nxt.ob, far.oa, kc);
        fetch(c.v, nxt.oa, nxt.ob, vc);
      }
      __syncthreads();
    };
    // the tiles up to the last that a row of this wave sees
    const int seen = wp1 < 0 ? 0 : (job.span.sink + max(wp1 / kKvBlock - job.span.from, 0)) / 2 + 1;
    const int stop = min(max(seen, job.begin), job.end);
    int t = job.begin;
    for (; t < stop; ++t) {
      const int buf = (t - job.begin) & 1;
      step(cur.ta, cur.xa, sa, s_v[buf][0], sb, s_k[buf][1]);
      step(cur.tb, cur.xb, sb, s_v[buf][1], sa, s_k[buf ^ 1][0]);
      advance(t, buf);
    }
    for (; t < job.end; ++t) advance(t, (t - job.begin) & 1);
  }

  // ---- out: register 4 a + e of o[d] is dim 32 d + 8 a + 4 h + e ---------------------------------------
  st.l += __shfl_xor(st.l, 32);
  if (!live) return;
  if constexpr (MODE == ATTEND_SHARED) {
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int a = 0; a < 4; ++a)
        put_state<D>(A, split, job.s.row0 + j, hq, 32 * d + 8 * a + 4 * h,
                     f32x4{o[d][4 * a], o[d][4 * a + 1], o[d][4 * a + 2], o[d][4 * a + 3]}, st);
    return;
  }
  if (job.splits > 1) {
    float* to = A.partial + (((size_t)slot * c.kv_heads + head) * A.splits + split) * ((size_t)kTileRows * (D + 4)) +
                (size_t)(32 * wave + col) * (D + 4);
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int a = 0; a < 4; ++a)
        *reinterpret_cast<f32x4*>(to + 32 * d + 8 * a + 4 * h) =
            f32x4{o[d][4 * a], o[d][4 * a + 1], o[d][4 * a + 2], o[d][4 * a + 3]};
    if (h == 0) *reinterpret_cast<f32x4*>(to + D) = f32x4{st.rr, st.mm, st.l, 0.f};
    return;
  }
  if constexpr (MODE == ATTEND_OWN)
    if (job.shared > 0) {
      RowState joined = st;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          f32x4 v = {o[d][4 * a], o[d][4 * a + 1], o[d][4 * a + 2], o[d][4 * a + 3]};
          joined = st;
          join_state<D>(A, parts_of(A, job.shared), job.s.row0 + j, hq, 32 * d + 8 * a + 4 * h, v, joined);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[d][4 * a + e] = v[e];
        }
      static_cast<RowState&>(st) = joined;
    }
  T* out = static_cast<T*>(A.out.data) + (int64_t)(job.s.row0 + j) * A.out.token + (int64_t)hq * A.out.head;
  const float half = out_half(st), inv = 1.0f / st.l;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      typedef T T4 __attribute__((ext_vector_type(4)));
      T4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = rounded<ACT>(st.l != 0.0f ? o[d][4 * a + e] * inv * half * half : 0.0f);
      *reinterpret_cast<T4*>(out + 32 * d + 8 * a + 4 * h) = v;
    }
  if (h == 0 && A.lse != nullptr) A.lse[(size_t)(job.s.row0 + j) * A.heads + hq] = row_lse(st);
}

// Joins the splits of kJoinRows rows of a workgroup's tile, in their order: a thread has four dims of a row, and
// the loads of kJoinBatch splits are on their way together (one after the other, 64 splits of 72 rows took 70 us).
constexpr int kJoinBatch = 8;
constexpr int join_rows(int dim) { return kTileThreads / (dim / 4); }
template <int MODE, int ACT, int D>
__global__ __launch_bounds__(kTileThreads) void k_kv_tile_join(const AttendArgs<MODE> A) {
  using T = typename ActT<ACT>::T;
  typedef T T4 __attribute__((ext_vector_type(4)));
  constexpr int kPart = kTileRows * (D + 4);
  const KvView& c = A.c;
  const int head = blockIdx.x % c.kv_heads, slot = blockIdx.x / c.kv_heads;
  TileJob job;
  if (!tile_job<MODE>(A, slot, 0, job) || job.splits == 1) return;
  const int local = join_rows(D) * blockIdx.y + (int)threadIdx.x / (D / 4), d = 4 * ((int)threadIdx.x % (D / 4));
  const int r = job.r0 + local;
  if (r >= job.R) return;
  const float* from = A.partial + ((size_t)slot * c.kv_heads + head) * A.splits * kPart + (size_t)local * (D + 4);
  RowState a{-INFINITY, -INFINITY, 0.0f};
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int p0 = 0; p0 < job.splits; p0 += kJoinBatch) {
    f32x4 x[kJoinBatch], y[kJoinBatch];
#pragma unroll
    for (int e = 0; e < kJoinBatch; ++e) {
      const float* at = from + (size_t)min(p0 + e, job.splits - 1) * kPart;
      x[e] = *reinterpret_cast<const f32x4*>(at + D);
      y[e] = *reinterpret_cast<const f32x4*>(at + d);
    }
#pragma unroll
    for (int e = 0; e < kJoinBatch; ++e)
      if (p0 + e < job.splits) {
        float fa, fb;
        join(a, RowState{x[e].x, x[e].y, x[e].z}, fa, fb);
        v = v * fa + y[e] * fb;
      }
  }
  const int j = r / A.group, hq = head * A.group + r - j * A.group;
  if constexpr (MODE == ATTEND_OWN)
    if (job.shared > 0) join_state<D>(A, parts_of(A, job.shared), job.s.row0 + j, hq, d, v, a);
  T* out = static_cast<T*>(A.out.data) + (int64_t)(job.s.row0 + j) * A.out.token + (int64_t)hq * A.out.head + d;
  const float half = out_half(a);
  T4 w;
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = rounded<ACT>(out_value(v[e], a.l, half));
  *reinterpret_cast<T4*>(out) = w;
  if (d == 0 && A.lse != nullptr) A.lse[(size_t)(job.s.row0 + j) * A.heads + hq] = row_lse(a);
}

template <int MODE, int ACT, int CODE, int D>
hipError_t tile_go(AttendArgs<MODE> a, hipStream_t s) {
  const long long slots = MODE == ATTEND_SHARED ? shared_tiles(a.c.rows, a.group, items_of<MODE>(a))
                                                : (long long)a.c.rows * a.group / kTileRows + items_of<MODE>(a);
  const long long items = slots * a.c.kv_heads;
  if (items > 0x7fffffff) return hipErrorInvalidValue;
  a.slots = (int)slots;
  if constexpr (MODE == ATTEND_SHARED) a.splits = a.parts;
  else a.splits = items > kTileParts / 2 ? 1 : (int)(kTileParts / items);
  hipLaunchKernelGGL((k_kv_tile<MODE, ACT, CODE, D>), dim3((unsigned)(items * a.splits)), dim3(kTileThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1 || MODE == ATTEND_SHARED) return e;
  hipLaunchKernelGGL((k_kv_tile_join<MODE, ACT, D>), dim3((unsigned)items, kTileRows / join_rows(D)), dim3(kTileThreads), 0, s,
                     a);
  return hipGetLastError();
}

template <int MODE, int ACT>
hipError_t tile_code(int code, const AttendArgs<MODE>& a, hipStream_t s) {
  if (code == CODE_E4M3)
    return a.c.dim == 128 ? tile_go<MODE, ACT, CODE_E4M3, 128>(a, s) : tile_go<MODE, ACT, CODE_E4M3, 64>(a, s);
  return a.c.dim == 128 ? tile_go<MODE, ACT, CODE_INT8, 128>(a, s) : tile_go<MODE, ACT, CODE_INT8, 64>(a, s);
}

template <int MODE>
hipError_t tile_act(int act, int code, const AttendArgs<MODE>& a, hipStream_t s) {
  return act == ACT_F16 ? tile_code<MODE, ACT_F16>(code, a, s) : tile_code<MODE, ACT_BF16>(code, a, s);
}

}  // namespace

}  // namespace pik
