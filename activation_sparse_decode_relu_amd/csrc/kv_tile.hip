// Attention of many rows: prompts, and pieces of prompts over what earlier pieces left.
//
// Bound by the matrix instructions and, as much, by the exponentials: a row and token costs 4 D operations of
// the one and one of the other.  A workgroup takes 128 rows (query heads of a cached head times tokens),
// four waves of 32, and passes over the tokens they see in tiles of 64.  The codes of a tile are
// decoded once, to fp16 operands in LDS that every wave reads in whole lines (the 32x32x16 fragments,
// lane after lane), into one of two buffers while the other is being used; the next tile's codes are on
// their way from memory meanwhile.  Scores, softmax and output never leave the registers (kv_softmax.h).
// Tiles that no row of a wave sees are skipped, and only those at the diagonal or at a window's edge
// are masked.
//
// Workgroups that read the same cached head stand kv_heads apart, so with 8 heads or a multiple they share
// an L2, and the longest rows come first.  With few workgroups the tokens are split over several of
// them; their states (fp32) are joined by a second kernel.
#include "kv_softmax.h"

namespace pik {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileWaves = 4, kTileThreads = kTileWaves * WAVE;
static_assert(kTileRows == 32 * kTileWaves, "a wave takes 32 rows");
constexpr int kMinTiles = 4;    // 64-token tiles a split is worth at least

// One workgroup's rows, tokens and share of them.
struct TileJob {
  KvSeq s;
  int r0, R;            // first of its rows and how many the sequence has (tokens times group)
  int p0;               // position of the sequence's first row
  Span span;
  int begin, end;       // 64-token tiles of the span
  int splits;           // how many workgroups share the span
  __device__ __forceinline__ int pos(int r, int group) const { return p0 + r / group; }
};

__device__ __forceinline__ bool tile_job(const KvAttendArgs& A, int slot, int split, TileJob& j) {
  int local;
  const int i = slot_owner(A.c, slot, A.group, kTileRows, 1, local);
  j.s = kv_seq(A.c, i);
  j.R = min(j.s.rows, A.max_new) * A.group;
  j.r0 = local * kTileRows;
  if (j.r0 >= j.R) return false;
  j.p0 = j.s.len - j.s.rows;
  j.span = span_of(j.pos(j.r0, A.group), j.pos(min(j.R, j.r0 + kTileRows) - 1, A.group), A.window, A.sinks);
  if (j.s.seq < 0) j.span = Span{0, 0, 0};
  const int tiles = (j.span.count() + 1) / 2;
  const int per = max((tiles + A.splits - 1) / A.splits, kMinTiles);
  j.splits = max((tiles + per - 1) / per, 1);
  j.begin = split * per;
  j.end = min(j.begin + per, tiles);
  return split < j.splits;
}

// The two blocks of a tile: first token and exponents (K's, V's << 8), the latter -1 where there is no page.
struct Tile {
  int ta, tb, xa, xb;
};

template <int ACT, int CODE, int D>
__global__ __launch_bounds__(kTileThreads, 2) void k_kv_tile(const KvAttendArgs A) {
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
  const int split = rest % A.splits, slot = A.slots - 1 - rest / A.splits;
  TileJob job;
  if (!tile_job(A, slot, split, job)) return;

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
  u32x4 codes[kMine];
  const int unit = tid % kUnits, side = kUnits < kTileThreads ? wave / (kTileWaves / 2) : 0;
  int k_to, v_to;
  {
    const int t = unit / D, chunk = (unit / 16) % (D / 16), rr = unit % 16;
    k_to = 2 * chunk * 32 + 8 * (2 * (rr >> 3) + t) + 4 * ((rr >> 2) & 1) + (rr & 3);   // the row where the token's scores shall come out
    const int p = unit / 64, g = (unit / 16) % 4;
    v_to = ((((g >> 1) * (D / 32) + p) * 2) + (g & 1)) * 32 + unit % 16;
  }
  auto fetch = [&](int tile) {
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
    const size_t at[2] = {off(k), off(k + 1)};
#pragma unroll
    for (int e = 0; e < kMine; ++e) {
      const uint8_t* p = (e < kMine / 2 ? c.k : c.v) + (kMine == 4 ? at[e & 1] : side ? at[1] : at[0]);
      codes[e] = *(reinterpret_cast<const u32x4*>(p) + unit);
    }
    return Tile{lane_of(vblk, k) * kKvBlock, lane_of(vblk, k + 1) * kKvBlock, lane_of(vexps, k), lane_of(vexps, k + 1)};
  };
  // this thread's units, decoded, to their places
  auto stage = [&](int buf, const Tile& m) {
    // V's codes of tokens that are not there may be anything, and their weight of 0 is not enough
    if (m.xa < 0 || m.xb < 0 || max(m.ta, m.tb) + kKvBlock > job.s.len) {
#pragma unroll
      for (int e = kMine / 2; e < kMine; ++e) {
        const bool b = kMine == 4 ? e & 1 : side != 0;
        const int left = (b ? m.xb : m.xa) < 0 ? 0 : min(max(job.s.len - ((b ? m.tb : m.ta) + 8 * ((unit / 16) % 4)), 0), 8);
        const unsigned lo = left >= 4 ? ~0u : (1u << (8 * left)) - 1u;
        const unsigned hi = left >= 8 ? ~0u : (left > 4 ? (1u << (8 * (left - 4))) - 1u : 0u);
        codes[e] &= u32x4{lo, hi, lo, hi};
      }
    }
#pragma unroll
    for (int e = 0; e < kMine; ++e) {
      const int b = kMine == 4 ? e & 1 : side;
      f16x8* to = e < kMine / 2 ? &s_k[buf][b][k_to] : &s_v[buf][b][v_to];
      to[0] = decode8<CODE>(codes[e].x, codes[e].y);
      to[e < kMine / 2 ? 32 : 16] = decode8<CODE>(codes[e].z, codes[e].w);
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
  // does a row of this wave see the block; do all of them see all of it
  auto seen = [&](int t0, int ex) {
    return ex >= 0 && t0 <= wp1 && (A.window == 0 || t0 < A.sinks || t0 + kKvBlock - 1 > wp0 - A.window);
  };
  auto whole = [&](int t0, int ex) {
    return ex >= 0 && t0 + kKvBlock - 1 <= wp0 && (A.window == 0 || t0 > wp1 - A.window);
  };
  auto compute = [&](int buf, const Tile& m) {
    const float ka = score_factor(row_mul, max((m.xa & 255) - 127, -126)), kb = score_factor(row_mul, max((m.xb & 255) - 127, -126));
    const float va = (float)max(((m.xa >> 8) & 255) - 127, -126), vb = (float)max(((m.xb >> 8) & 255) - 127, -126);
    if (!seen(m.ta, m.xa) && !seen(m.tb, m.xb)) return;
    f32x16 sa = scores(s_k[buf][0]), sb = scores(s_k[buf][1]);
    if (!whole(m.ta, m.xa) || !whole(m.tb, m.xb)) {
      mask(sa, m.ta, m.xa);
      mask(sb, m.tb, m.xb);
    }
    const float ma = top_of(sa) * ka, mb = top_of(sb) * kb;
    if (__any(passes(st, ma, va) || passes(st, mb, vb))) {
      float f = move_refs(st, fmaxf(ma, __shfl_xor(ma, 32)), va);
      f *= move_refs(st, fmaxf(mb, __shfl_xor(mb, 32)), vb);
#pragma unroll
      for (int d = 0; d < D / 32; ++d) o[d] *= f;
    }
    values(s_v[buf][0], sa, ka, va);
    values(s_v[buf][1], sb, kb, vb);
  };

  if (job.begin < job.end) {
    Tile cur = fetch(job.begin), nxt = cur;
    stage(0, cur);
    if (job.begin + 1 < job.end) nxt = fetch(job.begin + 1);
    __syncthreads();
    for (int t = job.begin; t < job.end; ++t) {
      const int buf = (t - job.begin) & 1;
      compute(buf, cur);
      if (t + 1 < job.end) {
        stage(buf ^ 1, nxt);
        cur = nxt;
        if (t + 2 < job.end) nxt = fetch(t + 2);
      }
      __syncthreads();
    }
  }

  // ---- out: register 4 a + e of o[d] is dim 32 d + 8 a + 4 h + e ---------------------------------------
  st.l += __shfl_xor(st.l, 32);
  if (!live) return;
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
  T* out = static_cast<T*>(A.out.data) + (int64_t)(job.s.row0 + j) * A.out.token + (int64_t)hq * A.out.head;
  const float half = out_half(st), inv = 1.0f / st.l;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      typedef T T4 __attribute__((ext_vector_type(4)));
      T4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (T)(st.l != 0.0f ? o[d][4 * a + e] * inv * half * half : 0.0f);
      *reinterpret_cast<T4*>(out + 32 * d + 8 * a + 4 * h) = v;
    }
  if (h == 0 && A.lse != nullptr) A.lse[(size_t)(job.s.row0 + j) * A.heads + hq] = row_lse(st);
}

// Joins the splits of 32 rows of a workgroup's tile, in their order.
template <int ACT, int D>
__global__ __launch_bounds__(kTileThreads) void k_kv_tile_join(const KvAttendArgs A) {
  using T = typename ActT<ACT>::T;
  const KvView& c = A.c;
  const int head = blockIdx.x % c.kv_heads, slot = blockIdx.x / c.kv_heads;
  TileJob job;
  if (!tile_job(A, slot, 0, job) || job.splits == 1) return;
  for (int k = threadIdx.x; k < 32 * (D / 4); k += kTileThreads) {
    const int local = 32 * blockIdx.y + k / (D / 4), d = 4 * (k % (D / 4)), r = job.r0 + local;
    if (r >= job.R) return;
    const float* from = A.partial + ((size_t)slot * c.kv_heads + head) * A.splits * ((size_t)kTileRows * (D + 4)) +
                        (size_t)local * (D + 4);
    RowState a{-INFINITY, -INFINITY, 0.0f};
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < job.splits; ++p, from += (size_t)kTileRows * (D + 4)) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(from + D), y = *reinterpret_cast<const f32x4*>(from + d);
      float fa, fb;
      join(a, RowState{x.x, x.y, x.z}, fa, fb);
      v = v * fa + y * fb;
    }
    const int j = r / A.group, hq = head * A.group + r - j * A.group;
    T* out = static_cast<T*>(A.out.data) + (int64_t)(job.s.row0 + j) * A.out.token + (int64_t)hq * A.out.head + d;
    const float half = out_half(a);
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = (T)out_value(v[e], a.l, half);
    if (d == 0 && A.lse != nullptr) A.lse[(size_t)(job.s.row0 + j) * A.heads + hq] = row_lse(a);
  }
}

template <int ACT, int CODE, int D>
hipError_t tile_go(KvAttendArgs a, hipStream_t s) {
  const long long slots = (long long)a.c.rows * a.group / kTileRows + a.c.n, items = slots * a.c.kv_heads;
  if (items > 0x7fffffff) return hipErrorInvalidValue;
  a.slots = (int)slots;
  a.splits = items > kTileParts / 2 ? 1 : (int)(kTileParts / items);
  hipLaunchKernelGGL((k_kv_tile<ACT, CODE, D>), dim3((unsigned)(items * a.splits)), dim3(kTileThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((k_kv_tile_join<ACT, D>), dim3((unsigned)items, kTileRows / 32), dim3(kTileThreads), 0, s, a);
  return hipGetLastError();
}

template <int ACT>
hipError_t tile_code(int code, const KvAttendArgs& a, hipStream_t s) {
  if (code == CODE_E4M3) return a.c.dim == 128 ? tile_go<ACT, CODE_E4M3, 128>(a, s) : tile_go<ACT, CODE_E4M3, 64>(a, s);
  return a.c.dim == 128 ? tile_go<ACT, CODE_INT8, 128>(a, s) : tile_go<ACT, CODE_INT8, 64>(a, s);
}

}  // namespace

hipError_t launch_kv_tile(int act, int code, const KvAttendArgs& a, hipStream_t s) {
  return act == ACT_F16 ? tile_code<ACT_F16>(code, a, s) : tile_code<ACT_BF16>(code, a, s);
}

}  // namespace pik
