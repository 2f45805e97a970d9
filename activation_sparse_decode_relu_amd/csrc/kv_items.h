// What the attention kernels take as an item: a sequence, a group of sequences with the tokens they share, or a
// sequence with the tokens behind these.  Everything that only the device knows is bounded here, as in kv_device.h.
#pragma once

#include "kv_softmax.h"

namespace pik {

// (Not by an expression of the modes: their enumeration has no name, and the compiler's passes for host and device number
// such types apart, so a kernel with one in its signature would not be found.)
template <int MODE> struct AttendArgsOf { using T = KvSharedArgs; };
template <> struct AttendArgsOf<ATTEND_ALL> { using T = KvAttendArgs; };
template <int MODE> using AttendArgs = typename AttendArgsOf<MODE>::T;

template <int MODE>
__host__ __device__ __forceinline__ int items_of(const AttendArgs<MODE>& A) {
  if constexpr (MODE == ATTEND_SHARED) return A.n_groups;
  else return A.c.n;
}

// Entry `at` of the plan: whole blocks, within what a sequence can hold.
__device__ __forceinline__ int shared_of(const KvSharedArgs& A, int at) {
  return min(max(A.plan[at], 0), A.c.max_pages * A.c.page_blocks * kKvBlock) & ~(kKvBlock - 1);
}

// First sequence of group g; that of the group after it, of the last too.
__device__ __forceinline__ int group_at(const int* groups, int g, int n) { return min(max(groups[g], 0), n); }

// First row of an item; item items_of() is the end.
template <int MODE>
__device__ __forceinline__ int item_start(const AttendArgs<MODE>& A, int i) {
  if constexpr (MODE == ATTEND_SHARED) i = group_at(A.groups, i, A.c.n);
  return min(max(A.c.starts[i], 0), A.c.rows);
}

template <int MODE>
__device__ __forceinline__ KvSeq item_seq(const AttendArgs<MODE>& A, int i) {
  if constexpr (MODE == ATTEND_SHARED) {
    // the group's tokens are read where its first sequence has them; groups that share nothing have no rows here
    const int g0 = group_at(A.groups, i, A.c.n);
    const int q = g0 < A.c.n ? A.c.seqs[g0] : -1;
    KvSeq s;
    s.seq = q >= 0 && q < A.c.max_seqs ? q : -1;
    s.len = shared_of(A, i);
    s.row0 = item_start<MODE>(A, i);
    s.rows = s.len > 0 ? max(item_start<MODE>(A, i + 1) - s.row0, 0) : 0;
    return s;
  } else {
    return kv_seq(A.c, i);
  }
}

// Position of an item's first row.  Every row of a group stands behind all that the group shares.
template <int MODE>
__device__ __forceinline__ int item_first(const KvSeq& s) {
  if constexpr (MODE == ATTEND_SHARED) return s.len;
  else return s.len - s.rows;
}

template <int MODE>
__host__ __device__ __forceinline__ Span item_span(const AttendArgs<MODE>& A, int len, int shared, int p0, int p1) {
  if constexpr (MODE == ATTEND_SHARED) return Span{0, 0, len / kKvBlock};
  Span s = span_of(p0, p1, A.window, A.sinks);
  // at the last block, where a plan that does not fit says more: the block behind it may lie past the table
  if constexpr (MODE == ATTEND_OWN) s.from = min(shared / kKvBlock, max(s.end - 1, 0));
  return s;
}

// slot_owner() over items.  Groups begin their slots at floor((rows before - i) / unit) + i: as many as a unit's
// rounding up needs, and no more with one group.
template <int MODE>
__device__ __forceinline__ int item_owner(const AttendArgs<MODE>& A, int slot, int unit, int& local) {
  if constexpr (MODE != ATTEND_SHARED) return slot_owner(A.c, slot, A.group, unit, 1, local);
  const int lane = threadIdx.x & (WAVE - 1), items = items_of<MODE>(A);
  int owner = 0;
  local = slot;
  for (int base = 0; base < items; base += WAVE) {
    const int i = base + lane;
    const long long at = i < items ? ((long long)item_start<MODE>(A, i) * A.group + (long long)i * (unit - 1)) / unit
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

// ---- the states of shared tokens ----------------------------------------------------------------------

// The kernel of many rows splits the 64-token tiles of a group: into how many parts, and of how many tiles.
constexpr int kMinTiles = 4;    // tiles a part is worth at least
__device__ __forceinline__ int tiles_each(int tiles, int splits) { return max((tiles + splits - 1) / splits, kMinTiles); }
__device__ __forceinline__ int parts_of(const KvSharedArgs& A, int shared) {
  if (A.parts == 1) return 1;
  const int tiles = (shared / kKvBlock + 1) / 2, per = tiles_each(tiles, A.parts);
  return (tiles + per - 1) / per;
}

template <int D>
__device__ __forceinline__ float* state_at(const KvSharedArgs& A, int part, int row, int head) {
  return A.state + (((size_t)part * A.c.rows + row) * A.heads + head) * (D + 4);
}
// Four dims of a row's O', and with the first its state.
template <int D>
__device__ __forceinline__ void put_state(const KvSharedArgs& A, int part, int row, int head, int d, const f32x4& v,
                                          const RowState& a) {
  float* to = state_at<D>(A, part, row, head);
  *reinterpret_cast<f32x4*>(to + d) = v;
  if (d == 0) *reinterpret_cast<f32x4*>(to + D) = f32x4{a.rr, a.mm, a.l, 0.f};
}
// Four dims of a row's O' and its state, joined with what put_state left in `parts` parts, in their order.
template <int D>
__device__ __forceinline__ void join_state(const KvSharedArgs& A, int parts, int row, int head, int d, f32x4& v, RowState& a) {
  constexpr int kBatch = 4;   // parts whose loads are on their way together
  const float* from = state_at<D>(A, 0, row, head);
  const size_t step = (size_t)A.c.rows * A.heads * (D + 4);
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  RowState b{-INFINITY, -INFINITY, 0.0f};
  float fb, fa;
  for (int p0 = 0; p0 < parts; p0 += kBatch) {
    f32x4 u[kBatch], s[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const float* at = from + min(p0 + e, parts - 1) * step;
      u[e] = *reinterpret_cast<const f32x4*>(at + d);
      s[e] = *reinterpret_cast<const f32x4*>(at + D);
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (p0 + e < parts) {
        join(b, RowState{s[e].x, s[e].y, s[e].z}, fb, fa);
        sum = sum * fb + u[e] * fa;
      }
  }
  join(b, a, fb, fa);
  v = sum * fb + v * fa;
  a = b;
}

}  // namespace pik
