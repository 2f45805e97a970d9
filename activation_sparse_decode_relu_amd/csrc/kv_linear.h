// Host-side launch interface of the products with 4-bit weights (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pik {

// A slab: 256 columns of 16 rows, 2 KB of codes and then 256 bytes of scales.
constexpr int kSlabRows = 16, kSlabCols = 256, kSlabBytes = 2304;

struct LinearArgs {
  const uint8_t* packed;   // [tiles][slabs][kSlabBytes]
  const float* factor;     // [tiles * 16]: powers of two that the rows' scales were divided by
  const float* bias;       // [d_out] or NULL
  const void* x;
  const void* add;         // or NULL
  void* y;
  int64_t x_stride, add_stride, y_stride;
  int rows, d_in, d_out;
  int tiles, slabs;
  void* scratch;             // as linear_scratch() lays it out in scratch_bytes
  size_t scratch_bytes;
  const float* row_factor;   // set by the launch: powers of two that rows of x were divided by, or NULL
  float* partial;            // set by the launch: [splits][rows][d_out]
  int splits;                // set by the launch: ranges of slabs
};

// Up to kExactRows rows x stays in its type.  More are taken in tiles of kTileM rows and kTileTiles tiles of outputs; where
// these leave the card with too few workgroups, the slabs are split over up to kMostSplits, each of at least two, and no
// more than `given` bytes of scratch hold the sums of.
constexpr int kExactRows = 64, kTileM = 128, kTileTiles = 8, kMostSplits = 8, kLinearGroups = 512;
struct LinearScratch {
  size_t x, factor, partial, total;   // fp16 rows and their factors (bf16 alone), the ranges' sums
  int splits;
};
inline long long linear_groups(int rows, int d_out) {
  return (long long)((d_out + 16 * kTileTiles - 1) / (16 * kTileTiles)) * ((rows + kTileM - 1) / kTileM);
}
inline LinearScratch linear_scratch(int act, int rows, int d_in, int d_out, size_t given = SIZE_MAX) {
  LinearScratch l{};
  l.splits = 1;
  if (rows <= kExactRows) return l;
  auto align = [](size_t v) { return (v + 255) / 256 * 256; };
  if (act != 0) {
    l.factor = align((size_t)rows * d_in * 2);
    l.total = l.partial = align(l.factor + (size_t)rows * 4);
  }
  const int slabs = (d_in + kSlabCols - 1) / kSlabCols;
  const long long groups = linear_groups(rows, d_out);
  if (groups < kLinearGroups / 2) {
    long long want = kLinearGroups / groups;
    if (want > kMostSplits) want = kMostSplits;
    const size_t room = given > l.partial ? (given / 256 * 256 - l.partial) / ((size_t)rows * d_out * 4) : 0;
    if ((unsigned long long)want > room) want = (long long)room;
    if (want > slabs / 2) want = slabs / 2;
    if (want < 1) want = 1;
    const int per = (int)((slabs + want - 1) / want);
    l.splits = (slabs + per - 1) / per;
  }
  if (l.splits > 1) l.total = align(l.partial + (size_t)l.splits * rows * d_out * 4);
  return l;
}
// The most that a call of up to `rows` rows takes: more rows are more workgroups, and may take fewer ranges and less.
inline size_t linear_scratch_upto(int act, int rows, int d_in, int d_out) {
  size_t most = linear_scratch(act, rows, d_in, d_out).total;
  for (int r = kTileM; r < rows && linear_groups(r, d_out) < kLinearGroups / 2; r += kTileM) {
    const size_t bytes = linear_scratch(act, r, d_in, d_out).total;
    if (bytes > most) most = bytes;
  }
  return most;
}
hipError_t launch_linear_pack(const void* w, const void* scales, void* packed, float* factor, int d_in, int d_out,
                              hipStream_t s);
hipError_t launch_linear(int act, const LinearArgs& a, hipStream_t s);

}  // namespace pik
