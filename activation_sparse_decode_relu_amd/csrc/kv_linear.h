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
};

hipError_t launch_linear_pack(int act, const void* w, const void* scales, void* packed, float* factor, int d_in, int d_out,
                              hipStream_t s);
hipError_t launch_linear(int act, const LinearArgs& a, hipStream_t s);

}  // namespace pik
