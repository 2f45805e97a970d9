// Host-side launch interface of the norms and rotation of queries and keys (internal to the library).
#pragma once

#include "kv.h"

namespace pik {

constexpr int kMaxPairs = 64;   // of a head of 128 dims

struct KvRotateArgs {
  KvView c;                // of it the sequences, the lengths and the sizes of the table
  KvRows q, q_out, k, k_out;
  const void* q_norm;      // [D] of the activations' type, or NULL
  const void* k_norm;
  const int* positions;    // [rows], or NULL: from the lengths
  int heads, rot;          // rot: dims that are turned
  float eps, gain;
  uint64_t turns[kMaxPairs];   // of each pair, for one position, in 2^-64 of a turn
};
hipError_t launch_kv_rotate(int act, int layout, const KvRotateArgs& a, hipStream_t s);

}  // namespace pik
