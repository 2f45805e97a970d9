// Attention of sequences whose caches begin with the same pages: the shared tokens once for all rows of a group, what
// each sequence holds behind them, and how many are shared.
//
// Two launches of the kernels of kv_step.h and kv_tile.h, each by its own number of rows.  The first takes groups as
// items, all of a group's rows over its shared blocks, with no mask since every row stands behind them, and leaves each
// row's O' and state (fp32) in the caller's scratch.  The second takes the sequences from their first own block
// on, and joins that with the states where it would store its rows.
#include "kv_step.h"
#include "kv_tile.h"

namespace pik {

namespace {

constexpr int kShareThreads = 1024;

// One workgroup a group: the leading columns of the table that name the same page for all of its sequences, up to the
// tokens that every one of them held before this call's.
__global__ __launch_bounds__(kShareThreads) void k_kv_share(const KvShareArgs A) {
  __shared__ int s_limit, s_cols;
  const KvView& c = A.c;
  const int tid = threadIdx.x, g = blockIdx.x;
  const int g0 = group_at(A.groups, g, c.n), g1 = max(group_at(A.groups, g + 1, c.n), g0), members = g1 - g0;
  if (tid == 0) s_limit = s_cols = 0x7fffffff;
  __syncthreads();
  for (int i = g0 + tid; i < g1; i += kShareThreads) {
    const KvSeq s = kv_seq(c, i);
    atomicMin(&s_limit, max(s.len - s.rows, 0));
  }
  __syncthreads();
  const int page_tokens = c.page_blocks * kKvBlock, limit = members > 1 ? s_limit : 0;
  const int cols = (limit + page_tokens - 1) / page_tokens;   // none where a sequence is out of range: it holds nothing
  if (cols > 0) {
    const int* first = c.table + (size_t)c.seqs[g0] * c.max_pages;
    int differ = cols;
    // a wave takes 64 columns of a sequence at a time
    const int chunks = (cols + WAVE - 1) / WAVE;
    for (int k = tid / WAVE; k < chunks * members; k += kShareThreads / WAVE) {
      const int m = k % members, j = k / members * WAVE + tid % WAVE;
      if (j >= cols) continue;
      const int p = first[j], q = c.table[(size_t)c.seqs[g0 + m] * c.max_pages + j];
      if (p != q || p < 0 || p >= c.pages) differ = min(differ, j);
    }
    if (differ < cols) atomicMin(&s_cols, differ);
  }
  __syncthreads();
  const int shared = (int)min((long long)limit, (long long)min(s_cols, cols) * page_tokens) & ~(kKvBlock - 1);
  if (tid == 0) A.plan[g] = shared;
  // sequences before the first group and behind the last share nothing
  for (int i = (g == 0 ? 0 : g0) + tid; i < (g == A.n_groups - 1 ? c.n : g1); i += kShareThreads)
    A.plan[A.n_groups + i] = i >= g0 && i < g1 ? shared : 0;
}

}  // namespace

hipError_t launch_kv_share(const KvShareArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_kv_share, dim3((unsigned)a.n_groups), dim3(kShareThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_step_shared(int act, int code, int mode, const KvSharedArgs& a, hipStream_t s) {
  return mode == ATTEND_SHARED ? step_act<ATTEND_SHARED>(act, code, a, s) : step_act<ATTEND_OWN>(act, code, a, s);
}

hipError_t launch_kv_tile_shared(int act, int code, int mode, const KvSharedArgs& a, hipStream_t s) {
  return mode == ATTEND_SHARED ? tile_act<ATTEND_SHARED>(act, code, a, s) : tile_act<ATTEND_OWN>(act, code, a, s);
}

}  // namespace pik
