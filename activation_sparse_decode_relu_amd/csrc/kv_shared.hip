// Attention of sequences whose caches begin with the same pages: the shared tokens once for all rows of a group, what
// each sequence holds behind them, and how many are shared.
//
// Two launches of the kernels of kv_step.h and kv_tile.h, each by its own number of rows.  The first takes groups as
// items, all of a group's rows over its shared blocks, with no mask since every row stands behind them, and leaves each
// row's O' and state (fp32) in the caller's scratch, in several parts where many rows' tokens are split.  The second takes
// the sequences from their first own block on, and joins that with the states where it would store its rows.  Parts are
// joined there too while it has up to 32 rows of a cached head (two layers of 64 sequences on 4096 shared tokens: 108 us,
// 116 with a launch between the two); where it has more, a lane's rows lie far apart, and a launch of its own joins them
// (two layers of 2 x 4 sequences, 80 rows of a head, on 20000: 174 us; 212 without, where the first launch took 9 us more).
//
// The first launch is bound as its kernel is: by the vector ALU and the matrix instructions for many rows (4 sequences, 4
// tokens each, 128 heads on 8 of 64 dims in int8, on 100003 tokens: 97 us, their products alone 45 at a library product's
// rate), by latency for few.  The second is bound by reading codes and states, and at its start and end (64 sequences of 30
// to 800 own tokens, 8 heads of 128: 20 to 23 us for 54 MB of codes and 31 of states).
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

// One workgroup for 256 / (D / 4) heads of a row: the parts of its states, in their order, become the first.
template <int D>
__global__ __launch_bounds__(256) void k_kv_state_join(const KvSharedArgs A) {
  static_assert(WAVE % (D / 4) == 0, "a row's head is one wave's: its state is read before it is replaced");
  const int across = (A.heads * (D / 4) + 255) / 256, row = blockIdx.x / across;
  int local;
  const int i = slot_owner(A.c, row, 1, 1, 0, local);
  const KvSeq s = kv_seq(A.c, i);
  if (row < s.row0 || row >= s.row0 + s.rows) return;
  const int shared = shared_of(A, A.n_groups + i), parts = shared > 0 ? parts_of(A, shared) : 0;
  if (parts < 2) return;
  const int k = (int)(blockIdx.x % across) * 256 + threadIdx.x, head = k / (D / 4), d = 4 * (k % (D / 4));
  if (head >= A.heads) return;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  RowState a{-INFINITY, -INFINITY, 0.0f};
  join_state<D>(A, parts, row, head, d, v, a);
  put_state<D>(A, 0, row, head, d, v, a);
}

}  // namespace

hipError_t launch_kv_state_join(const KvSharedArgs& a, hipStream_t s) {
  const long long grid = (long long)a.c.rows * ((a.heads * (a.c.dim / 4) + 255) / 256);
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  if (a.c.dim == 128)
    hipLaunchKernelGGL((k_kv_state_join<128>), dim3((unsigned)grid), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_kv_state_join<64>), dim3((unsigned)grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

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
