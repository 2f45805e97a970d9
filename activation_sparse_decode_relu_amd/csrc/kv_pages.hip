// Freeing, forking, growing and compacting sequences: table, lengths and reference counts, and the
// copies of pages.
//
// Everything is decided on the device, so no call waits for the host and all can stand in a graph.  Who
// gets which page has to follow one order (the lowest free page first, in the order of the call), which is
// a prefix sum over the pool; one workgroup makes it, reading 4 reference counts a thread and stopping
// when it has found enough, and leaves the list of copies to a second launch over the whole chip.  The first
// is bound by loads that wait for each other (32 sequences with a token each, half of them forks: 7.8 us), the
// second by copying: a page is read and written once, in 16-byte units.
#include "kv_device.h"
#include "kernels_impl.h"

namespace pik {

namespace {

constexpr int kPlan = 1024;      // threads of the deciding workgroup
constexpr int kCopyUnits = 4;    // 16-byte units a thread has in flight
constexpr int kCopyGroups = 2048;   // workgroups of a copying launch: 8 a compute unit

__global__ __launch_bounds__(256) void k_kv_free(const KvPool P, const int* __restrict__ seqs) {
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= P.max_seqs) return;
  int* row = P.table + (size_t)s * P.max_pages;
  for (int j = threadIdx.x; j < P.max_pages; j += blockDim.x) {
    const int p = atomicExch(row + j, -1);
    if (p >= 0 && p < P.pages) atomicSub(P.refs + p, 1);
  }
  if (threadIdx.x == 0) {
    P.lens[s] = 0;
    P.refused[s] = 0;
  }
}

__global__ __launch_bounds__(256) void k_kv_fork(const KvPool P, const int* __restrict__ srcs,
                                                 const int* __restrict__ dsts) {
  const int a = srcs[blockIdx.x], b = dsts[blockIdx.x];
  if (a < 0 || a >= P.max_seqs || b < 0 || b >= P.max_seqs || a == b) return;
  const int* from = P.table + (size_t)a * P.max_pages;
  int* to = P.table + (size_t)b * P.max_pages;
  for (int j = threadIdx.x; j < P.max_pages; j += blockDim.x) {
    const int p = from[j];
    to[j] = p;
    if (p >= 0 && p < P.pages) atomicAdd(P.refs + p, 1);
  }
  if (threadIdx.x == 0) {
    P.lens[b] = P.lens[a];
    P.refused[b] = P.refused[a];
  }
}

// What one sequence of a reserve call needs.
struct Need {
  int s = 0, count = 0, len = 0, end = 0, have = 0, cols = 0;   // cols: the columns from `have` on that it grows into
  int pages = 0;        // new ones, a copy's among them; -1: cannot grow
  int shared = -1;      // the last page, if it has to be copied, else -1
};

// A column past a sequence's length may still name a page (a caller has lowered the length): one that no other entry
// names is used again.
__device__ __forceinline__ bool keeps(const KvPool& P, int page) {
  return page >= 0 && page < P.pages && P.refs[page] == 1;
}

// All but what such columns save.
__device__ __forceinline__ Need need_of(const KvPool& P, const int* seqs, const int* counts, int i) {
  Need r;
  r.s = seqs[i];
  r.pages = -1;
  const int c = r.count = counts[i];
  if (r.s < 0 || r.s >= P.max_seqs) return r;
  r.len = P.lens[r.s];
  if (r.len < 0 || c < 0) return r;
  const long long end = (long long)r.len + c;
  if (end > (long long)P.max_pages * P.page_tokens) return r;
  r.end = (int)end;
  r.have = (r.len + P.page_tokens - 1) / P.page_tokens;
  r.cols = (r.end + P.page_tokens - 1) / P.page_tokens - r.have;
  if (c > 0 && r.len % P.page_tokens != 0) {
    const int last = P.table[(size_t)r.s * P.max_pages + r.have - 1];
    if (last < 0 || last >= P.pages) return r;
    if (P.refs[last] > 1) r.shared = last;
  }
  // the columns of a row name no more pages than there are; one too many is as good as any number that cannot be had,
  // and keeps the call's sum in 32 bits
  r.pages = min(r.cols, P.pages + 1) + (r.shared >= 0 ? 1 : 0);
  return r;
}

// The needs of sequences base .. base + kPlan, one a thread, by the whole workgroup.  The columns are looked through by
// a wave for each sequence (a thread for each took 26 us for the 128 of one prompt); sets `named` where any names a page.
__device__ Need needs_of(const KvPool& P, const int* seqs, const int* counts, int n, int base, int* named) {
  __shared__ int s_cols[kPlan], s_kept[kPlan];
  __shared__ long long s_row[kPlan];
  const int tid = threadIdx.x, lane = tid & (WAVE - 1), i = base + tid;
  Need r = i < n ? need_of(P, seqs, counts, i) : Need{};
  const bool look = r.cols > 0 && r.pages >= 0 && r.pages <= P.pages;
  if (!__syncthreads_or(look)) return r;
  s_cols[tid] = look ? r.cols : 0;
  s_row[tid] = (long long)r.s * P.max_pages + r.have;
  s_kept[tid] = 0;
  __syncthreads();
  const int most = min(n - base, kPlan);
  for (int q = tid / WAVE; q < most; q += kPlan / WAVE) {
    const int cols = s_cols[q];
    const int* row = P.table + s_row[q];
    int kept = 0;
#pragma unroll 4
    for (int j = lane; j < cols; j += WAVE) {
      const int page = row[j];
      if (page >= 0) {
        *named = 1;
        kept += keeps(P, page) ? 1 : 0;
      }
    }
    if (kept > 0) atomicAdd(&s_kept[q], kept);
  }
  __syncthreads();
  r.pages -= s_kept[tid];
  return r;
}

// Writes list[0 .. found): the lowest `want` pages that are free.  Returns found <= want.
__device__ int list_free(const KvPool& P, int want) {
  int found = 0;
  for (int base = 0; base < P.pages && found < want; base += 4 * kPlan) {
    const int p0 = base + 4 * (int)threadIdx.x;
    bool f[4];
    int mine = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = p0 + e < P.pages && P.refs[p0 + e] <= 0;
      mine += f[e] ? 1 : 0;
    }
    int total;
    int at = found + block_exclusive_scan<kPlan>(mine, &total);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (f[e]) {
        if (at < want) P.list[at] = p0 + e;
        ++at;
      }
    found += total;
  }
  return min(found, want);
}

__global__ __launch_bounds__(kPlan) void k_kv_reserve(const KvPool P, const int* __restrict__ seqs,
                                                      const int* __restrict__ counts, int n) {
  __shared__ int s_failed, s_given, s_named;
  const int tid = threadIdx.x;
  if (tid == 0) s_failed = s_given = s_named = 0;
  __syncthreads();
  // how many pages the call wants in all
  int want = 0;
  Need mine;                             // of the first kPlan sequences: seldom are there more
  for (int base = 0; base < n; base += kPlan) {
    const Need r = needs_of(P, seqs, counts, n, base, &s_named);
    if (base == 0) mine = r;
    int total;
    block_exclusive_scan<kPlan>(max(r.pages, 0), &total);
    want = min(want + total, P.pages + 1);   // more than there are is as good as one too many
  }
  const int found = list_free(P, want);
  __threadfence_block();
  __syncthreads();
  // Hand them out in order; what a sequence needs is worked out before anything of it changes, and shared pages keep
  // their counts until all have been looked at.  Where columns name pages already, all pages do.
  const bool named = s_named != 0;
  int given = 0;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + tid;
    const Need r = base == 0 ? mine : needs_of(P, seqs, counts, n, base, &s_named);
    int total;
    const int at = given + block_exclusive_scan<kPlan>(max(r.pages, 0), &total);
    const bool grows = i < n && r.pages >= 0 && at + r.pages <= found;
    if (i < n && !grows) atomicAdd(&s_failed, 1);
    int from = -1, to = -1;
    if (grows) {
      int* row = P.table + (size_t)r.s * P.max_pages;
      int k = at, j = r.have;
      if (r.shared >= 0) {
        from = r.shared;
        to = P.list[k];
        row[r.have - 1] = to;
        if (named)
          P.drop[k] = -1;
        else
          P.refs[to] = 1;
        ++k;
      }
      if (named) {
        for (; k < at + r.pages && j < r.have + r.cols; ++j) {
          const int old = row[j];
          if (keeps(P, old)) continue;
          P.drop[k] = old >= 0 && old < P.pages && P.refs[old] > 1 ? old : -1;
          row[j] = P.list[k++];
        }
        atomicMax(&s_given, at + r.pages);
      } else {
        for (; k < at + r.pages; ++k, ++j) {
          const int p = P.list[k];
          row[j] = p;
          P.refs[p] = 1;
        }
      }
      P.lens[r.s] = r.end;
    }
    if (i < n) {
      P.src[i] = from;
      P.dst[i] = to;
      // see k_kv_append; a request for no tokens says nothing about those of another
      if (r.s >= 0 && r.s < P.max_seqs && r.count > 0) P.refused[r.s] = grows ? 0 : r.len + 1;
    }
    given = min(given + total, P.pages + 1);
  }
  __threadfence_block();
  __syncthreads();
  for (int i = tid; i < n; i += kPlan)
    if (P.src[i] >= 0) atomicSub(P.refs + P.src[i], 1);
  // those handed out are the first of the list: who comes after one that fails fails too
  for (int k = tid; named && k < s_given; k += kPlan) {
    const int taken = P.list[k], left = P.drop[k];
    P.refs[taken] = 1;
    if (left >= 0) atomicSub(P.refs + left, 1);
  }
  if (tid == 0) {
    *P.count = n;
    if (s_failed != 0) *P.failed += s_failed;
  }
}

// Copies page src[i] to dst[i], i < *count, in every layer: K, V and their exponents.  A workgroup takes
// pieces of 256 * kCopyUnits 16-byte units in turn.
__device__ void copy_pages(const KvPool& P, int n) {
  const int units = (int)(P.page_bytes / 16), piece = 256 * kCopyUnits;
  const int pieces = (units + piece - 1) / piece;
  const long long jobs = (long long)n * P.layers * 2 * pieces;
  for (long long job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int part = (int)(job % pieces);
    const long long rest = job / pieces;
    const bool is_v = rest & 1;
    const int layer = (int)((rest >> 1) % P.layers), i = (int)((rest >> 1) / P.layers);
    const int from = P.src[i], to = P.dst[i];
    if (from < 0 || to < 0) continue;
    const size_t a = (size_t)layer * P.pages + from, b = (size_t)layer * P.pages + to;
    uint8_t* codes = is_v ? P.v : P.k;
    const u32x4* src = reinterpret_cast<const u32x4*>(codes + a * P.page_bytes);
    u32x4* dst = reinterpret_cast<u32x4*>(codes + b * P.page_bytes);
    u32x4 t[kCopyUnits];
#pragma unroll
    for (int u = 0; u < kCopyUnits; ++u) {
      const int at = part * piece + u * 256 + (int)threadIdx.x;
      if (at < units) t[u] = ld_stream(src + at);
    }
#pragma unroll
    for (int u = 0; u < kCopyUnits; ++u) {
      const int at = part * piece + u * 256 + (int)threadIdx.x;
      if (at < units) __builtin_nontemporal_store(t[u], dst + at);
    }
    if (part == 0) {
      uint8_t* exps = is_v ? P.v_exp : P.k_exp;
      for (int e = threadIdx.x; e < P.exp_bytes; e += blockDim.x)
        exps[b * P.exp_bytes + e] = exps[a * P.exp_bytes + e];
    }
  }
}

__global__ __launch_bounds__(256) void k_kv_copy(const KvPool P) { copy_pages(P, *P.count); }

__global__ __launch_bounds__(kPlan) void k_kv_compact(const KvPool P) {
  const int tid = threadIdx.x;
  int mine = 0, live;
  for (int p = tid; p < P.pages; p += kPlan) mine += P.refs[p] > 0 ? 1 : 0;
  block_exclusive_scan<kPlan>(mine, &live);
  // ranks of the free pages below `live` and of the used ones above: as many of one as of the other
  int holes = 0, movers = 0;
  for (int base = 0; base < P.pages; base += 4 * kPlan) {
    const int p0 = base + 4 * tid;
    int nh = 0, nm = 0;
    bool h[4], m[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = p0 + e;
      const bool used = p < P.pages && P.refs[p] > 0;
      h[e] = p < live && !used;
      m[e] = p >= live && used;
      nh += h[e] ? 1 : 0;
      nm += m[e] ? 1 : 0;
    }
    int th, tm;
    int ah = holes + block_exclusive_scan<kPlan>(nh, &th);
    int am = movers + block_exclusive_scan<kPlan>(nm, &tm);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (h[e]) P.dst[ah++] = p0 + e;
      if (m[e]) P.src[am++] = p0 + e;
    }
    holes += th;
    movers += tm;
  }
  __threadfence_block();
  __syncthreads();
  for (int i = tid; i < movers; i += kPlan) {
    const int from = P.src[i], to = P.dst[i];
    P.list[from] = to;
    P.refs[to] = P.refs[from];
    P.refs[from] = 0;
  }
  if (tid == 0) {
    P.count[0] = movers;
    P.count[1] = live;
  }
}

// The copies, and the table's entries that name a page that moved (those at `live` and above).
__global__ __launch_bounds__(256) void k_kv_move(const KvPool P) {
  const int live = P.count[1];
  if (P.count[0] == 0) return;
  const long long entries = (long long)P.max_seqs * P.max_pages;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < entries;
       i += (long long)gridDim.x * blockDim.x) {
    const int p = P.table[i];
    if (p >= live && p < P.pages) P.table[i] = P.list[p];
  }
  copy_pages(P, P.count[0]);
}

}  // namespace

hipError_t launch_kv_free(const KvPool& p, const int* seqs, int n, hipStream_t s) {
  hipLaunchKernelGGL(k_kv_free, dim3(n), dim3(256), 0, s, p, seqs);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const KvPool& p, const int* src, const int* dst, int n, hipStream_t s) {
  hipLaunchKernelGGL(k_kv_fork, dim3(n), dim3(256), 0, s, p, src, dst);
  return hipGetLastError();
}

hipError_t launch_kv_reserve(const KvPool& p, const int* seqs, const int* counts, int n, hipStream_t s) {
  hipLaunchKernelGGL(k_kv_reserve, dim3(1), dim3(kPlan), 0, s, p, seqs, counts, n);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_kv_copy, dim3(kCopyGroups), dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const KvPool& p, hipStream_t s) {
  hipLaunchKernelGGL(k_kv_compact, dim3(1), dim3(kPlan), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_kv_move, dim3(kCopyGroups), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace pik
