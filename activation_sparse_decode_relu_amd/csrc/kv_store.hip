// Storing tokens in the attention cache and reading them back.
//
// One workgroup of 2 D threads takes one block (32 tokens) of one head, K and V together: a thread holds
// 16 elements of each, so a block's largest magnitude is one reduction and nobody else touches its
// exponent.  A block that held tokens before is decoded, joined with the new ones and rounded to the new
// exponent in the same pass.  Both operators only move bytes.
#include "kv_device.h"

namespace pik {

namespace {

// A value as it is stored: infinities become the type's largest finite value, NaN zero.
template <int ACT>
__device__ __forceinline__ float stored(float x) {
  const float c = fminf(fmaxf(x, -ActT<ACT>::kMax), ActT<ACT>::kMax);
  return x == x ? c : 0.0f;
}

template <int CODE>
__device__ __forceinline__ void decode16(const u32x4& w, float (&x)[16]) {
  const unsigned ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f16x2 lo, hi;
    decode4<CODE>(ws[q], lo, hi);
    x[4 * q] = (float)lo.x;
    x[4 * q + 1] = (float)lo.y;
    x[4 * q + 2] = (float)hi.x;
    x[4 * q + 3] = (float)hi.y;
  }
}

template <int CODE>
__device__ __forceinline__ u32x4 encode16(const float (&x)[16], float mul) {
  u32x4 w;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    w[q] = encode4<CODE>(x[4 * q] * mul, x[4 * q + 1] * mul, x[4 * q + 2] * mul, x[4 * q + 3] * mul);
  return w;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 1; m < WAVE; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// Thread t's 16 elements of a K block: one token, 16 dims.
template <int D> struct KPlace {
  int u, chunk, at;
  __device__ __forceinline__ explicit KPlace(int t)
      : u(t / (D / 16)), chunk(t % (D / 16)), at((k_half(u) * (D / 16) + chunk) * 256 + k_row(u) * 16) {}
};

// Thread t's 16 elements of a V block: eight tokens from 8 g, two dims 16 apart.
struct VPlace {
  int g, dim, at;
  __device__ __forceinline__ explicit VPlace(int t) : g((t >> 4) & 3), dim((t >> 6) * 32 + (t & 15)), at(t * 16) {}
};

template <int ACT, int CODE, int D>
__global__ __launch_bounds__(2 * D) void k_kv_append(const KvStoreArgs A) {
  using T = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  constexpr int NWV = 2 * D / WAVE;
  __shared__ float s_max[2][NWV];
  const KvView& c = A.c;
  const int tid = threadIdx.x, head = blockIdx.x % c.kv_heads;
  int local;
  const int i = slot_owner(c, blockIdx.x / c.kv_heads, 1, kKvBlock, 2, local);
  const KvSeq s = kv_seq(c, i);
  const int before = s.len - s.rows;                     // tokens held earlier
  const int block = max(before, 0) / kKvBlock + local;
  if (s.rows == 0 || block * kKvBlock >= s.len) return;
  const int page = kv_page(c, s.seq, block);
  if (page < 0) return;
  const size_t at = block_at(c, page, head, block % c.page_blocks);
  const bool has_old = block * kKvBlock < before;
  const KPlace<D> kp(tid);
  const VPlace vp(tid);

  // the new tokens (zero elsewhere)
  float x[16], y[16];
  {
    const int pos = block * kKvBlock + kp.u;
    const bool fresh = pos >= before && pos < s.len;
    const T* p = static_cast<const T*>(A.k.data) + (int64_t)(s.row0 + (fresh ? pos - before : 0)) * A.k.token +
                 head * A.k.head + kp.chunk * 16;
    V8 a = {}, b = {};
    if (fresh) {
      a = *reinterpret_cast<const V8*>(p);
      b = *reinterpret_cast<const V8*>(p + 8);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = stored<ACT>((float)a[e]);
      x[8 + e] = stored<ACT>((float)b[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int pos = block * kKvBlock + 8 * vp.g + e;
    const bool fresh = pos >= before && pos < s.len;
    const T* p = static_cast<const T*>(A.v.data) + (int64_t)(s.row0 + (fresh ? pos - before : 0)) * A.v.token +
                 head * A.v.head + vp.dim;
    y[e] = fresh ? stored<ACT>((float)p[0]) : 0.0f;
    y[8 + e] = fresh ? stored<ACT>((float)p[16]) : 0.0f;
  }
  float mx = 0.0f, my = 0.0f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    mx = fmaxf(mx, fabsf(x[e]));
    my = fmaxf(my, fabsf(y[e]));
  }
  mx = wave_max(mx);
  my = wave_max(my);
  if ((tid & (WAVE - 1)) == 0) {
    s_max[0][tid / WAVE] = mx;
    s_max[1][tid / WAVE] = my;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NWV; ++w) {
    mx = fmaxf(mx, s_max[0][w]);
    my = fmaxf(my, s_max[1][w]);
  }
  int ek = block_exponent<CODE>(mx), ev = block_exponent<CODE>(my);

  u32x4* kb = reinterpret_cast<u32x4*>(c.k + at * (kKvBlock * D) + kp.at);
  u32x4* vb = reinterpret_cast<u32x4*>(c.v + at * (kKvBlock * D) + vp.at);
  if (has_old) {   // the whole workgroup: its tokens' codes at the exponents they have
    const int ok = (int)c.k_exp[at] - 127, ov = (int)c.v_exp[at] - 127;
    float o[16];
    decode16<CODE>(*kb, o);
    const float fk = pow2i(min(max(ok, -126), 127));
    if (block * kKvBlock + kp.u < before) {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = o[e] * fk;
    }
    decode16<CODE>(*vb, o);
    const float fv = pow2i(min(max(ov, -126), 127));
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (block * kKvBlock + 8 * vp.g + e < before) {
        y[e] = o[e] * fv;
        y[8 + e] = o[8 + e] * fv;
      }
    ek = max(ek, ok);
    ev = max(ev, ov);
    __syncthreads();   // every thread has read the old exponents
  }
  *kb = encode16<CODE>(x, pow2i(-ek));
  *vb = encode16<CODE>(y, pow2i(-ev));
  if (tid == 0) {
    c.k_exp[at] = (uint8_t)(ek + 127);
    c.v_exp[at] = (uint8_t)(ev + 127);
  }
}

template <int ACT, int CODE, int D>
__global__ __launch_bounds__(2 * D) void k_kv_read(const KvStoreArgs A) {
  using T = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  const KvView& c = A.c;
  const int tid = threadIdx.x, head = blockIdx.x % c.kv_heads;
  int local;
  const int i = slot_owner(c, blockIdx.x / c.kv_heads, 1, kKvBlock, 2, local);
  const KvSeq s = kv_seq(c, i);
  const int first = A.first != nullptr ? min(A.first[i], 1 << 30) : 0;   // past any sequence's end all is 0
  // blocks are counted from the one that holds token `first`; tokens below 0 have no block
  const int lo = max(first, 0), block = lo / kKvBlock + local;
  const long long end = (long long)first + s.rows;      // past the last token asked for
  if (s.rows == 0 || (long long)block * kKvBlock >= end) return;
  const int page = block * kKvBlock < s.len ? kv_page(c, s.seq, block) : -1;
  const size_t at = page >= 0 ? block_at(c, page, head, block % c.page_blocks) : 0;
  const KPlace<D> kp(tid);
  const VPlace vp(tid);
  float x[16], y[16];
  u32x4 wk = {0, 0, 0, 0}, wv = {0, 0, 0, 0};
  float fk = 0.0f, fv = 0.0f;
  if (page >= 0) {
    wk = *reinterpret_cast<const u32x4*>(c.k + at * (kKvBlock * D) + kp.at);
    wv = *reinterpret_cast<const u32x4*>(c.v + at * (kKvBlock * D) + vp.at);
    fk = pow2i(max((int)c.k_exp[at] - 127, -126));
    fv = pow2i(max((int)c.v_exp[at] - 127, -126));
  }
  decode16<CODE>(wk, x);
  decode16<CODE>(wv, y);
  constexpr float kMax = ActT<ACT>::kMax;
  {
    const int pos = block * kKvBlock + kp.u;
    if (pos >= first && pos < end) {
      const bool held = page >= 0 && pos < s.len;
      V8 a, b;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = held ? (T)fminf(fmaxf(x[e] * fk, -kMax), kMax) : (T)0.0f;
        b[e] = held ? (T)fminf(fmaxf(x[8 + e] * fk, -kMax), kMax) : (T)0.0f;
      }
      T* p = static_cast<T*>(A.k.data) + (int64_t)(s.row0 + (pos - first)) * A.k.token + head * A.k.head + kp.chunk * 16;
      *reinterpret_cast<V8*>(p) = a;
      *reinterpret_cast<V8*>(p + 8) = b;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int pos = block * kKvBlock + 8 * vp.g + e;
    if (pos >= first && pos < end) {
      const bool held = page >= 0 && pos < s.len;
      T* p = static_cast<T*>(A.v.data) + (int64_t)(s.row0 + (pos - first)) * A.v.token + head * A.v.head + vp.dim;
      p[0] = held ? (T)fminf(fmaxf(y[e] * fv, -kMax), kMax) : (T)0.0f;
      p[16] = held ? (T)fminf(fmaxf(y[8 + e] * fv, -kMax), kMax) : (T)0.0f;
    }
  }
}

template <int ACT, int CODE, int D>
hipError_t store_go(const KvStoreArgs& a, bool read, hipStream_t s) {
  const size_t grid = ((size_t)a.c.rows / kKvBlock + 2 * (size_t)a.c.n) * a.c.kv_heads;
  if (grid > 0x7fffffffu) return hipErrorInvalidValue;
  if (read)
    hipLaunchKernelGGL((k_kv_read<ACT, CODE, D>), dim3((unsigned)grid), dim3(2 * D), 0, s, a);
  else
    hipLaunchKernelGGL((k_kv_append<ACT, CODE, D>), dim3((unsigned)grid), dim3(2 * D), 0, s, a);
  return hipGetLastError();
}

hipError_t store_any(int act, int code, const KvStoreArgs& a, bool read, hipStream_t s) {
  const bool wide = a.c.dim == 128;
  if (a.c.dim != 64 && a.c.dim != 128) return hipErrorInvalidValue;
  if (act == ACT_F16 && code == CODE_E4M3)
    return wide ? store_go<ACT_F16, CODE_E4M3, 128>(a, read, s) : store_go<ACT_F16, CODE_E4M3, 64>(a, read, s);
  if (act == ACT_F16 && code == CODE_INT8)
    return wide ? store_go<ACT_F16, CODE_INT8, 128>(a, read, s) : store_go<ACT_F16, CODE_INT8, 64>(a, read, s);
  if (act == ACT_BF16 && code == CODE_E4M3)
    return wide ? store_go<ACT_BF16, CODE_E4M3, 128>(a, read, s) : store_go<ACT_BF16, CODE_E4M3, 64>(a, read, s);
  if (act == ACT_BF16 && code == CODE_INT8)
    return wide ? store_go<ACT_BF16, CODE_INT8, 128>(a, read, s) : store_go<ACT_BF16, CODE_INT8, 64>(a, read, s);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_kv_append(int act, int code, const KvStoreArgs& a, hipStream_t s) {
  return store_any(act, code, a, false, s);
}

hipError_t launch_kv_read(int act, int code, const KvStoreArgs& a, hipStream_t s) {
  return store_any(act, code, a, true, s);
}

}  // namespace pik
