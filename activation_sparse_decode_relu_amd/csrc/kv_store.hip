// Storing tokens in the attention cache and reading them back.
//
// One workgroup of 2 D threads takes one block (32 tokens) of one head, K and V together: a thread holds 16 dims of a
// token of each, loaded and stored in whole 16-byte units, so a block's largest magnitude is one reduction and nobody
// else touches its exponent.  V's codes stand in memory with their tokens side by side; they change places in
// LDS.  A block that held tokens before is decoded, joined with the new ones and rounded to the new exponent
// in the same pass.  Both operators only move bytes: storing and reading back 14 thousand tokens of 32 heads, 722 MB,
// takes 82.6 + 70.2 us, 4.7 TB/s, where a plain copy reaches 4.9 (with V's elements loaded and stored one by
// one, 2 bytes each, 101.8 + 86.4).
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

// Thread t's 16 elements of a block: one token, 16 dims; `at` is their place among K's codes.
template <int D> struct Place {
  int u, chunk, at;
  __device__ __forceinline__ explicit Place(int t)
      : u(t / (D / 16)), chunk(t % (D / 16)), at((k_half(u) * (D / 16) + chunk) * 256 + k_row(u) * 16) {}
  // byte of dim 16 chunk + e in a V block as it lies in LDS: 16 bytes between its KBs keep a
  // wave's lanes on banks of their own
  __device__ __forceinline__ int v_byte(int e) const {
    return (chunk / 2) * 1040 + (16 * (u / 8) + e) * 16 + 8 * (chunk % 2) + u % 8;
  }
};
template <int D> constexpr int kVBytes = D / 32 * 1040;
// where the 16-byte unit t of a V block lies in LDS
__device__ __forceinline__ int v_unit(int t) { return (t / 64) * 1040 + (t % 64) * 16; }

template <int ACT>
__device__ __forceinline__ void load16(const typename ActT<ACT>::T* p, bool fresh, float (&x)[16]) {
  using V8 = typename ActT<ACT>::V8;
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

template <int ACT>
__device__ __forceinline__ void store16(typename ActT<ACT>::T* p, bool held, float mul, const float (&x)[16]) {
  using T = typename ActT<ACT>::T;
  using V8 = typename ActT<ACT>::V8;
  constexpr float kMax = ActT<ACT>::kMax;
  V8 a, b;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a[e] = held ? (T)fminf(fmaxf(x[e] * mul, -kMax), kMax) : (T)0.0f;
    b[e] = held ? (T)fminf(fmaxf(x[8 + e] * mul, -kMax), kMax) : (T)0.0f;
  }
  *reinterpret_cast<V8*>(p) = a;
  *reinterpret_cast<V8*>(p + 8) = b;
}

template <int ACT, int CODE, int D>
__global__ __launch_bounds__(2 * D) void k_kv_append(const KvStoreArgs A) {
  using T = typename ActT<ACT>::T;
  constexpr int NWV = 2 * D / WAVE;
  __shared__ float s_max[2][NWV];
  __shared__ __align__(16) uint8_t s_v[kVBytes<D>];
  const KvView& c = A.c;
  const int tid = threadIdx.x, head = blockIdx.x % c.kv_heads;
  int local;
  const int i = slot_owner(c, blockIdx.x / c.kv_heads, 1, kKvBlock, 2, local);
  const KvSeq s = kv_seq(c, i);
  const int before = s.len - s.rows;                     // tokens held earlier
  const int block = max(before, 0) / kKvBlock + local;
  // a sequence that reserve refused has no room for these: its last tokens are others, and stay
  const bool refused = s.seq >= 0 && A.refused[s.seq] == s.len + 1;
  if (s.rows == 0 || block * kKvBlock >= s.len || refused) return;
  const int page = kv_page(c, s.seq, block);
  if (page < 0) return;
  const size_t at = block_at(c, page, head, block % c.page_blocks);
  const bool has_old = block * kKvBlock < before;
  const Place<D> my_place(tid);
  const int pos = block * kKvBlock + my_place.u;

  // the new tokens (zero elsewhere)
  float x[16], y[16];
  const bool fresh = pos >= before && pos < s.len;
  const int64_t row = s.row0 + (fresh ? pos - before : 0);
  load16<ACT>(static_cast<const T*>(A.k.data) + row * A.k.token + head * A.k.head + my_place.chunk * 16, fresh, x);
  load16<ACT>(static_cast<const T*>(A.v.data) + row * A.v.token + head * A.v.head + my_place.chunk * 16, fresh, y);
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

  u32x4* kb = reinterpret_cast<u32x4*>(c.k + at * (kKvBlock * D) + my_place.at);
  u32x4* vb = reinterpret_cast<u32x4*>(c.v + at * (kKvBlock * D)) + tid;
  u32x4* v_lds = reinterpret_cast<u32x4*>(s_v + v_unit(tid));
  if (has_old) {   // the whole workgroup: its tokens' codes at the exponents they have
    const int ok = (int)c.k_exp[at] - 127, ov = (int)c.v_exp[at] - 127;
    const u32x4 k_old = *kb;
    *v_lds = *vb;
    __syncthreads();   // and every thread has read the old exponents
    if (pos < before) {
      float o[16];
      decode16<CODE>(k_old, o);
      const float fk = pow2i(min(max(ok, -126), 127)), fv = pow2i(min(max(ov, -126), 127));
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = o[e] * fk;
      u32x4 w;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        unsigned b = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) b |= (unsigned)s_v[my_place.v_byte(4 * q + e)] << (8 * e);
        w[q] = b;
      }
      decode16<CODE>(w, o);
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = o[e] * fv;
    }
    ek = max(ek, ok);
    ev = max(ev, ov);
    __syncthreads();   // the old codes have been read
  }
  *kb = encode16<CODE>(x, pow2i(-ek));
  const u32x4 w = encode16<CODE>(y, pow2i(-ev));
#pragma unroll
  for (int e = 0; e < 16; ++e) s_v[my_place.v_byte(e)] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
  __syncthreads();
  *vb = *v_lds;
  if (tid == 0) {
    c.k_exp[at] = (uint8_t)(ek + 127);
    c.v_exp[at] = (uint8_t)(ev + 127);
  }
}

template <int ACT, int CODE, int D>
__global__ __launch_bounds__(2 * D) void k_kv_read(const KvStoreArgs A) {
  using T = typename ActT<ACT>::T;
  __shared__ __align__(16) uint8_t s_v[kVBytes<D>];
  const KvView& c = A.c;
  const int tid = threadIdx.x, head = blockIdx.x % c.kv_heads;
  int local;
  const int i = slot_owner(c, blockIdx.x / c.kv_heads, 1, kKvBlock, 2, local);
  const KvSeq s = kv_seq(c, i);
  const int first = A.first != nullptr ? min(A.first[i], 1 << 30) : 0;   // past any sequence's end all is 0
  // blocks are counted from the one that holds token `first`, below token 0 too: what is not there reads as 0
  const int block = (first >> 5) + local;
  static_assert(kKvBlock == 1 << 5, "rounds down");
  const long long end = (long long)first + s.rows;      // past the last token asked for
  if (s.rows == 0 || (long long)block * kKvBlock >= end) return;
  const int page = block >= 0 && block * kKvBlock < s.len ? kv_page(c, s.seq, block) : -1;
  const size_t at = page >= 0 ? block_at(c, page, head, block % c.page_blocks) : 0;
  const Place<D> my_place(tid);
  float fk = 0.0f, fv = 0.0f;
  u32x4 wk = {0, 0, 0, 0}, wv = {0, 0, 0, 0};
  if (page >= 0) {
    wk = *reinterpret_cast<const u32x4*>(c.k + at * (kKvBlock * D) + my_place.at);
    *reinterpret_cast<u32x4*>(s_v + v_unit(tid)) = *(reinterpret_cast<const u32x4*>(c.v + at * (kKvBlock * D)) + tid);
    fk = pow2i(max((int)c.k_exp[at] - 127, -126));
    fv = pow2i(max((int)c.v_exp[at] - 127, -126));
  }
  __syncthreads();
  const int pos = block * kKvBlock + my_place.u;
  if (pos < first || pos >= end) return;
  const bool held = page >= 0 && pos < s.len;
  if (held) {
#pragma unroll
    for (int e = 0; e < 16; ++e) wv[e / 4] |= (unsigned)s_v[my_place.v_byte(e)] << (8 * (e % 4));
  }
  const int64_t row = s.row0 + (pos - first);
  float x[16];
  decode16<CODE>(wk, x);
  store16<ACT>(static_cast<T*>(A.k.data) + row * A.k.token + head * A.k.head + my_place.chunk * 16, held, fk, x);
  decode16<CODE>(wv, x);
  store16<ACT>(static_cast<T*>(A.v.data) + row * A.v.token + head * A.v.head + my_place.chunk * 16, held, fv, x);
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
