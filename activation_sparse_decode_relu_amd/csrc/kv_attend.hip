// Attention over the cache.
#include "kv_device.h"

namespace pik {

namespace {

// One wave a row and head: 32 tokens at a time, a lane taking half the dims of one token's score, then
// D / 64 dims of the output.
template <int ACT, int CODE, int D>
__global__ __launch_bounds__(WAVE) void k_kv_attend(const KvAttendArgs A) {
  using T = typename ActT<ACT>::T;
  const KvView& c = A.c;
  const int lane = threadIdx.x, h = blockIdx.y, kvh = h / A.group;
  int local;
  const int i = slot_owner(c, blockIdx.x, 1, 1, 1, local);
  const KvSeq s = kv_seq(c, i);
  if (local >= s.rows) return;
  const int row = s.row0 + local, pos = s.len - s.rows + local;
  const T* q = static_cast<const T*>(A.q.data) + row * A.q.token + h * A.q.head;
  __shared__ float s_q[D], s_p[kKvBlock];
  for (int e = lane; e < D; e += WAVE) s_q[e] = (float)q[e];
  __syncthreads();
  float m = -INFINITY, l = 0.0f, o[D / WAVE] = {};
  const int u = lane & 31, half = lane >> 5;
  for (int b = 0; b * kKvBlock <= pos; ++b) {
    const int page = kv_page(c, s.seq, b);
    if (page < 0) continue;
    const size_t at = block_at(c, page, kvh, b % c.page_blocks);
    const uint8_t* kb = c.k + at * (kKvBlock * D);
    const uint8_t* vb = c.v + at * (kKvBlock * D);
    float x = 0.0f;
    for (int ch = half * (D / 32); ch < (half + 1) * (D / 32); ++ch) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(kb + (k_half(u) * (D / 16) + ch) * 256 + k_row(u) * 16);
      for (int e = 0; e < 4; ++e) {
        f16x2 lo, hi;
        decode4<CODE>(w[e], lo, hi);
        const float* sq = s_q + ch * 16 + e * 4;
        x += sq[0] * (float)lo.x + sq[1] * (float)lo.y + sq[2] * (float)hi.x + sq[3] * (float)hi.y;
      }
    }
    x += __shfl_xor(x, 32);
    x *= A.scale * pow2i(max((int)c.k_exp[at] - 127, -126));
    const int tok = b * kKvBlock + u;
    const bool seen = tok <= pos && (A.window == 0 || tok > pos - A.window || tok < A.sinks);
    if (!seen) x = -INFINITY;
    float mb = x;
    for (int k = 1; k < 32; k <<= 1) mb = fmaxf(mb, __shfl_xor(mb, k));
    const float mn = fmaxf(m, mb);
    if (mn == -INFINITY) continue;
    const float p = expf(x - mn), f = expf(m - mn);
    float sum = p;
    for (int k = 1; k < 32; k <<= 1) sum += __shfl_xor(sum, k);
    l = l * f + sum;
    m = mn;
    __syncthreads();
    if (lane < 32) s_p[lane] = p;
    __syncthreads();
    const float ev = pow2i(max((int)c.v_exp[at] - 127, -126));
    for (int d = 0; d < D / WAVE; ++d) {
      const int dim = d * WAVE + lane;
      float acc = 0.0f;
      for (int t = 0; t < kKvBlock; t += 4) {
        const unsigned w = *reinterpret_cast<const unsigned*>(vb + (dim / 32) * 1024 + (16 * (t / 8) + dim % 16) * 16 +
                                                              8 * ((dim / 16) % 2) + t % 8);
        f16x2 lo, hi;
        decode4<CODE>(w, lo, hi);
        const float v[4] = {(float)lo.x, (float)lo.y, (float)hi.x, (float)hi.y};
        for (int e = 0; e < 4; ++e)
          if (b * kKvBlock + t + e < s.len) acc += s_p[t + e] * v[e];
      }
      o[d] = o[d] * f + acc * ev;
    }
  }
  T* out = static_cast<T*>(A.out.data) + row * A.out.token + h * A.out.head;
  for (int d = 0; d < D / WAVE; ++d) out[d * WAVE + lane] = (T)(l > 0.0f ? o[d] / l : 0.0f);
  if (A.lse != nullptr && lane == 0) A.lse[(size_t)row * A.heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

template <int ACT, int CODE, int D>
hipError_t attend_go(const KvAttendArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_kv_attend<ACT, CODE, D>), dim3(a.c.rows + a.c.n, a.heads), dim3(WAVE), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_attend(int act, int code, const KvAttendArgs& a, hipStream_t s) {
  const bool wide = a.c.dim == 128;
  if (act == ACT_F16 && code == CODE_E4M3)
    return wide ? attend_go<ACT_F16, CODE_E4M3, 128>(a, s) : attend_go<ACT_F16, CODE_E4M3, 64>(a, s);
  if (act == ACT_F16 && code == CODE_INT8)
    return wide ? attend_go<ACT_F16, CODE_INT8, 128>(a, s) : attend_go<ACT_F16, CODE_INT8, 64>(a, s);
  if (act == ACT_BF16 && code == CODE_E4M3)
    return wide ? attend_go<ACT_BF16, CODE_E4M3, 128>(a, s) : attend_go<ACT_BF16, CODE_E4M3, 64>(a, s);
  return wide ? attend_go<ACT_BF16, CODE_INT8, 128>(a, s) : attend_go<ACT_BF16, CODE_INT8, 64>(a, s);
}

}  // namespace pik
