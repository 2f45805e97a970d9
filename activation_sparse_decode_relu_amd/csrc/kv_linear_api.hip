// C ABI of the products with 4-bit weights: argument checks and the kernels of each call.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <new>

#include "kv_linear.h"
#include "pi_linear.h"
#include "status.h"

namespace {

using pik::fail;
using pik::ok;

constexpr int kMaxIn = 1 << 20, kMaxOut = 1 << 24, kMaxRows = 1 << 24;
constexpr int kMaxStride = 1 << 23;   // 128 rows' offsets in bytes fit in 32 bits
constexpr uintptr_t kAlign = 256;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int tiles_of(const pi_linear_desc& d) { return (d.d_out + pik::kSlabRows - 1) / pik::kSlabRows; }
int slabs_of(const pi_linear_desc& d) { return (d.d_in + pik::kSlabCols - 1) / pik::kSlabCols; }
size_t slabs_bytes(const pi_linear_desc& d) { return (size_t)tiles_of(d) * slabs_of(d) * pik::kSlabBytes; }
size_t packed_of(const pi_linear_desc& d) { return slabs_bytes(d) + (size_t)tiles_of(d) * pik::kSlabRows * sizeof(float); }

pi_status check_desc(const pi_linear_desc* d) {
  if (d == nullptr) return fail(PI_ERR_INVALID, "desc is NULL");
  if (d->d_in < 32 || d->d_in > kMaxIn || d->d_in % 32 != 0)
    return fail(PI_ERR_INVALID, "d_in=%d must be a multiple of 32 up to 2^20", d->d_in);
  if (d->d_out < 1 || d->d_out > kMaxOut) return fail(PI_ERR_INVALID, "d_out=%d must lie in [1, 2^24]", d->d_out);
  if (d->act_dtype != PI_LINEAR_F16 && d->act_dtype != PI_LINEAR_BF16)
    return fail(PI_ERR_INVALID, "act_dtype=%d is not a pi_linear_act", d->act_dtype);
  return PI_OK;
}

}  // namespace

struct pi_linear {
  pi_linear_desc desc;
  const uint8_t* packed;
  const float* bias;

  const float* factor() const { return reinterpret_cast<const float*>(packed + slabs_bytes(desc)); }
};

extern "C" {

int32_t pi_linear_abi_version(void) { return PI_LINEAR_ABI_VERSION; }

pi_status pi_linear_packed_bytes(const pi_linear_desc* desc, size_t* bytes) {
  if (bytes == nullptr) return fail(PI_ERR_INVALID, "bytes is NULL");
  const pi_status st = check_desc(desc);
  if (st != PI_OK) return st;
  *bytes = packed_of(*desc);
  return ok();
}

pi_status pi_linear_create(const pi_linear_desc* desc, const void* w, const void* scales, const float* bias, void* packed,
                           size_t packed_bytes, void* stream, pi_linear** out) {
  if (out == nullptr) return fail(PI_ERR_INVALID, "out is NULL");
  *out = nullptr;
  const pi_status st = check_desc(desc);
  if (st != PI_OK) return st;
  if (w == nullptr || !aligned(w, 4)) return fail(PI_ERR_INVALID, "w is NULL or not 4-byte aligned");
  if (scales == nullptr || !aligned(scales, 2)) return fail(PI_ERR_INVALID, "scales is NULL or not 2-byte aligned");
  if (!aligned(bias, 4)) return fail(PI_ERR_INVALID, "bias is not 4-byte aligned");
  const size_t need = packed_of(*desc);
  if (packed == nullptr || !aligned(packed, kAlign) || packed_bytes < need)
    return fail(PI_ERR_WORKSPACE, "packed must be %zu bytes, %zu-byte aligned", need, (size_t)kAlign);
  pi_linear* h = new (std::nothrow) pi_linear{*desc, static_cast<const uint8_t*>(packed), bias};
  if (h == nullptr) return fail(PI_ERR_INVALID, "out of host memory");
  const hipError_t e = pik::launch_linear_pack(w, scales, packed, const_cast<float*>(h->factor()), desc->d_in,
                                               desc->d_out, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) {
    delete h;
    return fail(PI_ERR_HIP, "laying the weights out failed: %s", hipGetErrorString(e));
  }
  *out = h;
  return ok();
}

pi_status pi_linear_destroy(pi_linear* h) {
  if (h == nullptr) return fail(PI_ERR_INVALID, "handle is NULL");
  delete h;
  return ok();
}

pi_status pi_linear_scratch_bytes(const pi_linear* h, int32_t rows, size_t* bytes) {
  if (h == nullptr) return fail(PI_ERR_INVALID, "handle is NULL");
  if (bytes == nullptr) return fail(PI_ERR_INVALID, "bytes is NULL");
  if (rows < 0 || rows > kMaxRows) return fail(PI_ERR_INVALID, "rows=%d must lie in [0, %d]", rows, kMaxRows);
  *bytes = pik::linear_scratch(h->desc.act_dtype, rows, h->desc.d_in, h->desc.d_out).total;
  return ok();
}

pi_status pi_linear_scratch_bytes_upto(const pi_linear* h, int32_t rows, size_t* bytes) {
  if (h == nullptr) return fail(PI_ERR_INVALID, "handle is NULL");
  if (bytes == nullptr) return fail(PI_ERR_INVALID, "bytes is NULL");
  if (rows < 0 || rows > kMaxRows) return fail(PI_ERR_INVALID, "rows=%d must lie in [0, %d]", rows, kMaxRows);
  *bytes = pik::linear_scratch_upto(h->desc.act_dtype, rows, h->desc.d_in, h->desc.d_out);
  return ok();
}

pi_status pi_linear_forward(pi_linear* h, const pi_linear_args* args, void* stream) {
  if (h == nullptr) return fail(PI_ERR_INVALID, "handle is NULL");
  if (args == nullptr) return fail(PI_ERR_INVALID, "args is NULL");
  const pi_linear_desc& d = h->desc;
  if (args->rows < 0 || args->rows > kMaxRows) return fail(PI_ERR_INVALID, "rows=%d must lie in [0, %d]", args->rows, kMaxRows);
  if (args->rows == 0) return ok();
  if (args->x == nullptr || !aligned(args->x, 16)) return fail(PI_ERR_INVALID, "x is NULL or not 16-byte aligned");
  if (args->y == nullptr || !aligned(args->y, 2)) return fail(PI_ERR_INVALID, "y is NULL or not 2-byte aligned");
  if (!aligned(args->add, 2)) return fail(PI_ERR_INVALID, "add is not 2-byte aligned");
  if (args->rows > 1 && (args->x_stride < 0 || args->x_stride % 8 != 0 || args->x_stride > kMaxStride))
    return fail(PI_ERR_INVALID, "x_stride=%lld must be a multiple of 8 elements in [0, 2^23]", (long long)args->x_stride);
  if (args->rows > 1 && args->add != nullptr && args->add_stride < 0)
    return fail(PI_ERR_INVALID, "add_stride=%lld must not be negative", (long long)args->add_stride);
  if (args->rows > 1 && args->y_stride < d.d_out)
    return fail(PI_ERR_INVALID, "y_stride=%lld is less than d_out=%d", (long long)args->y_stride, d.d_out);
  const size_t given = args->scratch != nullptr ? args->scratch_bytes : 0;
  const size_t need = pik::linear_scratch(d.act_dtype, args->rows, d.d_in, d.d_out, given).total;
  if (need > 0 && (!aligned(args->scratch, 16) || given < need))
    return fail(PI_ERR_WORKSPACE, "scratch must be at least %zu bytes, 16-byte aligned",
                pik::linear_scratch(d.act_dtype, args->rows, d.d_in, d.d_out, 0).total);
  pik::LinearArgs a{};
  a.scratch = args->scratch;
  a.scratch_bytes = given;
  a.packed = h->packed;
  a.factor = h->factor();
  a.bias = h->bias;
  a.x = args->x;
  a.add = args->add;
  a.y = args->y;
  a.x_stride = args->rows > 1 ? args->x_stride : 0;
  a.add_stride = args->add_stride;
  a.y_stride = args->y_stride;
  a.rows = args->rows;
  a.d_in = d.d_in;
  a.d_out = d.d_out;
  a.tiles = tiles_of(d);
  a.slabs = slabs_of(d);
  const hipError_t e = pik::launch_linear(d.act_dtype, a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(PI_ERR_HIP, "linear launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"
