// C ABI of the attention cache: argument checks, workspace layout and the kernels of each call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "kernels.h"
#include "kv.h"
#include "pi_kv.h"
#include "status.h"

namespace {

using pik::fail;
using pik::ok;

constexpr size_t kAlign = 256;
constexpr int kMaxRows = 1 << 24;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

struct Layout {
  size_t tickets, count, src, dst, list, drop, partial, total;
};

Layout layout_for(const pi_kv_desc& d) {
  Layout L{};
  const size_t copies = (size_t)(d.pages > d.max_seqs ? d.pages : d.max_seqs);
  size_t off = 0;
  L.tickets = off; off = align_up(off + pik::kStepTickets * sizeof(unsigned));
  L.count = off; off = align_up(off + 2 * sizeof(int));
  L.src = off;   off = align_up(off + copies * sizeof(int));
  L.dst = off;   off = align_up(off + copies * sizeof(int));
  L.list = off;  off = align_up(off + (size_t)d.pages * sizeof(int));
  L.drop = off;  off = align_up(off + (size_t)d.pages * sizeof(int));
  L.partial = off; off = align_up(off + std::max(pik::step_partial_floats(d.head_dim),
                                              pik::tile_partial_floats(d.head_dim)) * sizeof(float));
  L.total = off;
  return L;
}

pi_status check_desc(const pi_kv_desc* d) {
  if (d == nullptr) return fail(PI_ERR_INVALID, "desc is NULL");
  if (d->kv_heads < 1 || d->heads < 1 || d->heads > 1024 || d->heads % d->kv_heads != 0)
    return fail(PI_ERR_INVALID, "heads=%d must be a multiple of kv_heads=%d, up to 1024", d->heads, d->kv_heads);
  if (d->head_dim < 1) return fail(PI_ERR_INVALID, "head_dim=%d must be positive", d->head_dim);
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(PI_ERR_UNSUPPORTED, "head_dim=%d: the kernels take 64 or 128", d->head_dim);
  if (d->page_tokens < 32 || d->page_tokens > 4096 || d->page_tokens % PI_KV_BLOCK != 0)
    return fail(PI_ERR_INVALID, "page_tokens=%d must be a multiple of %d up to 4096", d->page_tokens, PI_KV_BLOCK);
  if (d->pages < 1 || d->pages > 1 << 20) return fail(PI_ERR_INVALID, "pages=%d must lie in [1, 2^20]", d->pages);
  if (d->layers < 1 || d->layers > 65536) return fail(PI_ERR_INVALID, "layers=%d must lie in [1, 65536]", d->layers);
  if (d->max_seqs < 1 || d->max_seqs > 65536)
    return fail(PI_ERR_INVALID, "max_seqs=%d must lie in [1, 65536]", d->max_seqs);
  if (d->max_seq_pages < 1 || (int64_t)d->max_seq_pages * d->page_tokens > (int64_t)1 << 30)
    return fail(PI_ERR_INVALID, "max_seq_pages=%d: a sequence holds 1 page to 2^30 tokens", d->max_seq_pages);
  if (d->act_dtype != PI_KV_F16 && d->act_dtype != PI_KV_BF16)
    return fail(PI_ERR_INVALID, "act_dtype=%d is not a pi_kv_act", d->act_dtype);
  if (d->code != PI_KV_E4M3 && d->code != PI_KV_INT8) return fail(PI_ERR_INVALID, "code=%d is not a pi_kv_code", d->code);
  return PI_OK;
}

}  // namespace

struct pi_kv {
  pi_kv_desc desc;
  pi_kv_buffers buf;
  char* ws;
  Layout L;

  size_t page_bytes() const { return (size_t)desc.kv_heads * desc.page_tokens * desc.head_dim; }
  size_t exp_bytes() const { return (size_t)desc.kv_heads * (desc.page_tokens / PI_KV_BLOCK); }
};

namespace {

pik::KvView view_of(const pi_kv* h, int layer, const pi_kv_batch* b) {
  const pi_kv_desc& d = h->desc;
  const size_t page = (size_t)layer * d.pages;
  pik::KvView c{};
  c.k = static_cast<uint8_t*>(h->buf.k) + page * h->page_bytes();
  c.v = static_cast<uint8_t*>(h->buf.v) + page * h->page_bytes();
  c.k_exp = static_cast<uint8_t*>(h->buf.k_exp) + page * h->exp_bytes();
  c.v_exp = static_cast<uint8_t*>(h->buf.v_exp) + page * h->exp_bytes();
  c.table = h->buf.table;
  c.lens = h->buf.lens;
  c.seqs = b->seqs;
  c.starts = b->starts;
  c.n = b->n;
  c.rows = b->rows;
  c.kv_heads = d.kv_heads;
  c.dim = d.head_dim;
  c.page_blocks = d.page_tokens / PI_KV_BLOCK;
  c.pages = d.pages;
  c.max_seqs = d.max_seqs;
  c.max_pages = d.max_seq_pages;
  return c;
}

pik::KvPool pool_of(const pi_kv* h) {
  const pi_kv_desc& d = h->desc;
  pik::KvPool p{};
  p.k = static_cast<uint8_t*>(h->buf.k);
  p.v = static_cast<uint8_t*>(h->buf.v);
  p.k_exp = static_cast<uint8_t*>(h->buf.k_exp);
  p.v_exp = static_cast<uint8_t*>(h->buf.v_exp);
  p.table = h->buf.table;
  p.lens = h->buf.lens;
  p.refs = h->buf.refs;
  p.failed = h->buf.failed;
  p.refused = h->buf.refused;
  p.src = reinterpret_cast<int*>(h->ws + h->L.src);
  p.dst = reinterpret_cast<int*>(h->ws + h->L.dst);
  p.list = reinterpret_cast<int*>(h->ws + h->L.list);
  p.drop = reinterpret_cast<int*>(h->ws + h->L.drop);
  p.count = reinterpret_cast<int*>(h->ws + h->L.count);
  p.page_bytes = (int64_t)h->page_bytes();
  p.exp_bytes = (int)h->exp_bytes();
  p.pages = d.pages;
  p.layers = d.layers;
  p.max_seqs = d.max_seqs;
  p.max_pages = d.max_seq_pages;
  p.page_tokens = d.page_tokens;
  return p;
}

pi_status check_ints(const int32_t* p, const char* name) {
  if (p == nullptr || !aligned(p, 4)) return fail(PI_ERR_INVALID, "%s is NULL or not 4-byte aligned", name);
  return PI_OK;
}

pi_status check_count(const pi_kv* h, int32_t n) {
  if (h == nullptr) return fail(PI_ERR_INVALID, "handle is NULL");
  if (n < 1 || n > h->desc.max_seqs) return fail(PI_ERR_INVALID, "n=%d must lie in [1, max_seqs=%d]", n, h->desc.max_seqs);
  return PI_OK;
}

pi_status check_batch(const pi_kv* h, int32_t layer, const pi_kv_batch* b) {
  if (h == nullptr) return fail(PI_ERR_INVALID, "handle is NULL");
  if (b == nullptr) return fail(PI_ERR_INVALID, "batch is NULL");
  if (layer < 0 || layer >= h->desc.layers)
    return fail(PI_ERR_INVALID, "layer=%d must lie in [0, %d)", layer, h->desc.layers);
  pi_status st = check_count(h, b->n);
  if (st != PI_OK) return st;
  if (b->rows < 0 || b->rows > kMaxRows) return fail(PI_ERR_INVALID, "rows=%d must lie in [0, %d]", b->rows, kMaxRows);
  if ((st = check_ints(b->seqs, "seqs")) != PI_OK) return st;
  return check_ints(b->starts, "starts");
}

pi_status check_rows(const pi_kv_rows* t, const char* name) {
  if (t == nullptr || t->data == nullptr) return fail(PI_ERR_INVALID, "%s is NULL", name);
  if (!aligned(t->data, 16)) return fail(PI_ERR_INVALID, "%s is not 16-byte aligned", name);
  if (t->token_stride < 0 || t->head_stride < 0 || t->token_stride % 8 != 0 || t->head_stride % 8 != 0)
    return fail(PI_ERR_INVALID, "%s: strides (%lld, %lld) must be non-negative multiples of 8 elements", name,
                (long long)t->token_stride, (long long)t->head_stride);
  return PI_OK;
}

pik::KvRows rows_of(const pi_kv_rows* t) { return pik::KvRows{t->data, t->token_stride, t->head_stride}; }

pi_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(PI_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

int32_t pi_kv_abi_version(void) { return PI_KV_ABI_VERSION; }

pi_status pi_kv_workspace_bytes(const pi_kv_desc* desc, size_t* bytes) {
  if (bytes == nullptr) return fail(PI_ERR_INVALID, "bytes is NULL");
  const pi_status st = check_desc(desc);
  if (st != PI_OK) return st;
  *bytes = layout_for(*desc).total;
  return ok();
}

pi_status pi_kv_create(const pi_kv_desc* desc, const pi_kv_buffers* buffers, void* workspace, size_t workspace_bytes,
                       void* stream, pi_kv** out) {
  if (out == nullptr) return fail(PI_ERR_INVALID, "out is NULL");
  *out = nullptr;
  pi_status st = check_desc(desc);
  if (st != PI_OK) return st;
  if (buffers == nullptr) return fail(PI_ERR_INVALID, "buffers is NULL");
  if (buffers->k == nullptr || buffers->v == nullptr || !aligned(buffers->k, 16) || !aligned(buffers->v, 16))
    return fail(PI_ERR_INVALID, "k or v is NULL or not 16-byte aligned");
  if (buffers->k_exp == nullptr || buffers->v_exp == nullptr) return fail(PI_ERR_INVALID, "k_exp or v_exp is NULL");
  if ((st = check_ints(buffers->table, "table")) != PI_OK || (st = check_ints(buffers->lens, "lens")) != PI_OK ||
      (st = check_ints(buffers->refs, "refs")) != PI_OK || (st = check_ints(buffers->failed, "failed")) != PI_OK ||
      (st = check_ints(buffers->refused, "refused")) != PI_OK)
    return st;
  const Layout L = layout_for(*desc);
  if (workspace == nullptr || !aligned(workspace, kAlign) || workspace_bytes < L.total)
    return fail(PI_ERR_WORKSPACE, "workspace must be %zu bytes, %zu-byte aligned", L.total, kAlign);
  pi_kv* h = new (std::nothrow) pi_kv{};
  if (h == nullptr) return fail(PI_ERR_INVALID, "out of host memory");
  h->desc = *desc;
  h->buf = *buffers;
  h->ws = static_cast<char*>(workspace);
  h->L = L;
  const hipError_t e = pik::launch_fill_u32(reinterpret_cast<unsigned*>(h->ws), (int)(L.src / sizeof(unsigned)), 0u,
                                            static_cast<hipStream_t>(stream));
  if (e != hipSuccess) {
    delete h;
    return fail(PI_ERR_HIP, "clearing the workspace failed: %s", hipGetErrorString(e));
  }
  *out = h;
  return ok();
}

pi_status pi_kv_destroy(pi_kv* h) {
  if (h == nullptr) return fail(PI_ERR_INVALID, "handle is NULL");
  delete h;
  return ok();
}

pi_status pi_kv_append(pi_kv* h, int32_t layer, const pi_kv_rows* k, const pi_kv_rows* v, const pi_kv_batch* batch,
                       void* stream) {
  pi_status st = check_batch(h, layer, batch);
  if (st != PI_OK) return st;
  if (batch->rows == 0) return ok();
  if ((st = check_rows(k, "k")) != PI_OK || (st = check_rows(v, "v")) != PI_OK) return st;
  pik::KvStoreArgs a{view_of(h, layer, batch), rows_of(k), rows_of(v), nullptr, h->buf.refused};
  return launched(pik::launch_kv_append(h->desc.act_dtype, h->desc.code, a, static_cast<hipStream_t>(stream)), "append");
}

pi_status pi_kv_read(pi_kv* h, int32_t layer, const pi_kv_rows* k, const pi_kv_rows* v, const pi_kv_batch* batch,
                     const int32_t* first, void* stream) {
  pi_status st = check_batch(h, layer, batch);
  if (st != PI_OK) return st;
  if (first != nullptr && (st = check_ints(first, "first")) != PI_OK) return st;
  if (batch->rows == 0) return ok();
  if ((st = check_rows(k, "k")) != PI_OK || (st = check_rows(v, "v")) != PI_OK) return st;
  pik::KvStoreArgs a{view_of(h, layer, batch), rows_of(k), rows_of(v), first, nullptr};
  return launched(pik::launch_kv_read(h->desc.act_dtype, h->desc.code, a, static_cast<hipStream_t>(stream)), "read");
}

pi_status pi_kv_attend(pi_kv* h, int32_t layer, const pi_kv_attend_args* args, const pi_kv_batch* batch, void* stream) {
  pi_status st = check_batch(h, layer, batch);
  if (st != PI_OK) return st;
  if (args == nullptr) return fail(PI_ERR_INVALID, "args is NULL");
  if (args->window < 0 || args->sinks < 0)
    return fail(PI_ERR_INVALID, "window=%d and sinks=%d must not be negative", args->window, args->sinks);
  if (!(args->scale > 0.0f) || !std::isfinite(args->scale))
    return fail(PI_ERR_INVALID, "scale=%g must be positive and finite", (double)args->scale);
  if (batch->rows == 0) return ok();
  if (args->max_new < 1 || args->max_new > batch->rows)
    return fail(PI_ERR_INVALID, "max_new=%d must lie in [1, rows=%d]", args->max_new, batch->rows);
  if ((st = check_rows(&args->q, "q")) != PI_OK || (st = check_rows(&args->out, "out")) != PI_OK) return st;
  if (!aligned(args->lse, 4)) return fail(PI_ERR_INVALID, "lse is not 4-byte aligned");
  pik::KvAttendArgs a{};
  a.c = view_of(h, layer, batch);
  a.q = rows_of(&args->q);
  a.out = rows_of(&args->out);
  a.lse = args->lse;
  a.heads = h->desc.heads;
  a.group = h->desc.heads / h->desc.kv_heads;
  a.max_new = args->max_new;
  a.window = args->window;
  a.sinks = args->sinks;
  a.scale = args->scale;
  a.partial = reinterpret_cast<float*>(h->ws + h->L.partial);
  a.tickets = reinterpret_cast<unsigned*>(h->ws + h->L.tickets);
  // Rows of a cached head for which the codes go straight to the matrix instructions; more go through LDS.  33 to 64
  // rows of 128 dims are slow there (one workgroup a compute unit, and large parts to join), which pays only where
  // there are items enough: eight tokens on one head of eight query heads, sequences of 4000, took 34.9 us against
  // 24.1 through LDS with 16 items, 36.4 against 31.1 with 32, 41.2 against 41.8 with 64 and 56 against 82 with 128.
  // With 64 dims, four tokens of 16 query heads, 48.6 against 62.7 us over 100003 tokens, 18.1 against 14.2 over 2000.
  // That kernel counts the call's blocks of 32 tokens in 32 bits: a table with room for more (2^30 tokens each of eight
  // sequences on eight heads, say) goes through LDS, whatever it holds.
  const int64_t shared = (int64_t)a.max_new * a.group, items = (int64_t)a.c.n * a.c.kv_heads;
  const int64_t cap = (int64_t)a.c.max_pages * a.c.page_blocks;
  const int64_t seen = a.window > 0 ? std::min(cap, ((int64_t)a.window + a.sinks + a.max_new) / PI_KV_BLOCK + 4) : cap;
  const bool counts = (seen + pik::kStepGrain) * items <= INT32_MAX;
  if (counts && shared <= (a.c.dim == 64 || items >= 64 ? pik::kStepRows : 32))
    return launched(pik::launch_kv_step(h->desc.act_dtype, h->desc.code, a, static_cast<hipStream_t>(stream)), "attend");
  return launched(pik::launch_kv_tile(h->desc.act_dtype, h->desc.code, a, static_cast<hipStream_t>(stream)), "attend");
}

pi_status pi_kv_reserve(pi_kv* h, const int32_t* seqs, const int32_t* counts, int32_t n, void* stream) {
  pi_status st = check_count(h, n);
  if (st != PI_OK) return st;
  if ((st = check_ints(seqs, "seqs")) != PI_OK || (st = check_ints(counts, "counts")) != PI_OK) return st;
  return launched(pik::launch_kv_reserve(pool_of(h), seqs, counts, n, static_cast<hipStream_t>(stream)), "reserve");
}

pi_status pi_kv_free(pi_kv* h, const int32_t* seqs, int32_t n, void* stream) {
  pi_status st = check_count(h, n);
  if (st != PI_OK) return st;
  if ((st = check_ints(seqs, "seqs")) != PI_OK) return st;
  return launched(pik::launch_kv_free(pool_of(h), seqs, n, static_cast<hipStream_t>(stream)), "free");
}

pi_status pi_kv_fork(pi_kv* h, const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  pi_status st = check_count(h, n);
  if (st != PI_OK) return st;
  if ((st = check_ints(src, "src")) != PI_OK || (st = check_ints(dst, "dst")) != PI_OK) return st;
  return launched(pik::launch_kv_fork(pool_of(h), src, dst, n, static_cast<hipStream_t>(stream)), "fork");
}

pi_status pi_kv_compact(pi_kv* h, void* stream) {
  if (h == nullptr) return fail(PI_ERR_INVALID, "handle is NULL");
  return launched(pik::launch_kv_compact(pool_of(h), static_cast<hipStream_t>(stream)), "compact");
}

}  // extern "C"
