// Host-side launch interface of the attention cache's kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pik {

constexpr int kKvBlock = 32;   // tokens that share an exponent

// One layer of the cache and the call's sequences, as every token kernel takes them (by value).
struct KvView {
  uint8_t* k;          // the layer's codes [pages][kv_heads][blocks a page][32 * D]
  uint8_t* v;
  uint8_t* k_exp;      // [pages][kv_heads][blocks a page]
  uint8_t* v_exp;
  const int* table;    // [max_seqs][max_pages]
  const int* lens;     // [max_seqs]
  const int* seqs;     // [n]
  const int* starts;   // [n + 1]
  int n, rows;
  int kv_heads, dim, page_blocks;   // page_blocks: blocks a page
  int pages, max_seqs, max_pages;
};

// A packed tensor [rows][heads][D] of the activations' type: strides in elements.
struct KvRows {
  void* data;
  int64_t token, head;
};

struct KvStoreArgs {
  KvView c;
  KvRows k, v;
  const int* first;    // read: first token of each sequence, or NULL
  const int* refused;  // append: the length, plus 1, at which reserve refused a sequence, else 0 [max_seqs]
};
hipError_t launch_kv_append(int act, int code, const KvStoreArgs& a, hipStream_t s);
hipError_t launch_kv_read(int act, int code, const KvStoreArgs& a, hipStream_t s);

struct KvAttendArgs {
  KvView c;
  KvRows q, out;
  float* lse;          // [rows][heads] or NULL
  int heads, group;    // group: query heads of a cached head
  int max_new, window, sinks;
  float scale;
  int slots, splits;   // set by the launch of many rows
  float* partial;      // workspace: step_partial_floats(D) or tile_partial_floats(D) floats
  unsigned* tickets;   // workspace: kStepTickets counters, zero between calls
};

// Few rows of a cached head (max_new * group up to kStepRows): items (sequences times cached heads) in pieces, one
// workgroup each, see kv_step.hip.  S is at least kStepGrain blocks.
constexpr int kStepRows = 64, kStepGrain = 8;
// tiles: 16-row tiles a wave holds.  One to four workgroups a compute unit, by the registers these take.  Eight
// waves instead of four where 33 to 64 rows have 64 dims: half as many parts to join (four tokens over 100003, 16
// query heads to a cached one: 46.0 against 50.5 us); with 128 dims LDS does not hold eight waves' parts.
constexpr int step_waves(int tiles, int dim) { return tiles == 4 && dim == 64 ? 8 : 4; }
constexpr int step_groups(int tiles, int dim) {
  return 256 * (tiles == 1 ? (dim == 64 ? 4 : 3) : tiles == 4 ? 1 : 2);
}
// The smallest S is the call's blocks over step_shares, and the pieces are at most step_pieces.  With one row tile two
// workgroups a compute unit stream as fast as three or four, and fewer parts have to be joined: up to 512 pieces
// instead of 768 took 44.8 against 50.4 us (one sequence of 100003), 22.4 against 24.5 (four of 8000), 27.1 against
// 32.5 (64 of 2000, 64 dims).  Many items of uneven length, though, end sooner in more pieces: 64 of 100 to 8192,
// 512 items, 66.8 us in up to 896 pieces against 68.5 in 768.
constexpr int step_shares(int tiles, int dim) { return tiles == 1 ? 768 : step_groups(tiles, dim); }
constexpr int step_pieces(int tiles, int dim, int items) {
  const int least = tiles == 1 ? 512 : step_groups(tiles, dim), most = items + step_shares(tiles, dim) / 2;
  return most > least ? most : least;
}
// Workgroups a call is launched with: one a piece, up to kStepOnce; for more pieces as many as the card holds at
// once, each of which takes several and looks through the lengths once (1000 sequences of 300: 155 us, with 4096
// workgroups 244; 300 of 100: 32.6 against 50.3; 256 of 500 on 32 heads: 174 against 193; but 300 of 50 to 8000,
// which the card deals out more evenly than their order does, 225 against 206).
constexpr int kStepOnce = 1024;
constexpr int step_launch(int tiles, int dim, int items) {
  const int pieces = step_pieces(tiles, dim, items);
  return pieces <= kStepOnce ? pieces : step_groups(tiles, dim);
}
// The pieces of items that are cut leave a part each: at most 2 * step_shares, so many tickets (of two levels) and
// places in the workspace there are.
constexpr int kStepTickets = 2 * 2 * 768;
constexpr size_t step_partial_floats(int dim) { return (size_t)2 * 512 * kStepRows * (dim + 4); }
static_assert(768 * 16 <= 512 * kStepRows && step_groups(2, 64) * 32 <= 512 * kStepRows &&
              step_groups(4, 64) * 64 <= 512 * kStepRows && step_groups(2, 128) <= 768, "workspace");
hipError_t launch_kv_step(int act, int code, const KvAttendArgs& a, hipStream_t s);
// Any number of rows, kTileRows a workgroup; where that leaves fewer than kTileParts / 2 workgroups, the
// tokens of each are split over up to kTileParts in all.
constexpr int kTileRows = 128, kTileParts = 512;
constexpr size_t tile_partial_floats(int dim) { return (size_t)kTileParts * kTileRows * (dim + 4); }
hipError_t launch_kv_tile(int act, int code, const KvAttendArgs& a, hipStream_t s);

// The pool as the page kernels take it.
struct KvPool {
  uint8_t* k;          // [layers][pages][k_bytes]
  uint8_t* v;
  uint8_t* k_exp;      // [layers][pages][e_bytes]
  uint8_t* v_exp;
  int* table;
  int* lens;
  int* refs;
  int* failed;
  int* refused;
  int* src;            // workspace: pages to copy from and to, -1 for none [max(pages, max_seqs)]
  int* dst;
  int* list;           // workspace: reserve's free pages, compact's new places [pages]
  int* drop;           // workspace: the shared page, past a lowered length, whose column each of list gets, or -1 [pages]
  int* count;          // workspace: how many copies
  int64_t page_bytes;  // of k and of v
  int exp_bytes;       // a page's exponents, of k and of v
  int pages, layers, max_seqs, max_pages, page_tokens;
};
hipError_t launch_kv_free(const KvPool& p, const int* seqs, int n, hipStream_t s);
hipError_t launch_kv_fork(const KvPool& p, const int* src, const int* dst, int n, hipStream_t s);
hipError_t launch_kv_reserve(const KvPool& p, const int* seqs, const int* counts, int n, hipStream_t s);
hipError_t launch_kv_compact(const KvPool& p, hipStream_t s);

}  // namespace pik
