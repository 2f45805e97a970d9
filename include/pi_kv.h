/*
 * pi_kv.h -- C ABI of the 8-bit paged attention cache (gfx950), in libpi_ffn.so.
 *
 * A decode step is attention followed by the sparse FFN of pi_ffn.h.  This half keeps the keys and
 * values of many sequences in pages of 8-bit codes and computes over them:
 *
 *   append   store the last tokens of each sequence
 *   attend   out = softmax(scale q K^T + mask) V for one token a sequence, a few, or whole prompts
 *   read     the stored keys and values, back in the activations' type
 *   reserve, free, fork, compact   move the pages; a page may belong to several sequences
 *
 * What is stored
 * --------------
 * - A block is 32 consecutive tokens of one head of K (or of V).  It has one exponent e, the smallest
 *   integer with amax <= TOP * 2^e (TOP: 448 for e4m3, 127 for int8), kept in [-126, 127], and -126 for
 *   a block of zeros; its codes are x * 2^-e rounded to nearest even, to e4m3 (4-bit exponent, 3-bit
 *   mantissa, no infinities) or to whole numbers.  A token's values are code * 2^e.
 * - A later token that needs a larger e raises it: the codes that are there are rounded to the new e.
 * - Cached values are finite: an infinity is stored as the largest finite value of the activations'
 *   type, a NaN as zero.
 *
 * Layout (sizes in bytes; D = head_dim, P = page_tokens)
 * ------------------------------------------------------
 * - k and v: [layers][pages][kv_heads][P / 32][32 * D].  k_exp and v_exp: [layers][pages][kv_heads][P / 32],
 *   one byte e + 127.  Within a block the bytes stand in the order the matrix instructions take them:
 *     K  token u, dim c  ->  (t * D/16 + c / 16) * 256 + r * 16 + c % 16,
 *                            t = (u / 4) % 2,  r = 4 * (u / 8) + u % 4
 *     V  token u, dim c  ->  (c / 32) * 1024 + (16 * (u / 8) + c % 16) * 16 + 8 * ((c / 16) % 2) + u % 8
 * - table: int32 [max_seqs][max_seq_pages], the pages of each sequence in order, -1 where there is none.
 *   lens: int32 [max_seqs], tokens of each sequence.  refs: int32 [pages], how many table entries name
 *   each page; a page with 0 is free.  refused: int32 [max_seqs], lens + 1 of a sequence whose last
 *   request for tokens pi_kv_reserve could not meet, else 0.  They are the caller's device memory and may
 *   be set by the caller between calls.
 * - A caller may lower a length (guessed tokens that were not taken).  The pages past it stay the
 *   sequence's: its next pi_kv_reserve uses them again, pi_kv_free drops them.  A block keeps the exponent
 *   that its dropped tokens brought.
 *
 * Conventions (as in pi_ffn.h: status codes, pi_last_error, host checks before anything is enqueued)
 * --------------------------------------------------------------------------------------------------
 * - Ownership: the caller allocates all device memory; a handle borrows it until pi_kv_destroy.
 * - Streams: calls only enqueue on `stream`.  A handle's calls share its workspace: serialise them on
 *   one stream, or order the streams.
 * - A call names its sequences in seqs (int32 [n], rows of the table, no row twice) and packs their
 *   tokens: those of seqs[i] are rows [starts[i], starts[i + 1]) of the call's tensors, starts being
 *   int32 [n + 1] from 0 to `rows`, in ascending order.
 * - Rows of q, k, v and out are [token][head][D] with the innermost dimension contiguous; the token and
 *   head strides are given, in elements.  Addresses and strides are multiples of 16 bytes.
 * - What only the device knows is bounded there: sequence numbers, page numbers and lengths outside
 *   their ranges read as nothing and write nothing.
 * - Results do not depend on the order in which workgroups run.
 */
#ifndef PI_KV_H
#define PI_KV_H

#include "pi_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PI_KV_ABI_VERSION 2

#define PI_KV_BLOCK 32 /* tokens that share an exponent */

typedef enum pi_kv_act { PI_KV_F16 = 0, PI_KV_BF16 = 1 } pi_kv_act;
typedef enum pi_kv_code { PI_KV_E4M3 = 0, PI_KV_INT8 = 1 } pi_kv_code;

typedef struct pi_kv_desc {
  int32_t heads;         /* query heads: a multiple of kv_heads, up to 1024               */
  int32_t kv_heads;      /* cached heads; query head h reads cached head h / (heads / kv_heads) */
  int32_t head_dim;      /* D: 64 or 128                                                  */
  int32_t page_tokens;   /* P: a positive multiple of 32, up to 4096                      */
  int32_t pages;         /* pages of the pool, up to 2^20                                 */
  int32_t layers;        /* layers that share table, lens and refs                        */
  int32_t max_seqs;      /* rows of the table, up to 65536                                */
  int32_t max_seq_pages; /* columns of the table; P * max_seq_pages up to 2^30            */
  int32_t act_dtype;     /* pi_kv_act: type of q, k, v and out                            */
  int32_t code;          /* pi_kv_code                                                    */
} pi_kv_desc;

typedef struct pi_kv_buffers {
  void* k;         /* codes, 16-byte aligned                                      */
  void* v;
  void* k_exp;     /* exponents, one byte each                                    */
  void* v_exp;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int32_t* failed; /* [1]: sequences that pi_kv_reserve could not grow, summed    */
  int32_t* refused; /* [max_seqs]: which these are, see above                     */
} pi_kv_buffers;

/* The tokens of one call: see the conventions above. */
typedef struct pi_kv_batch {
  const int32_t* seqs;   /* [n]                 */
  const int32_t* starts; /* [n + 1]             */
  int32_t n;             /* 1 .. max_seqs       */
  int32_t rows;          /* packed tokens, >= 0 */
} pi_kv_batch;

/* A packed tensor [rows][heads or kv_heads][D]: strides in elements. */
typedef struct pi_kv_rows {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} pi_kv_rows;

typedef struct pi_kv_attend_args {
  pi_kv_rows q, out;
  float* lse;      /* [rows][heads], natural logarithm, or NULL                   */
  int32_t max_new; /* at least the largest count of tokens of a sequence          */
  int32_t window;  /* 0: all earlier tokens; else how many, its own among them    */
  int32_t sinks;   /* with a window: first tokens that every later row sees too   */
  float scale;     /* positive and finite                                         */
} pi_kv_attend_args;

typedef struct pi_kv pi_kv;

/* ABI version of this half of the library (PI_KV_ABI_VERSION). */
int32_t pi_kv_abi_version(void);

/* Bytes of device workspace a handle with this descriptor needs.  Host only. */
pi_status pi_kv_workspace_bytes(const pi_kv_desc* desc, size_t* bytes);

/*
 * Bind buffers and workspace (256-byte aligned) to a new handle and clear the workspace's counters
 * with a kernel on `stream`.  The buffers' contents are the caller's to set: table -1, lens, refs,
 * failed and refused 0 for an empty cache; codes and exponents need no initial value.
 */
pi_status pi_kv_create(const pi_kv_desc* desc, const pi_kv_buffers* buffers, void* workspace, size_t workspace_bytes,
                       void* stream, pi_kv** out);

/* Release the handle (host memory only). */
pi_status pi_kv_destroy(pi_kv* h);

/*
 * Store the last tokens of each sequence: row starts[i] + j is token lens[s] - count + j of s = seqs[i],
 * count = starts[i + 1] - starts[i].  lens already counts them (pi_kv_reserve), and their pages are in
 * the table.  Other tokens of a block that has them keep their values, up to the rounding that a larger
 * exponent brings; tokens past the sequence's end become zeros.  rows = 0 enqueues nothing.
 *
 * Nothing is stored for a sequence that pi_kv_reserve refused at the length it still has (refused[s] =
 * lens[s] + 1): its last tokens are not those of this call.  So a step that is enqueued as a whole keeps
 * what is stored, pages shared with other sequences among it; pi_kv_attend then stands at the tokens that
 * are there, and its rows of that sequence mean nothing.  A reserve that grows it, or a free, ends that.
 */
pi_status pi_kv_append(pi_kv* h, int32_t layer, const pi_kv_rows* k, const pi_kv_rows* v, const pi_kv_batch* batch,
                       void* stream);

/*
 * Read tokens back: row starts[i] + j gets token first[i] + j of seqs[i] (first NULL: from token 0), as
 * code * 2^e clamped to the finite range of the activations' type and rounded to it once.  Tokens past
 * the end, before token 0, or of no page, read as 0.
 */
pi_status pi_kv_read(pi_kv* h, int32_t layer, const pi_kv_rows* k, const pi_kv_rows* v, const pi_kv_batch* batch,
                     const int32_t* first, void* stream);

/*
 * Attention of the last tokens of each sequence over the cache, which holds them already.  Row
 * starts[i] + j stands at position p = lens[s] - count + j and sees the tokens u <= p with
 * u > p - window or u < sinks (all u <= p where window is 0).  With x_u = scale * <q, K_u>:
 *   lse = log sum_u exp(x_u)     out = sum_u exp(x_u - lse) V_u
 * in fp32 (the products of the matrix instructions take exp() rounded to fp16, see the kernels), out
 * clamped to the finite range of the activations' type and rounded once.  A row that sees no token gets
 * out 0 and lse -inf.
 */
pi_status pi_kv_attend(pi_kv* h, int32_t layer, const pi_kv_attend_args* args, const pi_kv_batch* batch, void* stream);

/*
 * Make room for counts[i] more tokens of seqs[i] and count them in lens: free pages are taken from the
 * lowest number up, in the order of seqs, and a last page that is partly filled and shared (refs > 1 before
 * the call) is copied, in every layer, to a page of the sequence's own.  Columns past the length that
 * still name a page keep it if no other entry names it (refs 1 before the call); a shared one's refs goes
 * down by one and a free page takes its place.  A sequence whose table row is
 * too short stays as it is; so do the first for which too few pages are free and all after it.  Each of
 * these is counted in `failed` and, unless it asked for 0 tokens, marked in `refused`.
 */
pi_status pi_kv_reserve(pi_kv* h, const int32_t* seqs, const int32_t* counts, int32_t n, void* stream);

/* Drop the sequences' pages: refs of each goes down by one, table rows become -1, lens 0. */
pi_status pi_kv_free(pi_kv* h, const int32_t* seqs, int32_t n, void* stream);

/*
 * Let dst[i] continue src[i]: the same pages, shared.  dst rows hold nothing before the call
 * (pi_kv_free), no row is twice in dst, and none of them in src.
 */
pi_status pi_kv_fork(pi_kv* h, const int32_t* src, const int32_t* dst, int32_t n, void* stream);

/*
 * Move the pages in use to the front of the pool: with L pages in use, those numbered L and above
 * move, in ascending order, to the free pages below L, in ascending order, in every layer; table and
 * refs follow.  Afterwards pages L and above are free.
 */
pi_status pi_kv_compact(pi_kv* h, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PI_KV_H */
