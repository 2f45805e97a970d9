/*
 * pi_kv.h -- C ABI of the 8-bit paged attention cache (gfx950), in libpi_ffn.so.
 *
 * A decode step is attention followed by the sparse FFN of pi_ffn.h.  This half keeps the keys and
 * values of many sequences in pages of 8-bit codes and computes over them:
 *
 *   append   store the last tokens of each sequence
 *   attend   out = softmax(scale q K^T + mask) V for one token a sequence, a few, or whole prompts
 *   share, attend_shared   the same for sequences that begin with the same pages, read and multiplied once for all
 *   read     the stored keys and values, back in the activations' type
 *   reserve, free, fork, compact   move the pages; a page may belong to several sequences
 *   rotate   norms of queries and keys for each head, and their rotation by position, before append and attend
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

#define PI_KV_ABI_VERSION 3

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

/*
 * The rotation of a head's first rot_dims dims by position.  Pair i of them turns by p * f_i at position p:
 *   (a, b) -> gain * (a cos t - b sin t, a sin t + b cos t),   t = p f_i,
 * with f_i = base^(-2 i / rot_dims), scaled for contexts longer than those a model was trained on.
 */
typedef enum pi_rope_layout {
  PI_ROPE_HALF = 0,       /* pair i: dims i and i + rot_dims / 2 */
  PI_ROPE_INTERLEAVED = 1 /* pair i: dims 2 i and 2 i + 1        */
} pi_rope_layout;
typedef enum pi_rope_scaling {
  PI_ROPE_NONE = 0,
  PI_ROPE_LINEAR = 1, /* f_i / factor                                                              */
  PI_ROPE_NTK = 2,    /* base * factor^(rot_dims / (rot_dims - 2)) in the place of base            */
  PI_ROPE_BANDS = 3   /* by the turns r = original f_i / (2 pi) a pair makes within the original length:
                         f_i where r >= high, f_i / factor where r <= low, and in between
                         k f_i + (1 - k) f_i / factor, k = (r - low) / (high - low)                  */
} pi_rope_scaling;
typedef struct pi_rope_desc {
  int32_t head_dim;    /* D: 64 or 128                                               */
  int32_t rot_dims;    /* a multiple of 16 up to D, 0 for none (norms alone)         */
  int32_t layout;      /* pi_rope_layout                                             */
  int32_t scaling;     /* pi_rope_scaling                                            */
  double base;         /* at least 1                                                 */
  double factor;       /* at least 1                                                 */
  double original;     /* PI_ROPE_BANDS: tokens, positive                            */
  double low, high;    /* PI_ROPE_BANDS: 0 <= low < high                             */
  double gain;         /* factor of the cosines and sines, positive; 1 for none      */
  const double* freqs; /* host, [rot_dims / 2], each in [0, pi]: f_i itself, in the place of base and scaling; or NULL */
} pi_rope_desc;
typedef struct pi_rope pi_rope;

/* Outputs may be the inputs themselves, and overlap them in no other way. */
typedef struct pi_kv_rotate_args {
  pi_kv_rows q, q_out;      /* [rows][heads][D]                                              */
  pi_kv_rows k, k_out;      /* [rows][kv_heads][D]                                           */
  const void* q_norm;       /* [D] of the activations' type, 16-byte aligned, or NULL        */
  const void* k_norm;
  const int32_t* positions; /* [rows], or NULL: those of the batch's tokens                  */
  float eps;                /* positive and finite (looked at with a norm)                   */
} pi_kv_rotate_args;

/*
 * Groups of a call's sequences that begin with the same pages (forks of one prompt): group g is the sequences
 * seqs[groups[g]] .. seqs[groups[g + 1] - 1], groups ascending from 0 to n.
 */
typedef struct pi_kv_shared_args {
  const int32_t* groups; /* [n_groups + 1]                                                     */
  const int32_t* plan;   /* [n_groups + n], as pi_kv_share leaves it                           */
  void* state;           /* scratch of the call: pi_kv_state_bytes of its rows or more, 16-byte aligned */
  size_t state_bytes;
  int32_t n_groups;      /* 1 .. n                                                             */
  int32_t max_rows;      /* at least the largest count of tokens (rows) of a group             */
} pi_kv_shared_args;

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
 * How much the sequences of each group share: plan[g] is the number of leading tokens of group g whose pages all
 * of its sequences name alike and that all of them held before this batch's tokens, rounded down to whole blocks; 0 for a
 * group of one.  plan[n_groups + i] is that of seqs[i]'s group.  It holds for every layer, and until lens or table
 * change, for the same seqs, starts and groups.
 */
pi_status pi_kv_share(pi_kv* h, const pi_kv_batch* batch, const int32_t* groups, int32_t n_groups, int32_t* plan,
                      void* stream);

/* Bytes of scratch that pi_kv_attend_shared takes for any number of rows up to `rows`.  Host only. */
pi_status pi_kv_state_bytes(const pi_kv* h, int32_t rows, size_t* bytes);

/*
 * pi_kv_attend for groups: the same results up to the order of sums, but the first plan[g] tokens of a group are read
 * once, from its first sequence's pages, for all rows of the group.  Whole sequences: window and sinks are 0.  A plan
 * that was not made for these sequences gives rows that mean nothing (and touches no other memory).
 *
 * It makes two launches where pi_kv_attend makes one, and leaves states between them: some 10 us more a call.  pi_kv_attend finds
 * what sequences share in the caches after the first of them, so this one is the faster only from some 300 MB on of codes
 * that it spares: (sequences of a group - 1) * shared tokens * kv_heads * 2 * head_dim bytes, summed; and from some four times as
 * much where each brings several tokens of grouped heads.
 */
pi_status pi_kv_attend_shared(pi_kv* h, int32_t layer, const pi_kv_attend_args* args, const pi_kv_shared_args* shared,
                              const pi_kv_batch* batch, void* stream);

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

/* Work the frequencies out (host only; a rope has no device memory) and release them. */
pi_status pi_rope_create(const pi_rope_desc* desc, pi_rope** out);
pi_status pi_rope_destroy(pi_rope* rope);
/* The frequencies f_i [rot_dims / 2], as scaled, in radians a position.  Host only. */
pi_status pi_rope_freqs(const pi_rope* rope, double* freqs);

/*
 * Queries and keys as append and attend take them: with a norm, each head x becomes x / sqrt(mean x^2 + eps) * norm;
 * then its first dims turn by their token's position, lens[s] - count + j for row starts[i] + j of s = seqs[i], as in
 * pi_kv_attend (lens counts the tokens already), or the given one.  In fp32 (a head's sum of squares has to be in
 * its range), rounded once; with the frequencies that pi_rope_freqs gives, angles are off by up to 2^-26 of a turn at any
 * position, and their sines and cosines by up to 2^-20.  Rows of no sequence stay as they are; those of a sequence
 * that is out of range mean nothing.
 */
pi_status pi_kv_rotate(pi_kv* h, const pi_rope* rope, const pi_kv_rotate_args* args, const pi_kv_batch* batch,
                       void* stream);

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
