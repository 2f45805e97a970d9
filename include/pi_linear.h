/*
 * pi_linear.h -- C ABI of products with 4-bit weights (gfx950), in libpi_ffn.so.
 *
 * The projections of an attention layer, for a step of one token or many and for prompts:
 *
 *   y[t] = W x[t] + bias + add[t]          W [d_out][d_in] in q4g32, the FFN's format (pi_ffn.h)
 *
 * Weights are laid out once, by pi_linear_create, in the order in which the matrix instructions take them;
 * the q4g32 rows are not needed afterwards.
 *
 * Layout of the packed weights
 * ----------------------------
 * [ceil(d_out / 16)][ceil(d_in / 256)] slabs of 2304 bytes: two KB of codes, one for each 128 columns, and fp16
 * scales [16 rows][8 groups].  Word j of the 16 bytes 16 l .. of a KB holds the columns 32 j + 8 (l / 16) .. + 8
 * of row l % 16, as u = q + 8: column 2 i at bit 4 i and column 2 i + 1 at bit 16 + 4 i, the word rotated left
 * by 6 bits.  Rows and columns that are not there have q = 0 and scale 0.  Behind the
 * slabs stands a power of two for each row (fp32) that its scales were divided by: less than 1 where the largest is below 8,
 * and up to 8 where it is 2^13 or more.  Scales are kept as they are, except beside one of 2^13 and more: there those below
 * 2^-11 are rounded to a multiple of up to 2^-21.
 *
 * Conventions (as in pi_ffn.h: status codes, pi_last_error, host checks before anything is enqueued)
 * --------------------------------------------------------------------------------------------------
 * - Ownership: the caller allocates all device memory; a handle borrows it until pi_linear_destroy.
 * - Streams: calls only enqueue on `stream`.  A handle has no workspace: its calls may run at the same time, each
 *   with a scratch of its own.
 * - Up to 64 rows: products of the whole numbers 24 + q with x are summed in fp32 by groups of 32, from -24 times the sum of
 *   x on, and the groups' sums, times their scales, in fp32.  So a group is off by up to 2^-12 of its sum of |x|, times its
 *   scale, also by an x whose q is 0.
 * - More than 64 rows give fewer bits: code times scale is rounded to fp16 (half a step, 2^-11 of it), so y is off by up to
 *   2^-11 sum |w x| before its own rounding, and bf16 rows are made fp16 relative to their largest (exact down to 2^-29 of it,
 *   and 2^-39 of it lost at most).  Products are summed in fp32.  Where 64 rows' accuracy is needed for more, call with 64.
 * - y is rounded once.  A row's result depends on its own x and on the number of rows of the call: as said, beyond 64, and in
 *   its last bits otherwise.  It does not depend on the order in which workgroups run.
 * - A row of x that holds a NaN, an infinity, or (bf16) a magnitude of 2^118 and more may come out as NaN, also where the
 *   sum would be infinite (up to 64 rows an infinity always does), other rows are not touched by it.
 */
#ifndef PI_LINEAR_H
#define PI_LINEAR_H

#include "pi_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PI_LINEAR_ABI_VERSION 2

typedef enum pi_linear_act { PI_LINEAR_F16 = 0, PI_LINEAR_BF16 = 1 } pi_linear_act;

typedef struct pi_linear_desc {
  int32_t d_in;      /* a multiple of 32, up to 2^20 */
  int32_t d_out;     /* 1 to 2^24                    */
  int32_t act_dtype; /* pi_linear_act: type of x, add and y */
} pi_linear_desc;

/* Rows of a call: y may be add itself, and else overlaps neither x nor add (which is not looked at). */
typedef struct pi_linear_args {
  const void* x;      /* [rows][d_in], 16-byte aligned                                      */
  const void* add;    /* [rows][d_out] or NULL                                              */
  void* y;            /* [rows][d_out]                                                      */
  int64_t x_stride;   /* from row to row, in elements: a multiple of 8 up to 2^23 (looked at for several rows) */
  int64_t add_stride; /* in elements                                                        */
  int64_t y_stride;   /* in elements, at least d_out                                        */
  void* scratch;      /* pi_linear_scratch_bytes, 16-byte aligned, or less: see there; not looked at where that is 0 */
  size_t scratch_bytes;
  int32_t rows;       /* 0 to 2^24; 0 enqueues nothing                                      */
} pi_linear_args;

typedef struct pi_linear pi_linear;

/* ABI version of this part of the library (PI_LINEAR_ABI_VERSION). */
int32_t pi_linear_abi_version(void);

/* Bytes of device memory the packed weights take.  Host only. */
pi_status pi_linear_packed_bytes(const pi_linear_desc* desc, size_t* bytes);

/*
 * Lay the weights w (q4g32 [d_out][d_in / 2], 4-byte aligned) and scales (fp16 [d_out][d_in / 32]) out in
 * `packed` (256-byte aligned) on `stream`, and bind that and bias (fp32 [d_out] or NULL) to a new handle.
 */
pi_status pi_linear_create(const pi_linear_desc* desc, const void* w, const void* scales, const float* bias, void* packed,
                           size_t packed_bytes, void* stream, pi_linear** out);

/* Release the handle (host memory only). */
pi_status pi_linear_destroy(pi_linear* h);

/*
 * Bytes of scratch a call with as many rows takes: 0 up to 64 rows.  Host only.
 *
 * Where the rows alone are too little work for the card, columns are split into up to 8 ranges, each with fp32 sums in the
 * scratch, so a call with more rows may take less.  A call makes as many ranges as its scratch holds, so what a number of
 * rows takes is enough for fewer rows too, if slower where these would be split (and with other last bits: the ranges' sums
 * are joined).
 */
pi_status pi_linear_scratch_bytes(const pi_linear* h, int32_t rows, size_t* bytes);

/* The most that pi_linear_scratch_bytes says for any number of rows up to `rows`: no call of these is slower for it. */
pi_status pi_linear_scratch_bytes_upto(const pi_linear* h, int32_t rows, size_t* bytes);

/* y = W x + bias + add for every row. */
pi_status pi_linear_forward(pi_linear* h, const pi_linear_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PI_LINEAR_H */
