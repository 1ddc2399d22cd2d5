/*
 * lora_f8.h -- adapters on a frozen base held in 8-bit floating point, with a
 * scale for each block of 128.
 *
 * A matrix is codes of one byte (e4m3 or e5m2) and fp32 scales: the value of
 * element (r, c) is its code's times the scale of its group.  A group is
 * LORA_F8_BLOCK consecutive columns of one row (activations and gradients,
 * quantised as they come) or a block of LORA_F8_BLOCK rows and as many columns
 * (the base's weights, quantised once):
 *   - lora_f8_quantize: bf16 or fp32 values to codes and scales, of either kind;
 *   - lora_base_f8: y = x W0^T of an 8-bit x [T, d_in] and W0 [d_out, d_in];
 *   - lora_base_f8_backward: dx = dy W0 of an 8-bit dy [T, d_out] and the same W0
 *     (which is frozen, so it has no gradient).
 * The adapters' term comes after: lora_apply (or lora_bgmv) adds it to y, from the
 * unquantised x, and lora_sgmv_backward adds the adapters' part to dx.
 *
 * Conventions are those of lora_sgmv.h: the caller owns every buffer, calls are
 * asynchronous on `stream`, allocate nothing and keep nothing between calls,
 * argument errors found on the host are returned before anything is launched,
 * and what only the device can see is OR-ed into *dev_err (may be NULL).  Calls
 * can be captured in CUDA graphs.  Results do not depend on timing.
 */
#ifndef LORA_F8_H
#define LORA_F8_H

#include "lora_sgmv.h"
#include "lora_train.h" /* LORA_DERR_NONFINITE */

#ifdef __cplusplus
extern "C" {
#endif

/* Types of codes.  Largest magnitudes: 448 and 57344. */
#define LORA_F8_E4M3 0
#define LORA_F8_E5M2 1
/* Types of what is not in 8 bits. */
#define LORA_F8_FROM_BF16 0
#define LORA_F8_FROM_F32 1
#define LORA_F8_BLOCK 128

/** An 8-bit matrix.  Groups at the right and lower edges may be short.  More than
 *  0x7fff0000 rows or columns are LORA_ERR_UNSUPPORTED. */
typedef struct {
  void* codes;        /* device, one byte an element, 16-byte aligned; rows of ld bytes */
  int64_t ld;         /* >= cols, a multiple of 16 */
  float* scales;      /* device: element (r, c) has scales[r / block_rows * scale_row + c / 128 * scale_col] */
  int64_t scale_row;  /* >= 0; 0 where a matrix that is only read shares scales between rows */
  int64_t scale_col;  /* >= 0 */
  int32_t rows;       /* >= 0 */
  int32_t cols;       /* >= 1 */
  int32_t block_rows; /* 1 or LORA_F8_BLOCK */
  int32_t type;       /* LORA_F8_E4M3 or LORA_F8_E5M2 */
} lora_f8_matrix_t;

/* Flags of lora_f8_quantize. */
#define LORA_F8_POW2 1 /* scales are powers of two */

/**
 * Quantise x (device, rows of ldx elements of `dtype`) into q: with a the largest
 * magnitude of a group and M that of the code's type,
 *     scale = fp32(a / M), or the least power of two s with M s >= a (LORA_F8_POW2),
 *     code  = the nearest code (ties to even) of fp32(x / scale).
 * A group with a < 2^-64 holds zeros, with scale 0.  A group with an infinity or
 * a NaN sets LORA_DERR_NONFINITE; its scale is that infinity or NaN, and what is
 * computed from the group is NaN.  Padding (columns cols .. ld - 1) is neither
 * read nor written.  q's scales must not share places; x and q must not overlap.
 */
lora_status_t lora_f8_quantize(const void* x, int64_t ldx, int32_t dtype, const lora_f8_matrix_t* q, uint32_t flags,
                               int32_t* dev_err, lora_stream_t stream);

/**
 * y[t, n] = sum_k x[t, k] W0[n, k], written only, as bf16 or fp32 (out_dtype, one
 * of LORA_F8_FROM_*; rounded once).  x: [T, d_in] with groups of one row; w:
 * [d_out, d_in] with blocks of 128 rows; either type of code each.  y: device,
 * rows of ldy >= d_out elements, aligned to the element.  The products of 128
 * consecutive k are summed in the tensor cores' fp32 and, times the fp32 product of
 * both scales, added to an fp32 sum, in ascending order of k (in up to eight spans of k, added in
 * order, where a call has few tiles).  T = 0: nothing to do.  A wait inside the
 * kernel that ran out sets LORA_DERR_TIMEOUT; the tiles it concerned are not written.
 */
lora_status_t lora_base_f8(const lora_f8_matrix_t* x, const lora_f8_matrix_t* w, void* y, int64_t ldy, int32_t out_dtype,
                           int32_t* dev_err, lora_stream_t stream);

/** dx[t, k] = sum_n dy[t, n] W0[n, k]: the same with dy [T, d_out] and dx [T, d_in]. */
lora_status_t lora_base_f8_backward(const lora_f8_matrix_t* dy, const lora_f8_matrix_t* w, void* dx, int64_t lddx,
                                    int32_t out_dtype, int32_t* dev_err, lora_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_F8_H */
