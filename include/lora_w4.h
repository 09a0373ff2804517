/* Base projection from 4-bit weights, beside lora_base_gemm of lora_sgmv.h:
 * y = x W^T with W stored as 4-bit codes and one scale (and optionally one
 * zero point) per row and group of k,
 *
 *     W[n][k] = (u[n][k] - z[k / group][n]) * s[k / group][n],   u in 0..15,
 *
 * z = 8 where no zero points are given (the symmetric codes -8 .. 7).  A
 * quantized base frees HBM for adapters, whose bf16 deltas are then added to y
 * ("Multi-LoRA serving: the single translator with a thousand glossaries",
 * sections "The maths that matters" and "Combined pattern").  Same status
 * codes and conventions as lora_sgmv.h.
 *
 * Codes are stored in tiles of 16 rows x 128 k, 1024 bytes each, tile (i, j)
 * (rows 16 i .., k 128 j ..) at byte 1024 (i * ceil(k / 128) + j).  A tile is
 * 64 runs of 16 bytes, run 16 g + r holding row 16 i + r; its four
 * little-endian 32-bit words w = 0..3 hold the codes of k = 128 j + 32 w + 8 g
 * + e, e = 0..7, element e in nibble 0, 4, 1, 5, 2, 6, 3, 7 (bits 4 * nibble
 * ..).  That is the order in which the matrix cores take their operand, so
 * one load instruction of a wave reads one whole tile and two codes leave a
 * word with one AND-OR.  lora_w4_pack writes this layout from row-major codes.
 * Codes of rows >= n and of k beyond the matrix are never used.             */
#ifndef LORA_W4_H
#define LORA_W4_H

#include "lora_sgmv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t n, k;        /* W is n x k; n a multiple of 8, at most 2^26, k of group, at most 2^24 */
  int32_t group;       /* 32, 64 or 128 */
  int32_t scale_dtype; /* LORA_F32 or LORA_BF16: element type of scales and zeros */
  const void *codes;   /* device, lora_w4_bytes(n, k) bytes */
  const void *scales;  /* device [k / group][n] */
  const void *zeros;   /* device [k / group][n], or NULL (8 everywhere) */
} lora_w4_weights;

/* Bytes of the codes of an n x k matrix: 1024 ceil(n / 16) ceil(k / 128).
 * Host only.  Errors: LORA_EINVAL (sizes, null bytes). */
lora_status lora_w4_bytes(int32_t n, int32_t k, int64_t *bytes);

/* Writes the tiled codes from row-major ones: rows [n][k / 2] device bytes, two
 * codes a byte, element 2i in the low nibble (the LORA_WFMT_INT4 order).
 * twos_complement 1: the nibbles are -8 .. 7 and u = value + 8; 0: they are u
 * itself.  Padding gets u = 8.  rows and codes 16-byte aligned; n a multiple of
 * 8, k of 32, below the limits above and 16 GiB of codes.  Done once when weights are loaded.  Errors: LORA_EINVAL,
 * LORA_EUNSUPPORTED, LORA_EHIP. */
lora_status lora_w4_pack(int32_t n, int32_t k, int32_t twos_complement, const void *rows, void *codes,
                         hipStream_t stream);

/* y[t] = x[t] W^T for m tokens, m >= 0: built for few (a decode batch), right for any
 * number (every 64 tokens read W once more).
 *   dtype      LORA_BF16: element type of x and y
 *   x          device, row t at x + t * x_stride elements; y likewise
 *   x_stride, y_stride  >= k and >= n, multiples of 8: y may be a column block of a
 *              wider array (the q, k and v projections of a layer side by side)
 * bf16 products and fp32 sums (matrix cores), the group's scale and zero point applied in
 * fp32, y rounded once to nearest even.  The codes enter as 128 + u, which
 * bf16 holds exactly; 128 + z times the group's sum of x is taken off in fp32.  With
 * zero points in 0..15 both sums have terms of at most 143 |x| and at most group + 4
 * roundings, so before scaling a group's sum is off by at most
 * 2^-24 (group + 4) 288 sum |x|: 2^-8.8 of sum |x| for groups of 128 if every rounding
 * went one way, 2^-15.5 in a model with random x.  143 group |x| < 2^128 keeps both sums
 * finite (|x| below 2^113.8 for groups of 128); a larger or non-finite x gives a
 * non-finite or unspecified y in its own row only.  Nothing is allocated, no workspace is
 * used, and results are bit-identical from run to run; a token's bits do not
 * depend on the other tokens of the call except through m's tile choice.
 * m == 0 is a no-op.  x and y must not overlap.
 * Errors: LORA_EINVAL (null or misaligned pointers, sizes, strides),
 * LORA_EUNSUPPORTED (dtype, scale_dtype, group, n or k not multiples as
 * above, an x_stride above 2^24), LORA_EHIP. */
lora_status lora_base_w4(int32_t dtype, int32_t m, const lora_w4_weights *w, const void *x,
                         int64_t x_stride, void *y, int64_t y_stride, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_W4_H */
