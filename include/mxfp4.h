/*
 * mxfp4.h -- C ABI of microscaled 4-bit floating point (MXFP4) in the same
 * library (libw4a16.so): quantization of weights and activations, the way back,
 * and the product of two quantized operands on the matrix cores that take
 * such operands as they are.
 *
 * Format (OCP Microscaling Formats (MX) Specification 1.0, E2M1 elements with an
 * E8M0 scale): 32 consecutive values of a row are a block.  A block's scale is
 * 2^(s - 127), s a byte; s = 255 makes every value of the block NaN.  An element's
 * code has a sign bit (bit 3), two exponent bits and one of mantissa: 0, 0.5, 1, 1.5,
 * 2, 3, 4 and 6 times the scale.
 *
 * Quantization: e = max(floor(log2(max|x|)) - 2, -127) over the block, s = e + 127,
 * code = x / 2^e to the nearest element, halves to the even mantissa, beyond 6 to 6
 * (the sign of x is kept with zeros too).  A block of zeros has s = 0; one with an
 * infinity or NaN has s = 255 and unspecified codes.  Every step is exact or one
 * rounding, so codes and scales are bit-exact.
 *
 * Layout
 *  - codes: uint8 [rows][k / 2], element 2 i in the low half of byte i.
 *  - scales: uint8 [ceil(k / 256)][rows][8]: block b of a row at [b / 8][row][b % 8], so
 *    that what a tile of rows needs for 256 elements lies side by side.  Bytes
 *    behind a row's last block are written as 0 and not used.
 *
 * Conventions (status codes, streams, ownership: as in w4a16.h)
 *  - type: MX4_F16, MX4_BF16 or, where it says so, MX4_F32.
 *  - k: a multiple of 32, at most 2^20.  rows, m, n_out in [1, 2^24], products of two
 *    sizes at most 2^34.
 *  - Alignment: x, codes and what dequantization writes 16 bytes, scales 8, y 2, workspace 16.
 *  - Rows of x may be further apart than k: `stride` elements, a multiple of 16 bytes.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include <stdint.h>

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MX4_F16 = 0, MX4_BF16 = 1, MX4_F32 = 2 };

/* x (any type) [rows][k] -> codes, scales. */
int mx4_quantize(const void *x, int32_t type, int64_t rows, int64_t k, int64_t stride, uint8_t *codes,
                 uint8_t *scales, void *stream);

/* codes, scales -> out (any type) [rows][k], contiguous: the values, rounded once where
 * the type does not hold them. */
int mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t k, int32_t type, void *out,
                   void *stream);

/*
 * y (MX4_F16 or MX4_BF16) [m][n_out] = x W^T for quantized x [m][k] and W [n_out][k]:
 * products and scales are exact, sums in binary32, one rounding to y's type.  A product
 * of two values whose scales multiply to less than 2^-126 may count as zero.  A block
 * with s = 255 makes the sums that it is part of NaN.  Results do not
 * depend on anything but the operands and sizes.
 * `workspace`: device memory of at least mx4_matmul_workspace_size bytes (may be NULL where that
 * is 0), overwritten; calls sharing one must not overlap.
 */
int mx4_matmul(const uint8_t *x_codes, const uint8_t *x_scales, const uint8_t *w_codes, const uint8_t *w_scales,
               int64_t m, int64_t n_out, int64_t k, int32_t type, void *workspace, int64_t workspace_bytes, void *y,
               void *stream);

/* Workspace bytes of mx4_matmul, for the sums of parts of a long k, and of mx4_linear, which also has the
 * quantized x there; 0 where a call needs none.  No HIP call is made. */
int64_t mx4_matmul_workspace_size(int64_t m, int64_t n_out, int64_t k);
int64_t mx4_linear_workspace_size(int64_t m, int64_t n_out, int64_t k);

/*
 * The linear layer y = Q(x) W^T: x (MX4_F16 or MX4_BF16) [m][k] is quantized as
 * mx4_quantize does, then multiplied as by mx4_matmul; y has x's type.
 * `workspace`: device memory of at least mx4_linear_workspace_size bytes (may be NULL where that
 * is 0), overwritten; calls sharing one must not overlap.
 */
int mx4_linear(const void *x, int32_t type, int64_t stride, const uint8_t *w_codes, const uint8_t *w_scales, int64_t m,
               int64_t n_out, int64_t k, void *workspace, int64_t workspace_bytes, void *y, void *stream);

/*
 * Kernel selection report, for tests and profiling: writes to `name` the kernels that mx4_linear or, with
 * `linear` 0, mx4_matmul launches for these sizes, in the form in which profilers print their names,
 * NUL-terminated and truncated to name_len bytes.  Nothing is launched and no HIP call is made.
 */
int mx4_linear_config(int64_t m, int64_t n_out, int64_t k, int32_t type, int32_t linear, char *name, int64_t name_len);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
