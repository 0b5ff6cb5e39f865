/*
 * libif4 -- 8-bit floating point with a scale for each block of 128, and the
 * matrix product of two such operands (C ABI): for the layers, or the steps of
 * training, that four bits (if4.h) cost too much.
 *
 * The format: a value is code * 2^(byte - 127), its code E4M3 (1.4.3 bits, bias 7,
 * largest 448, no infinities, NaN 0x7F) and its byte the exponent of its block.
 * A block is BLOCK = 128 consecutive values along the contraction dimension K of
 * one row, or, for weights, a square of 128 rows by 128 values (so that the
 * weight and its transpose hold the same values).  Blocks at the end of a row or
 * column are as long as what is left.
 *   exponent  e = byte - 127, the least one >= -127 with amax * 2^-e <= 448 (amax: the
 *             block's largest magnitude): -127, byte 0, in a block of zeros.
 *   code      E4M3 value nearest to x * 2^-e (ties to even), the sign of zeros kept.
 * Scaling by a power of two rounds nothing, so each value is rounded once, and the
 * matrix cores take the byte as it is.  A block that holds a NaN or an infinity has byte
 * 255 and codes 0x7F: its products are NaN.
 *
 * Layouts (row-major, uint8):
 *   codes   [rows, K]
 *   scales  [rows, ceil(K/128)], or [ceil(rows/128), ceil(K/128)] with squares
 *
 * Conventions, status codes and streams are those of if4.h: device pointers,
 * nothing allocated, arguments checked on the host, work only enqueued.
 */
#ifndef IF4_FP8_H
#define IF4_FP8_H

#include "if4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { IF4_FP8_BLOCK = 128 };

/*
 * Quantize x [rows, cols] with blocks along dim 1 (K = cols).
 *   x        device, IF4_F32 or IF4_BF16, 16-byte aligned, ld_x >= cols with
 *            ld_x * sizeof(dtype) a multiple of 16.
 *   square   0: blocks of one row; 1: squares.
 *   codes    device [rows, cols], 16-byte aligned.
 *   scales   device, see above.
 * cols must be a multiple of 16.
 */
int if4_fp8_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                     int square, uint8_t* codes, uint8_t* scales, void* stream);

/*
 * Quantize x^T (K = rows): codes [cols, rows], scales [cols, ceil(rows/128)] or, with
 * squares, [ceil(cols/128), ceil(rows/128)].  Byte for byte if4_fp8_quantize of a
 * transposed copy.  rows must be a multiple of 16; cols need not.  x as above.
 */
int if4_fp8_quantize_t(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                       int square, uint8_t* codes, uint8_t* scales, void* stream);

/*
 * C = A W^T: A [M, K] with blocks of one row, W [N, K] with blocks of one row
 * (w_square 0) or squares (1).
 * Sums are fp32.  For a c of IF4_F32 every product enters them whole, of values that bf16
 * holds.  It holds all of bytes 3 to 246; of bytes 0, 1 and 2 (blocks of amax up to 448 *
 * 2^-125) values that are no multiples of 2^-133 are rounded to one, and of bytes from 247
 * on those of 2^128 and more are infinities (NaN times zero).  For a c of IF4_BF16, where
 * bytes 0 to 254 are taken as they are, the FP8 matrix instructions add the products: of
 * each 8 neighbouring k they are brought to the exponent of the largest one and cut 13
 * bits below it before they are added, so that a result is off by up to 2^-10 of the sum
 * of its products' magnitudes besides its rounding.
 *   codes    device, 16-byte aligned; scales device.
 *   c        device [M, N], IF4_F32 or IF4_BF16 (rounded to nearest even once), leading
 *            dimension ldc >= N (elements).
 * K must be a multiple of 16; K == 0 writes zeros.  The sum over K may be split: it is
 * then joined in a fixed order through `workspace` (device, 16-byte aligned,
 * if4_fp8_gemm_workspace() bytes, NULL where that is 0; holds nothing between calls).
 * Results do not depend on timing.
 */
int if4_fp8_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes,
                 const uint8_t* w_scales, int w_square, int64_t M, int64_t N, int64_t K, void* c,
                 int c_dtype, int64_t ldc, void* workspace, int64_t workspace_bytes,
                 void* stream);

/* Bytes of workspace that if4_fp8_gemm needs for these sizes, or a negative status code. */
int64_t if4_fp8_gemm_workspace(int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* IF4_FP8_H */
