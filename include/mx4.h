/*
 * mx4.h - C ABI of microscaled 4-bit floating point: quantisation of matrices (many in one
 * call, each as it lies, transposed, or both), the way back, and the product of two matrices
 * held so.
 *
 * The format. A matrix of rows x cols is held in blocks of 32 consecutive values of a row
 * (along what a product sums over). A block has one scale, a power of two held as a byte
 * (exponent + 127; 255 is NaN), and each value a code of 4 bits: a sign and one of
 *   0, 1/2, 1, 3/2, 2, 3, 4, 6.
 * The scale is the smallest 2^k, k >= -127, with |x| <= 6 * 2^k over the block, so that no
 * value is cut off; a value becomes x / 2^k rounded to nearest, ties to the even code, or
 * stochastically. With h the distance between the codes around |x| / 2^k,
 *   |code| = h * floor(|x| / (2^k h) + (b + 1/2) / 65536),
 * b the 16 random bits of its place: values 2j and 2j + 1 of row i take the low and the high
 * half of mix(j ^ mix(i ^ key)), mix and the key of a seed as in adamw.h with t = 0. The
 * transposed matrix is rounded as a matrix of its own: row i is column i of the source.
 * A block that holds a NaN or an infinity has the scale 255 and codes 0, so that all of it is
 * NaN; other blocks are not touched by it. At the top of fp32's range (scale 2^126) what would
 * round to 2^128 is held as 3 * 2^126, so that every finite value is held as a finite one.
 *
 * The layout, made for the matrix cores' loads. Rows in panels of 16, columns in steps of 128;
 * codes: for each panel, for each step, 16 rows of 64 bytes (two codes a byte, the first in the
 * low half); scales: for each panel, for each step, 16 rows of 4 bytes. Rows and columns beyond
 * the matrix are there up to the next multiple of 16 and of 128, with codes and scales 0.
 *
 * The product. out (m x n, row-major) = A B^T for A (m x k) and B (n x k), summed in fp32 and
 * rounded once: out_ij = sum over k of A_ik B_jk. Sums run in a fixed order: equal inputs give
 * equal bits. k = 0 gives zeros.
 *
 * Conventions are those of muon.h (device buffers on the current device, validation before
 * anything is enqueued, no synchronisation, no allocation), but that sources and results need
 * be aligned to their elements only. Codes and scales are 16-byte aligned.
 */
#ifndef MUON_MX4_H
#define MUON_MX4_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the codes and of the scales of a rows x cols matrix (0 where one is 0; SIZE_MAX for
 * sizes outside [0, 2^31 - 256] or with more than 2^40 values). */
size_t muon_mx_codes_size(int64_t rows, int64_t cols);
size_t muon_mx_scales_size(int64_t rows, int64_t cols);

/* One matrix to quantise: row i starts at x + i * row_stride elements (row_stride >= cols, or
 * any where rows <= 1). codes and scales receive it as it lies, codes_t and scales_t the
 * transposed matrix (cols x rows); each pair may be NULL, not both. */
typedef struct {
  const void *x;
  int64_t rows;
  int64_t cols;
  int64_t row_stride;
  muon_dtype dtype;
  void *codes;
  void *scales;
  void *codes_t;
  void *scales_t;
} muon_mx_source;

/* Quantises n matrices (one launch for up to 60 of one dtype and the same results asked for).
 * stochastic 0 or 1; seed: of the random bits, which depend on it and on a value's place in
 * its matrix alone. No result may overlap another or a source. A source may have up to 2^23 tiles of
 * 64 x 128 values (128 x 128 where its transpose is asked for), else MUON_ERR_UNSUPPORTED. */
int muon_mx_quantize(const muon_mx_source *sources, int64_t n, int stochastic, uint64_t seed,
                     hipStream_t stream);

/* out (rows x cols, row-major, contiguous) receives the values that codes and scales stand
 * for, exactly (infinity beyond fp32's range, which scales of 2^126 and 2^127 can reach). Up to 2^25 tiles of
 * 16 x 128 values, else MUON_ERR_UNSUPPORTED. */
int muon_mx_dequantize(const void *codes, const void *scales, int64_t rows, int64_t cols,
                       void *out, muon_dtype dtype, hipStream_t stream);

/* Bytes of workspace that a product of these sizes needs (16-byte aligned, no initial contents
 * required; 0: none). SIZE_MAX for sizes outside the library's limits. */
size_t muon_mx_matmul_workspace_size(int64_t m, int64_t n, int64_t k);

/* out (m x n of dtype) = A B^T; m x n up to 2^23 tiles of 128 x 128, else MUON_ERR_UNSUPPORTED. */
int muon_mx_matmul(const void *a_codes, const void *a_scales, const void *b_codes,
                   const void *b_scales, int64_t m, int64_t n, int64_t k, void *out,
                   muon_dtype dtype, void *workspace, size_t workspace_bytes,
                   hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MUON_MX4_H */
