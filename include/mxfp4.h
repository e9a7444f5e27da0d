/*
 * mxfp4.h -- C ABI of the 4-bit microscaled floats (MXFP4) in libnf4: the
 * encoder and its inverse, the products on the scaled matrix cores of AMD
 * Instinct MI355X (gfx950), and the expert layer of a decode step.  Status
 * codes and all conventions (device pointers owned by the caller, asynchronous
 * work on `stream`, synchronous argument validation, no allocation, thread
 * safety) are those of nf4.h; the types of values are int8.h's int8_dtype.  What
 * a call writes (results, workspace) must not overlap what it reads.
 *
 * ---------------------------------------------------------------------------
 * The format (a matrix of `rows` rows of K elements: one token's activations
 * or one output channel's weights per row)
 * ---------------------------------------------------------------------------
 * A code has four bits: the sign and one of the magnitudes 0, 1/2, 1, 3/2, 2, 3,
 * 4, 6 (E2M1, in this order).  The codes of a row come in blocks of 32 with one
 * byte E each; value = code * 2^(E - 127), NaN where E is 255.
 *  q      uint8[rows][P]  two codes to a byte, the earlier one in its low half,
 *                         at a row pitch of P = mxfp4_pitch(K) bytes: K rounded
 *                         up to 128, halved.  The codes from K on are zero.
 *  scale  uint8[mxfp4_scale_size(rows, K)]  the bytes E in tiles of 32 rows x 8
 *                         blocks, 256 bytes each, the tiles of the same rows one
 *                         after the other.  Block b of row r has the byte
 *                           ((r / 32) * ceil(K / 256) + b / 8) * 256
 *                             + (b / 4 % 2) * 128 + (r % 32) * 4 + b % 4
 *                         The bytes of blocks past a row's last are zero; those
 *                         of rows past the last may hold anything.  (A matrix
 *                         instruction takes four of a row's bytes from one
 *                         register: so a wave loads 32 rows' with one load.)
 * The encoder works on each block alone: with a the largest magnitude of its
 * elements
 *
 *     E = max(floor(log2 a) - 2, -127) + 127         (0 for a block of zeros)
 *     code = x * 2^(127 - E) rounded to the nearest magnitude, ties to the code
 *            that is even; past 6 it is 6 (a is below 8 there).  The sign is
 *            kept, that of zeros too.
 *
 * A block that holds a NaN or an infinity gets E = 255 and codes of zero: what is
 * made from it is NaN.
 */
#ifndef MXFP4_H_
#define MXFP4_H_

#include <stddef.h>
#include <stdint.h>

#include "int8.h"
#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes from one row of codes to the next (0 for K <= 0). */
int64_t mxfp4_pitch(int64_t K);

/* Bytes of the scales of a matrix (0 for rows <= 0 or K <= 0). */
int64_t mxfp4_scale_size(int64_t rows, int64_t K);

/*
 * mxfp4_quantize -- the encoder above, for activations and for weights.
 *  x             : device, rows x K values of type x_dtype, contiguous,
 *                  natural alignment.
 *  rows, K       : 0 <= rows < 2^31, 0 <= K < 2^31, and rows times K / 128
 *                  (rounded up) < 2^31.
 *  q             : device, rows * mxfp4_pitch(K) bytes, 16-byte aligned.
 *  scale         : device, mxfp4_scale_size(rows, K) bytes, 16-byte aligned.
 *                  Rows past the last are left as they were.
 * Returns NF4_EINVAL for negative sizes, an unknown type, a NULL pointer with
 * rows * K > 0 or a misaligned pointer; NF4_EUNSUPPORTED for sizes out of
 * range.
 */
nf4_status mxfp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t K, uint8_t* q,
                          uint8_t* scale, void* stream);

/*
 * mxfp4_dequant -- the values of rows x K codes, each rounded to nearest even.
 *  out           : device, rows x K values of type out_dtype, contiguous.
 * Arguments and status as for mxfp4_quantize.
 */
nf4_status mxfp4_dequant(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t K, void* out,
                         int32_t out_dtype, void* stream);

/*
 * mxfp4_gemm -- y[m][n] = sum_k x[m][k] * w[n][k] of the values of two matrices
 * in the format, for any number of rows from a single token up.
 *  xq, xs        : codes and scales of M rows (activations).
 *  wq, ws        : codes and scales of N rows (weights).
 *  M, N, K       : 0 <= M, N < 2^31; 0 <= K <= 2^20.
 *  y             : device, M x N values of type y_dtype, row-major.
 *  workspace     : DEVICE scratch of workspace_bytes bytes, 256-byte aligned,
 *                  any contents, or NULL.  With mxfp4_gemm_workspace_size bytes
 *                  the product may split K over workgroups (fp32 partial sums,
 *                  added by a second kernel).  Nothing is kept between calls;
 *                  calls that may overlap in time need separate workspaces.
 * Each product of two values is exact; they are summed in fp32 in an order that
 * follows, on a device, from M, N, K and the room in the workspace alone, and the sum
 * is rounded to y_dtype.  Sums below fp32's subnormal numbers are zeros.  K == 0
 * gives zeros.  Returns NF4_EINVAL for negative sizes, an unknown type, NULL
 * pointers with M * N > 0, codes or scales that are not 16-byte aligned, y not
 * naturally aligned, or a workspace that is not 256-byte aligned;
 * NF4_EUNSUPPORTED outside the ranges above.
 */
nf4_status mxfp4_gemm(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws,
                      int64_t M, int64_t N, int64_t K, void* y, int32_t y_dtype, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Bytes of workspace mxfp4_gemm can use on the current device (0: none). */
size_t mxfp4_gemm_workspace_size(int64_t M, int64_t N, int64_t K);

/*
 * mxfp4_linear -- mxfp4_quantize of the activations and mxfp4_gemm in one call
 * (few rows take one launch, whose order of the sums need not be mxfp4_gemm's; it
 * follows from M, N, K and the room in the workspace alone too).
 *  x, x_dtype    : device, M x K activations, contiguous, natural alignment.
 *  workspace     : DEVICE scratch, 256-byte aligned, any contents (may be NULL
 *                  where mxfp4_linear_workspace_size is 0).  Where that is not 0
 *                  the codes and scales of the M rows need M * mxfp4_pitch(K)
 *                  and mxfp4_scale_size(M, K) bytes, each rounded up to 256;
 *                  what is left is used as in mxfp4_gemm.
 * Everything else as in mxfp4_gemm; also NF4_EINVAL for a workspace without
 * room for the codes and scales.
 */
nf4_status mxfp4_linear(const void* x, int32_t x_dtype, const uint8_t* wq, const uint8_t* ws,
                        int64_t M, int64_t N, int64_t K, void* y, int32_t y_dtype, void* workspace,
                        size_t workspace_bytes, void* stream);
size_t mxfp4_linear_workspace_size(int64_t M, int64_t N, int64_t K);

/*
 * mxfp4_gemv -- y[m][n] = sum_k x[m][k] * w[n][k] with the activations as they
 * are, for 1 <= M <= 16 rows.
 *  x, x_dtype    : device, M x K activations, contiguous, natural alignment.
 *  Everything else as in mxfp4_gemm.
 * The matrix cores multiply the weights' values, which bf16 holds, with the one
 * (bf16), two (fp16) or three (fp32) bf16 numbers that an activation is the sum
 * of: each product is exact (activations below 2^-110 lose what lies under
 * 2^-133; one past fp32's range is an infinity), and they are summed in fp32.  Weights
 * of 2^128 and more (E of 253 and 254), which bf16 does not hold, are infinities here:
 * an output that one meets is infinite or NaN.  The order of the sums follows, on a
 * device, from M, N, K and x_dtype alone: a row's result does not depend on what the
 * other rows hold, but its last bits may on how many they are.  Also NF4_EINVAL for M
 * outside [0, 16].
 */
nf4_status mxfp4_gemv(const void* x, int32_t x_dtype, const uint8_t* wq, const uint8_t* ws,
                      int64_t M, int64_t N, int64_t K, void* y, int32_t y_dtype, void* stream);

/*
 * mxfp4_gemm_grouped -- the product where rows are sorted by expert and each
 * expert has weights of its own: for every sorted row i in
 * [offsets[e], offsets[e + 1])
 *
 *     y[i][n] = sum_k x[s][k] * w[e N + n][k]
 *
 * with s = order[i] / top_k (the token of a slot, as moe_sort orders them), or
 * s = i where order is NULL.  Activations are read where they lie; no copy in
 * sorted order is made.
 *  xq, xs        : codes and scales of x_rows rows.
 *  x_rows        : rows of x; a row i whose s lies outside [0, x_rows) gives
 *                  zeros, whatever its expert's weights hold.
 *  order, top_k  : device int32[rows] or NULL; top_k >= 1 (ignored for NULL).
 *  wq, ws        : codes and scales of experts * N rows.
 *  offsets       : device int32[experts + 1], ascending from 0.  Values are
 *                  clamped into [0, rows]; an expert without rows is skipped.
 *  experts       : 0 <= experts <= 1024 (0 is a no-op).
 *  rows          : rows of y and entries of order, < 2^31.
 *  N, K          : as in mxfp4_gemm; experts * N < 2^31.
 *  y             : device, rows x N values; rows that no expert has, those from
 *                  offsets[experts] on among them, are left as they were.
 * Rounding and status as in mxfp4_gemm.
 */
nf4_status mxfp4_gemm_grouped(const uint8_t* xq, const uint8_t* xs, int64_t x_rows,
                              const int32_t* order, int32_t top_k, const uint8_t* wq,
                              const uint8_t* ws, const int32_t* offsets, int32_t experts,
                              int64_t rows, int64_t N, int64_t K, void* y, int32_t y_dtype,
                              void* stream);

/*
 * mxfp4_moe_mlp -- the expert layer of a few tokens in two launches, from the
 * router's choice (made for up to about 16 tokens; with more, mxfp4_gemm_grouped, which
 * takes quantized activations, reads an expert's weights less often):
 *
 *     y[t] = sum_j weights[t][j] * W2[e] act(W1[e] x[t]),   e = ids[t][j]
 *
 * with act(v) = silu(v[0..F-1]) * v[F..2F-1] where gated, else silu(v), and
 * silu(g) = g / (1 + exp(-g)).  A slot whose id lies outside [0, experts) is
 * dropped; a token without others gives zeros.  The same expert may stand in
 * several slots of a token: their weights are added up.
 *  x, dtype      : device [T][H], contiguous; y has the same type.
 *  w1q, w1s      : experts * (gated ? 2 F : F) rows of H: of each expert the gate
 *                  channels, then the others.
 *  w2q, w2s      : experts * H rows of F.
 *  ids           : device int32 (id_bytes 4) or int64 (id_bytes 8) [T][top_k].
 *  weights       : device fp32 [T][top_k], or NULL for ones.
 *  T, top_k      : 0 <= T <= 64, 1 <= top_k <= 32.
 *  experts       : 0 <= experts <= 1024 (0 gives zeros).
 *  H, F          : 0 <= H, F <= 2^20; rows of each matrix < 2^31.
 *  workspace     : DEVICE scratch, 256-byte aligned, any contents, of at least
 *                  mxfp4_moe_mlp_workspace_size bytes.
 * Activations and weights meet as in mxfp4_gemv.  What lies between the two
 * products is computed in fp32, multiplied by the router's weight and kept as the
 * sum of two bf16 numbers (16 bits; three, so all of fp32, where dtype is fp32).
 * The order of every sum follows, on a device, from the sizes, the type and the ids
 * alone.  Returns
 * NF4_EINVAL for negative sizes, another id_bytes, an unknown type, NULL or
 * misaligned pointers or a workspace that is too small; NF4_EUNSUPPORTED outside
 * the ranges above.
 */
nf4_status mxfp4_moe_mlp(const void* x, int32_t dtype, const uint8_t* w1q, const uint8_t* w1s,
                         const uint8_t* w2q, const uint8_t* w2s, const void* ids, int32_t id_bytes,
                         const float* weights, int64_t T, int32_t top_k, int32_t experts, int64_t H,
                         int64_t F, int32_t gated, void* y, void* workspace, size_t workspace_bytes,
                         void* stream);
/* Bytes of workspace mxfp4_moe_mlp needs on the current device. */
size_t mxfp4_moe_mlp_workspace_size(int64_t T, int32_t top_k, int32_t experts, int64_t H, int64_t F,
                                    int32_t dtype);

#ifdef __cplusplus
} /* extern "C" */
#endif
#endif /* MXFP4_H_ */
