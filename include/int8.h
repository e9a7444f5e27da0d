/*
 * int8.h -- C ABI of the 8-bit integer products in libnf4 (W8A8): activations
 * quantized per token, weights quantized per output channel, int32 sums, on
 * AMD Instinct MI355X (gfx950).  Status codes and all conventions (device
 * pointers owned by the caller, asynchronous work on `stream`, synchronous
 * argument validation, no allocation, thread safety) are those of nf4.h.  What a
 * call writes (results, workspace) must not overlap what it reads.
 *
 * ---------------------------------------------------------------------------
 * The format (a matrix of `rows` rows of K elements: one token's activations
 * or one output channel's weights per row)
 * ---------------------------------------------------------------------------
 *  q      int8[rows][P]  codes at a row pitch of P = int8_pitch(K) bytes, K
 *                        rounded up to 64.  The P - K padding bytes of a row
 *                        are zero (int8_quantize writes them so); a product
 *                        is right as long as one of its operands has them
 *                        zero.
 *  scale  fp32[rows]
 *  value  = fp32(q * scale[row])
 * The encoder works on each row alone:
 *
 *     a       = max(max_k |x_k|, 2^-100)
 *     scale   = a * (1 / 127),  inverse = 127 * (1 / a)   each step in fp32
 *     q_k     = x_k * inverse rounded to the nearest integer, ties to even
 *               (the product is not rounded before)
 *
 * so |q| <= 127, a row of zeros has zero codes, and both scale and inverse are
 * normal numbers.  They are not the quotients' nearest numbers but the ones that
 * tensor expressions for a / 127 and 127 / a give on the device, within two
 * roundings, (1 + 2^-24)^2, of the quotients; past a = 2^126, where 1 / a is
 * subnormal, the inverse is within 2^-21.  So each code is within 1/2 + 2^-16 of
 * 127 x_k / a (1/2 + 2^-14 there) and each value within (1/2 + 2^-14) a / 127 of
 * x_k (1/2 + 2^-13).  A row that holds a NaN or an infinity gets the scale NaN
 * and zero codes: every output made from that row is NaN, and no other is.
 */
#ifndef INT8_H_
#define INT8_H_

#include <stddef.h>
#include <stdint.h>

#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of the unquantized side; the first two equal nf4_dtype's. */
typedef enum { INT8_BF16 = 0, INT8_FP16 = 1, INT8_FP32 = 2 } int8_dtype;

/* Bytes from one row of codes to the next: K rounded up to 64 (0 for K <= 0). */
int64_t int8_pitch(int64_t K);

/*
 * int8_quantize -- the encoder above, for activations and for weights.
 *  x             : device, rows x K values of type x_dtype, contiguous,
 *                  natural alignment.
 *  rows, K       : 0 <= rows < 2^31, 0 <= K < 2^31.
 *  q             : device, rows * int8_pitch(K) bytes, 16-byte aligned.
 *  scale         : device, rows floats.
 * Returns NF4_EINVAL for negative sizes, an unknown type, a NULL pointer with
 * rows * K > 0 or a misaligned pointer; NF4_EUNSUPPORTED for sizes out of
 * range.
 */
nf4_status int8_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t K, int8_t* q,
                         float* scale, void* stream);

/*
 * int8_dequant -- the values of rows x K codes, each rounded to nearest even.
 *  out           : device, rows x K values of type out_dtype, contiguous.
 * Arguments and status as for int8_quantize.
 */
nf4_status int8_dequant(const int8_t* q, const float* scale, int64_t rows, int64_t K, void* out,
                        int32_t out_dtype, void* stream);

/*
 * int8_gemm -- y[m][n] = (sum_k xq[m][k] * wq[n][k]) * xs[m] * ws[n], for any
 * number of rows from a single token up.
 *  xq, xs        : codes and scales of M rows (activations).
 *  wq, ws        : codes and scales of N rows (weights).
 *  M, N, K       : 0 <= M, N < 2^31; 0 <= K <= 131071, which keeps the int32
 *                  sums exact for every pair of codes (K * 128 * 128 < 2^31).
 *  y             : device, M x N values of type y_dtype, row-major.
 *  workspace     : DEVICE scratch of workspace_bytes bytes, 256-byte aligned,
 *                  any contents, or NULL.  With int8_gemm_workspace_size bytes
 *                  the product may split K over workgroups (int32 partial sums,
 *                  added by a second kernel).  Integer sums do not depend on
 *                  the split: the bits are those of a NULL-workspace call.
 *                  Nothing is kept between calls; calls that may overlap in
 *                  time need separate workspaces.
 * The sum is exact; it is converted to fp32, multiplied by xs[m], then by
 * ws[n] (three fp32 roundings) and rounded to y_dtype.  Where the product with
 * xs[m] and the one with ws[n] are both normal fp32 numbers (or the sum is 0),
 * each output is within (1 + 2^-24)^3 of the exact value, relative, before
 * that last rounding.  A product with xs[m] past fp32's range is an infinity
 * whatever ws[n] is, and one below its normal range is a subnormal number, with
 * the bits that those have.
 * K == 0 gives the sums 0.  Returns NF4_EINVAL for negative sizes, an unknown
 * type, NULL pointers with M * N > 0, codes that are not 16-byte aligned,
 * scales or y not naturally aligned, or a workspace that is not 256-byte
 * aligned; NF4_EUNSUPPORTED outside the ranges above.
 */
nf4_status int8_gemm(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                     int64_t M, int64_t N, int64_t K, void* y, int32_t y_dtype, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Bytes of workspace int8_gemm can use on the current device (0: none). */
size_t int8_gemm_workspace_size(int64_t M, int64_t N, int64_t K);

/*
 * int8_linear -- int8_quantize of the activations followed by int8_gemm, with
 * the bits of those two calls (few rows take one launch instead of two).
 *  x, x_dtype    : device, M x K activations, contiguous, natural alignment.
 *  workspace     : DEVICE scratch, 256-byte aligned, any contents (may be NULL
 *                  where int8_linear_workspace_size is 0).  The codes and
 *                  scales of the M rows need M * int8_pitch(K) bytes and
 *                  4 * M, each rounded up to 256; what is left is used as in
 *                  int8_gemm.  int8_linear_workspace_size bytes hold all that
 *                  the product can use, and a workspace for one shape is large
 *                  enough for every shape with no more rows and no larger K,
 *                  without changing its bits.
 * Everything else as in int8_gemm; also NF4_EINVAL for a workspace without
 * room for the codes and scales.
 */
nf4_status int8_linear(const void* x, int32_t x_dtype, const int8_t* wq, const float* ws,
                       int64_t M, int64_t N, int64_t K, void* y, int32_t y_dtype, void* workspace,
                       size_t workspace_bytes, void* stream);
size_t int8_linear_workspace_size(int64_t M, int64_t N, int64_t K);

/*
 * int8_gemm_grouped -- the product where rows are sorted by expert and each
 * expert has weights of its own: for every sorted row i in
 * [offsets[e], offsets[e + 1])
 *
 *     y[i][n] = (sum_k xq[s][k] * wq[e][n][k]) * xs[s] * ws[e][n]
 *
 * with s = order[i] / top_k (the token of a slot, as moe_sort orders them), or
 * s = i where order is NULL.  Activations are read where they lie; no copy in
 * sorted order is made.
 *  xq, xs        : codes and scales of x_rows rows.
 *  x_rows        : rows of xq; a row i whose s lies outside [0, x_rows) gives
 *                  zeros, whatever its expert's scales hold.
 *  order, top_k  : device int32[rows] or NULL; top_k >= 1 (ignored for NULL).
 *  wq, ws        : codes and scales of experts * N rows.
 *  offsets       : device int32[experts + 1], ascending from 0.  Values are
 *                  clamped into [0, rows]; an expert without rows is skipped.
 *  experts       : 0 <= experts <= 1024 (0 is a no-op).
 *  rows          : rows of y and entries of order, < 2^31.
 *  N, K          : as in int8_gemm.
 *  y             : device, rows x N values; rows that no expert has, those from
 *                  offsets[experts] on among them, are left as they were.
 * Rounding and status as in int8_gemm.  y must not overlap the inputs.
 */
nf4_status int8_gemm_grouped(const int8_t* xq, const float* xs, int64_t x_rows,
                             const int32_t* order, int32_t top_k, const int8_t* wq,
                             const float* ws, const int32_t* offsets, int32_t experts,
                             int64_t rows, int64_t N, int64_t K, void* y, int32_t y_dtype,
                             void* stream);

#ifdef __cplusplus
} /* extern "C" */
#endif
#endif /* INT8_H_ */
