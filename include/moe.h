/*
 * moe.h -- C ABI of the routing around expert products in libnf4: token slots
 * sorted by expert, rows moved into that order and back with the router's
 * weights, and the gradients, on AMD Instinct MI355X (gfx950).  Status codes
 * and all conventions (device pointers owned by the caller, asynchronous work
 * on `stream`, synchronous argument validation, no allocation, thread safety)
 * are those of nf4.h; the row types are int8.h's int8_dtype.
 *
 * A batch has T tokens with top_k slots each; slot (t, j) is the flat index
 * t * top_k + j and names an expert in [0, experts).  A slot with any other
 * id (padding, an expert of another rank) is dropped: it has no row.  The
 * same expert may stand in several slots of a token.
 *
 *  offsets  int32[experts + 1]  expert e has the sorted rows
 *                               [offsets[e], offsets[e + 1]); offsets[0] = 0.
 *  order    int32[T * top_k]    the flat slot of each sorted row, ascending
 *                               within an expert; -1 from offsets[experts] on.
 *  pos      int32[T][top_k]     the sorted row of each slot, -1 if dropped.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#include "int8.h"
#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_sort -- offsets, order and pos of the slots' expert ids.
 *  ids           : device int32 (id_bytes 4) or int64 (id_bytes 8) [T][top_k].
 *  T, top_k      : T >= 0, top_k >= 1, T * top_k <= 2^30.
 *  experts       : 0 <= experts <= 1024.
 *  workspace     : DEVICE scratch, 256-byte aligned, any contents, of at least
 *                  moe_sort_workspace_size bytes (may be NULL where that is 0).
 * The order is that of a stable sort; nothing depends on timing.  Returns
 * NF4_EINVAL for negative sizes, another id_bytes, NULL or misaligned
 * pointers or a workspace that is too small; NF4_EUNSUPPORTED outside the
 * ranges above.  T == 0 fills offsets with zeros.
 */
nf4_status moe_sort(const void* ids, int32_t id_bytes, int64_t T, int32_t top_k, int32_t experts,
                    int32_t* offsets, int32_t* order, int32_t* pos, void* workspace,
                    size_t workspace_bytes, void* stream);
size_t moe_sort_workspace_size(int64_t T, int32_t top_k, int32_t experts);

/*
 * moe_gather -- xs[pos[t][j]] = x[t] for every slot that has a row.
 *  x             : device [T][H] of type dtype, contiguous.
 *  pos           : device int32 [T][top_k]; entries outside [0, rows) are
 *                  dropped slots.
 *  rows          : rows of xs.  Rows that no slot names are left as they were;
 *                  a row that two slots name (moe_sort gives none) holds
 *                  values of either.
 *  H             : 0 <= H < 2^31.
 * xs must not overlap x.  Returns NF4_EINVAL for negative sizes, an unknown
 * type, NULL or misaligned pointers; NF4_EUNSUPPORTED for T * top_k > 2^30 or
 * sizes out of range.
 */
nf4_status moe_gather(const void* x, int32_t dtype, const int32_t* pos, int64_t T, int32_t top_k,
                      int64_t rows, int64_t H, void* xs, void* stream);

/*
 * moe_combine -- y[t] = sum_j weights[t][j] * ys[pos[t][j]], dropped slots left
 * out (a token without rows gives zeros).  The sum is a chain of fp32 FMAs
 * from 0, j ascending; the result is rounded once to dtype.
 *  weights       : device fp32 [T][top_k], or NULL for ones: then it is the
 *                  gradient of moe_gather (ys the gradient of xs, y that of x).
 *  ys, y         : device [rows][H] and [T][H] of type dtype; must not overlap.
 * Arguments and status as for moe_gather.
 */
nf4_status moe_combine(const void* ys, int32_t dtype, const float* weights, const int32_t* pos,
                       int64_t T, int32_t top_k, int64_t rows, int64_t H, void* y, void* stream);

/*
 * moe_combine_grad -- the gradients of moe_combine: for every slot with a row
 *     dys[pos[t][j]] = weights[t][j] * dy[t]        (rounded once to dtype)
 *     dweights[t][j] = sum_h ys[pos[t][j]][h] * dy[t][h]     (fp32 sums)
 * and dweights = 0 for a dropped slot; rows of dys that no slot names, or two,
 * are as in moe_gather.  The order of each sum follows from T and H alone.
 *  dy            : device [T][H];  ys, dys : device [rows][H]; of type dtype.
 *  weights       : device fp32 [T][top_k], or NULL for ones.
 *  dys, dweights : either may be NULL (not wanted); ys is read only for
 *                  dweights and may be NULL without it.
 * The buffers must not overlap.  Arguments and status as for moe_gather.
 */
nf4_status moe_combine_grad(const void* dy, const void* ys, int32_t dtype, const float* weights,
                            const int32_t* pos, int64_t T, int32_t top_k, int64_t rows, int64_t H,
                            void* dys, float* dweights, void* stream);

#ifdef __cplusplus
} /* extern "C" */
#endif
#endif /* MOE_H_ */
