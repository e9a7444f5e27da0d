/*
 * nf4_probe.h -- bandwidth probes of libnf4 and a query of its choice of kernels
 * (measurement and test helpers, not part of the NF4 method).  The probes move
 * bytes with the same access patterns as the hot path's kernels and no
 * arithmetic, so that the hot path's achieved bandwidth can be set against what
 * plain streaming reaches on the same GPU.
 * Device pointers; asynchronous on `stream`; they allocate nothing.
 */
#ifndef NF4_PROBE_H_
#define NF4_PROBE_H_

#include <stddef.h>
#include <stdint.h>

#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * nf4_probe_stream_read -- reads `bytes` bytes at src once (16-byte streaming
 * loads, one contiguous range per wave, four loads in flight per lane: the
 * GEMV's weight stream without the decode).  Writes one dword to *sink only
 * for a data pattern that does not occur in practice (it keeps the loads
 * alive).  src 16-byte aligned, bytes a multiple of 16; sink 4 bytes.
 * Returns NF4_EINVAL for NULL or misaligned pointers or sizes.
 */
nf4_status nf4_probe_stream_read(const void* src, size_t bytes, uint32_t* sink, void* stream);

/*
 * nf4_probe_expand_copy -- reads `src_bytes` bytes and writes four times as
 * many: dst dword-quad i = (w, w ^ 1, w ^ 2, w ^ 3) for w = src dword i,
 * with 16-byte streaming stores (the dequant's 1 : 4 read : write stream
 * without the decode).  src 4-byte aligned, dst 16-byte aligned, src_bytes a
 * multiple of 4.  Returns NF4_EINVAL for NULL or misaligned pointers or sizes.
 */
nf4_status nf4_probe_expand_copy(const void* src, size_t src_bytes, void* dst, void* stream);

/*
 * nf4_probe_int8_plan -- which kernel an int8 product of these sizes goes to on
 * the current device (on 256 compute units where there is none); nothing is
 * launched.  Tests use it to show that their sizes reach every variant.
 *  M, N, K, experts : sizes as in int8_gemm (experts 0; M, N >= 1) or, with
 *                  M rows, in int8_gemm_grouped.
 *  room          : bytes of workspace (int8_gemm).
 *  plan          : host; -2 the one- and two-token kernel, -1 the few-row
 *                  kernel, 0-5 tiles, by size.
 *  detail        : host; the variant: blocks of 1024 bytes to a row (-2), units
 *                  of 64 bytes to a wave (-1), in how many pieces K is split
 *                  (0-4 and grouped), or a sum of 1 (whole tiles), 2 (a last
 *                  turn in halves) and 4 (in quarters) (5).
 * Returns NF4_EINVAL for a NULL pointer or bad sizes, NF4_EUNSUPPORTED for
 * sizes that the products refuse.
 */
nf4_status nf4_probe_int8_plan(int64_t M, int64_t N, int64_t K, int32_t experts, size_t room,
                               int32_t* plan, int32_t* detail);

/*
 * nf4_probe_mxfp4_plan -- the same of the products of 4-bit microscaled floats:
 * plan -1 the few-row kernel (detail: units of 64 bytes of codes to a wave where eight
 * share a row, minus the waves that do where fewer do), 0-5 tiles by size (detail as
 * above).  experts -1 is mxfp4_linear's, which encodes few rows on the way.
 */
nf4_status nf4_probe_mxfp4_plan(int64_t M, int64_t N, int64_t K, int32_t experts, size_t room,
                                int32_t* plan, int32_t* detail);

/*
 * nf4_probe_mxfp4_rows -- how mxfp4_moe_mlp takes sizes (T, top_k, experts, H, F and
 * dtype as there) or, with experts 0, mxfp4_gemv (T rows of H, F channels).
 *  plan          : host int32[5]; the waves that share a row's K and the units of 128
 *                  elements that each takes at a time; the elements of a row in LDS at a
 *                  time (less than H: in turns; 0: mxfp4_gemv's rows that do not fit); the
 *                  rows at a time; the variant of the way down (-1: mxfp4_gemv; 0 eight
 *                  channels to a workgroup; four rows of an expert at a time for up to 16
 *                  tokens (1) and for more (2); sixteen likewise (3, 4)).
 * Status as for nf4_probe_mxfp4_plan.
 */
nf4_status nf4_probe_mxfp4_rows(int64_t T, int32_t top_k, int32_t experts, int64_t H, int64_t F,
                                int32_t dtype, int32_t* plan);

#ifdef __cplusplus
}
#endif

#endif /* NF4_PROBE_H_ */
