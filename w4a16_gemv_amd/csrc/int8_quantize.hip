// int8_quantize.hip -- the int8 encoder (activations per token, weights per
// output channel) and its inverse.
//
// Encoder, per row: a = max(max|x|, 2^-100), scale = a / 127 and inverse =
// 127 / a (both correctly rounded), code = x * inverse rounded half to even.
// The rounding is one FMA: x * inverse + 1.5 * 2^23 has its last bit at one,
// so the fused product and sum round the exact product to an integer, ties to
// even, and the low byte of the result is the code.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "int8.h"
#include "int8_product.h"
#include "nf4_device.h"
#include "row_io.h"

namespace {

using namespace nf4dev;
using namespace rowio;
using namespace int8dev;

constexpr int kThreads = 256;

// A grid may not have 2^32 threads: beyond this many rows a workgroup takes
// several.
constexpr int64_t kMaxGroups = 1 << 20;

uint32_t groups_for(int64_t rows) { return static_cast<uint32_t>(rows < kMaxGroups ? rows : kMaxGroups); }

// A workgroup per row: one pass for the maximum, one for the codes (the row
// comes from the caches the second time).
template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const void* __restrict__ x,
                                                                 int64_t rows, int64_t K,
                                                                 int64_t pitch,
                                                                 int8_t* __restrict__ q,
                                                                 float* __restrict__ scale) {
  __shared__ uint32_t s_max[kThreads / 64];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
  const char* xr = static_cast<const char*>(x) + row * K * dtype_bytes(DT);
  uint32_t m = 0;
  for (int64_t at = 8 * threadIdx.x; at < K; at += 8 * kThreads)
    m = max(m, piece_peak<DT>(load_piece<DT>(xr, at, K)));
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) m = max(m, s_max[i]);
  const RowScale s = row_scale(m);
  if (threadIdx.x == 0) scale[row] = s.scale;
  int8_t* qr = q + row * pitch;
  for (int64_t at = 8 * threadIdx.x; at < pitch; at += 8 * kThreads)
    *reinterpret_cast<uint2*>(qr + at) = encode_piece<DT>(load_piece<DT>(xr, at, K), s);
  __syncthreads();  // s_max is read before the next row's
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void dequant_rows_kernel(const int8_t* __restrict__ q,
                                                                const float* __restrict__ scale,
                                                                int64_t rows, int64_t K,
                                                                int64_t pitch,
                                                                void* __restrict__ out) {
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
  const float s = scale[row];
  char* o = static_cast<char*>(out) + row * K * dtype_bytes(DT);
  for (int64_t at = 8 * threadIdx.x; at < K; at += 8 * kThreads) {
    const uint2 c = *reinterpret_cast<const uint2*>(q + row * pitch + at);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = static_cast<float>(static_cast<int8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)))) * s;
    store_piece<DT>(o, at, K, make_piece<DT>(f));
  }
  }
}

}  // namespace

namespace int8dev {

void quantize_launch(const void* x, int32_t dt, int64_t rows, int64_t K, int8_t* q, float* scale,
                     hipStream_t st) {
  with_dtype(dt, [&](auto t) {
    hipLaunchKernelGGL((quantize_rows_kernel<decltype(t)::value>), dim3(groups_for(rows)),
                       dim3(kThreads), 0, st, x, rows, K, pitch_of(K), q, scale);
  });
}

}  // namespace int8dev

extern "C" {

int64_t int8_pitch(int64_t K) { return int8dev::pitch_of(K); }

nf4_status int8_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t K, int8_t* q,
                         float* scale, void* stream) {
  if (rows < 0 || K < 0 || !known_dtype(x_dtype)) return NF4_EINVAL;
  if (rows == 0) return NF4_OK;
  if ((K > 0 && (!x || !q)) || !scale) return NF4_EINVAL;
  if (!aligned(x, dtype_bytes(x_dtype)) || !aligned(q, 16) || !aligned(scale, 4)) return NF4_EINVAL;
  if (rows > kMaxDim || K > kMaxDim) return NF4_EUNSUPPORTED;
  quantize_launch(x, x_dtype, rows, K, q, scale, reinterpret_cast<hipStream_t>(stream));
  return launch_status();
}

nf4_status int8_dequant(const int8_t* q, const float* scale, int64_t rows, int64_t K, void* out,
                        int32_t out_dtype, void* stream) {
  if (rows < 0 || K < 0 || !known_dtype(out_dtype)) return NF4_EINVAL;
  if (rows == 0 || K == 0) return NF4_OK;
  if (!q || !scale || !out) return NF4_EINVAL;
  if (!aligned(out, dtype_bytes(out_dtype)) || !aligned(q, 16) || !aligned(scale, 4))
    return NF4_EINVAL;
  if (rows > kMaxDim || K > kMaxDim) return NF4_EUNSUPPORTED;
  with_dtype(out_dtype, [&](auto t) {
    hipLaunchKernelGGL((dequant_rows_kernel<decltype(t)::value>), dim3(groups_for(rows)),
                       dim3(kThreads), 0, reinterpret_cast<hipStream_t>(stream), q, scale, rows, K,
                       pitch_of(K), out);
  });
  return launch_status();
}

}  // extern "C"
