// mxfp4_quantize.hip -- the encoder of the 4-bit microscaled floats and its
// inverse.
//
// Encoder, per block of 32: E - 127 = floor(log2 max|x|) - 2, the exponent field of
// the largest magnitude, and code = x / 2^(E - 127) rounded to E2M1, which is one
// instruction for two values (v_cvt_scalef32_pk_fp4_*).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxfp4.h"
#include "mxfp4_format.h"
#include "nf4_device.h"
#include "row_io.h"

namespace {

using namespace nf4dev;
using namespace rowio;
using namespace mxdev;

constexpr int kThreads = 256;
constexpr uint32_t kMaxGroups = 1 << 20;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true));
}

// Sixteen lanes take a group of 128 elements of a row, eight each: four lanes a
// block, and one lane the group's four scales.
template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ x, uint32_t all, uint32_t groups,
                                                            int64_t K, uint8_t* __restrict__ q,
                                                            uint8_t* __restrict__ scale) {
  const int in = threadIdx.x & 15;
  for (uint32_t i = blockIdx.x * (kThreads / 16) + threadIdx.x / 16; i < all; i += gridDim.x * (kThreads / 16)) {
    const uint32_t row = i / groups, group = i - row * groups;
    const char* xr = static_cast<const char*>(x) + row * K * dtype_bytes(DT);
    const int64_t at = int64_t(128) * group + 8 * in;
    Piece<DT> v = {};
    if (at + 8 <= K)
      v = whole_piece<DT, true>(xr, at);
    else if (at < K)
      v = load_piece<DT>(xr, at, K);
    uint32_t m = piece_peak<DT>(v);
    m = max(m, dpp<0xB1>(m));  // the neighbour
    m = max(m, dpp<0x4E>(m));  // the other pair of the four
    const uint32_t e = block_scale(m);
    *reinterpret_cast<uint32_t*>(q + static_cast<int64_t>(i) * 64 + 4 * in) = encode_piece<DT>(v, e);
    // the scales of the four blocks in the first lane: lane 4 to 0 and 12 to 8, then 8 to 0
    uint32_t s = e | dpp<0x104>(e) << 8;  // (row shift left by 4)
    s |= dpp<0x108>(s) << 16;             // (by 8)
    if (in == 0) *reinterpret_cast<uint32_t*>(scale + scale_at(row, (groups + 1) / 2, group)) = s;
    // the other half of a last tile that is half full
    if (in == 1 && group + 1 == groups && (groups & 1))
      *reinterpret_cast<uint32_t*>(scale + scale_at(row, (groups + 1) / 2, groups)) = 0;
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void dequant_kernel(const uint8_t* __restrict__ q,
                                                           const uint8_t* __restrict__ scale, uint32_t all,
                                                           uint32_t groups, int64_t K, void* __restrict__ out) {
  const int in = threadIdx.x & 15;
  for (uint32_t i = blockIdx.x * (kThreads / 16) + threadIdx.x / 16; i < all; i += gridDim.x * (kThreads / 16)) {
    const uint32_t row = i / groups, group = i - row * groups;
    const int64_t at = int64_t(128) * group + 8 * in;
    if (at >= K) continue;
    const uint32_t c = *reinterpret_cast<const uint32_t*>(q + static_cast<int64_t>(i) * 64 + 4 * in);
    const float s = scale_value(scale[scale_at(row, (groups + 1) / 2, group) + in / 4]);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
    const float f[8] = {a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
    store_piece<DT>(static_cast<char*>(out) + row * K * dtype_bytes(DT), at, K, make_piece<DT>(f));
  }
}

uint32_t grid_for(int64_t all) {
  const int64_t n = (all + kThreads / 16 - 1) / (kThreads / 16);
  return static_cast<uint32_t>(n < kMaxGroups ? n : kMaxGroups);
}

// The groups of a matrix, counted in 31 bits.
bool too_large(int64_t rows, int64_t K) {
  return rows > kMaxDim || K > kMaxDim || (K + 127) / 128 > kMaxDim / rows;
}

}  // namespace

namespace mxdev {

void quantize_launch(const void* x, int32_t dt, int64_t rows, int64_t K, uint8_t* q, uint8_t* scale,
                     hipStream_t st) {
  const int64_t groups = (K + 127) / 128, all = rows * groups;
  with_dtype(dt, [&](auto t) {
    hipLaunchKernelGGL((quantize_kernel<decltype(t)::value>), dim3(grid_for(all)), dim3(kThreads), 0, st, x,
                       static_cast<uint32_t>(all), static_cast<uint32_t>(groups), K, q, scale);
  });
}

}  // namespace mxdev

extern "C" {

int64_t mxfp4_pitch(int64_t K) { return mxdev::pitch_of(K); }

int64_t mxfp4_scale_size(int64_t rows, int64_t K) { return mxdev::scale_bytes(rows, K); }

nf4_status mxfp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t K, uint8_t* q,
                          uint8_t* scale, void* stream) {
  if (rows < 0 || K < 0 || !known_dtype(x_dtype)) return NF4_EINVAL;
  if (rows == 0 || K == 0) return NF4_OK;
  if (!x || !q || !scale) return NF4_EINVAL;
  if (!aligned(x, dtype_bytes(x_dtype)) || !aligned(q, 16) || !aligned(scale, 16)) return NF4_EINVAL;
  if (too_large(rows, K)) return NF4_EUNSUPPORTED;
  quantize_launch(x, x_dtype, rows, K, q, scale, reinterpret_cast<hipStream_t>(stream));
  return launch_status();
}

nf4_status mxfp4_dequant(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t K, void* out,
                         int32_t out_dtype, void* stream) {
  if (rows < 0 || K < 0 || !known_dtype(out_dtype)) return NF4_EINVAL;
  if (rows == 0 || K == 0) return NF4_OK;
  if (!q || !scale || !out) return NF4_EINVAL;
  if (!aligned(out, dtype_bytes(out_dtype)) || !aligned(q, 16) || !aligned(scale, 16)) return NF4_EINVAL;
  if (too_large(rows, K)) return NF4_EUNSUPPORTED;
  const int64_t groups = (K + 127) / 128, all = rows * groups;
  with_dtype(out_dtype, [&](auto t) {
    hipLaunchKernelGGL((dequant_kernel<decltype(t)::value>), dim3(grid_for(all)), dim3(kThreads), 0,
                       reinterpret_cast<hipStream_t>(stream), q, scale, static_cast<uint32_t>(all),
                       static_cast<uint32_t>(groups), K, out);
  });
  return launch_status();
}

}  // extern "C"
