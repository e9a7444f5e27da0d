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

// A workgroup takes a tile of the scales at a time, 32 rows x 256 elements, so that it
// writes its 256 bytes of them whole.  Sixteen lanes take a group of 128 elements of a row,
// eight each: four lanes a block, and one lane the group's four scales; a thread has four
// groups' loads in flight.  Bound by memory: 4097 x 11008 bf16 takes 19.4 us (5.9 TB/s), and
// back 19.0 (a copy of 1 GiB runs at 5.2); 1 x 4096 2.4, a launch's.
constexpr int kPasses = 4, kRowsAtOnce = kThreads / 32;  // rows of a pass
static_assert(kPasses * kRowsAtOnce == 32);

template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ x, uint32_t tiles, uint32_t steps,
                                                            int64_t rows, int64_t K, int64_t pitch,
                                                            uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  const int in = threadIdx.x & 15, half = threadIdx.x >> 4 & 1;
  for (uint32_t i = blockIdx.x; i < tiles; i += gridDim.x) {
    const uint32_t band = i / steps, step = i - band * steps;
    const int64_t row0 = int64_t(32) * band + (threadIdx.x >> 5), at = int64_t(256) * step + 128 * half + 8 * in;
    Piece<DT> v[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int64_t row = row0 + kRowsAtOnce * k;
      const char* xr = static_cast<const char*>(x) + row * K * dtype_bytes(DT);
      v[k] = Piece<DT>{};
      if (row < rows) {
        if (at + 8 <= K)
          v[k] = whole_piece<DT, true>(xr, at);
        else if (at < K)
          v[k] = load_piece<DT>(xr, at, K);
      }
    }
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int64_t row = row0 + kRowsAtOnce * k;
      if (row >= rows) break;
      uint32_t m = piece_peak<DT>(v[k]);
      m = max(m, dpp<0xB1>(m));  // the neighbour
      m = max(m, dpp<0x4E>(m));  // the other pair of the four
      const uint32_t e = block_scale(m);
      // (a last tile's second half may lie past the row's pitch; its scales are zeros)
      if (at < 2 * pitch) *reinterpret_cast<uint32_t*>(q + row * pitch + at / 2) = encode_piece<DT>(v[k], e);
      // the scales of the four blocks in the first lane: lane 4 to 0 and 12 to 8, then 8 to 0
      uint32_t s = e | dpp<0x104>(e) << 8;  // (row shift left by 4)
      s |= dpp<0x108>(s) << 16;             // (by 8)
      if (in == 0)
        *reinterpret_cast<uint32_t*>(scale + static_cast<int64_t>(i) * 256 + 128 * half + 4 * (row & 31)) = s;
    }
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void dequant_kernel(const uint8_t* __restrict__ q,
                                                           const uint8_t* __restrict__ scale, uint32_t tiles,
                                                           uint32_t steps, int64_t rows, int64_t K, int64_t pitch,
                                                           void* __restrict__ out) {
  const int in = threadIdx.x & 15, half = threadIdx.x >> 4 & 1;
  for (uint32_t i = blockIdx.x; i < tiles; i += gridDim.x) {
    const uint32_t band = i / steps, step = i - band * steps;
    const int64_t row0 = int64_t(32) * band + (threadIdx.x >> 5), at = int64_t(256) * step + 128 * half + 8 * in;
    if (at >= K) continue;
    uint32_t c[kPasses], e[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int64_t row = row0 + kRowsAtOnce * k;
      c[k] = e[k] = 0;
      if (row >= rows) continue;
      c[k] = *reinterpret_cast<const uint32_t*>(q + row * pitch + at / 2);
      e[k] = scale[static_cast<int64_t>(i) * 256 + 128 * half + 4 * (row & 31) + in / 4];
    }
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int64_t row = row0 + kRowsAtOnce * k;
      if (row >= rows) break;
      const float s = scale_value(e[k]);
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], s, 0),
                  b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], s, 1),
                  d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], s, 2),
                  g = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], s, 3);
      const float f[8] = {a[0], a[1], b[0], b[1], d[0], d[1], g[0], g[1]};
      store_piece<DT>(static_cast<char*>(out) + row * K * dtype_bytes(DT), at, K, make_piece<DT>(f));
    }
  }
}

// The tiles of a matrix, which 31 bits hold (too_large), and the workgroups for them.
uint32_t tiles_of(int64_t rows, int64_t K) { return static_cast<uint32_t>((rows + 31) / 32 * steps_of(K)); }
uint32_t groups_for(uint32_t tiles) { return tiles < kMaxGroups ? tiles : kMaxGroups; }

// The groups of a matrix, counted in 31 bits.
bool too_large(int64_t rows, int64_t K) {
  return rows > kMaxDim || K > kMaxDim || (K + 127) / 128 > kMaxDim / rows;
}

}  // namespace

namespace mxdev {

void quantize_launch(const void* x, int32_t dt, int64_t rows, int64_t K, uint8_t* q, uint8_t* scale,
                     hipStream_t st) {
  const uint32_t tiles = tiles_of(rows, K);
  with_dtype(dt, [&](auto t) {
    hipLaunchKernelGGL((quantize_kernel<decltype(t)::value>), dim3(groups_for(tiles)), dim3(kThreads), 0, st, x, tiles,
                       static_cast<uint32_t>(steps_of(K)), rows, K, pitch_of(K), q, scale);
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
  const uint32_t tiles = tiles_of(rows, K);
  with_dtype(out_dtype, [&](auto t) {
    hipLaunchKernelGGL((dequant_kernel<decltype(t)::value>), dim3(groups_for(tiles)), dim3(kThreads), 0,
                       reinterpret_cast<hipStream_t>(stream), q, scale, tiles, static_cast<uint32_t>(steps_of(K)), rows,
                       K, pitch_of(K), out);
  });
  return launch_status();
}

}  // extern "C"
