// mxfp4_format.h -- where the codes and scales of the 4-bit microscaled floats
// lie, and the conversions of the hardware to and from them (private to libnf4).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8.h"
#include "mxfp4.h"
#include "nf4_device.h"
#include "row_io.h"

namespace mxdev {

constexpr int64_t kMaxDim = 0x7FFFFFFF;
constexpr int64_t kMaxK = 1 << 20;  // of the products: 256 rows of codes are 2^27 bytes

// Rows of whole matrix instructions' depth (128 codes), 64 bytes each: 16-byte
// loads at every K.
__device__ __host__ inline int64_t pitch_of(int64_t K) { return K > 0 ? (K + 127) / 128 * 64 : 0; }
// Tiles of scales along K.
__device__ __host__ inline int64_t steps_of(int64_t K) { return K > 0 ? (K + 255) / 256 : 0; }
__device__ __host__ inline int64_t scale_bytes(int64_t rows, int64_t K) {
  return rows > 0 ? (rows + 31) / 32 * steps_of(K) * 256 : 0;
}

// Byte of the four scales of row's codes 128 group .. 128 group + 127, `steps`
// tiles to 32 rows.
__device__ __forceinline__ int64_t scale_at(int64_t row, int64_t steps, int64_t group) {
  return ((row >> 5) * steps + (group >> 1)) * 256 + (group & 1) * 128 + (row & 31) * 4;
}

// 2^(E - 127) as the conversions take it: they see the exponent field alone, and with the
// mantissa's first bit that is a NaN for 255 and 2^-127 for 0.
__device__ __forceinline__ float scale_value(uint32_t e) {
  return __builtin_bit_cast(float, e << 23 | 0x00400000u);
}

// E of a block whose largest magnitude has these bits: the exponent field less two;
// subnormal numbers have the field 0.
__device__ __forceinline__ uint32_t block_scale(uint32_t peak) {
  const uint32_t field = peak >> 23;
  return field == 255 ? 255u : field < 2 ? 0u : field - 2;
}

// Eight values of a block to eight codes.  The conversion divides by the scale,
// rounds ties to even and saturates, on exact values; in a block that is not finite
// the codes are zeros.
template <int DT>
__device__ __forceinline__ uint32_t encode_piece(const rowio::Piece<DT>& p, uint32_t e) {
  const float s = scale_value(e);
  uint32_t r = 0;
  if constexpr (DT == INT8_FP32) {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, rowio::element<DT>(p, 0), rowio::element<DT>(p, 1), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, rowio::element<DT>(p, 2), rowio::element<DT>(p, 3), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, rowio::element<DT>(p, 4), rowio::element<DT>(p, 5), s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, rowio::element<DT>(p, 6), rowio::element<DT>(p, 7), s, 3);
  } else if constexpr (DT == INT8_FP16) {
    auto two = [&](int i) {
      const uint32_t w = p.v[0][i];
      return __builtin_bit_cast(nf4dev::f16x2, w);
    };
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, two(0), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, two(1), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, two(2), s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, two(3), s, 3);
  } else {
    auto two = [&](int i) {
      const uint32_t w = p.v[0][i];
      return __builtin_bit_cast(nf4dev::bf16x2, w);
    };
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, two(0), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, two(1), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, two(2), s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, two(3), s, 3);
  }
  return e == 255 ? 0u : r;
}

// Largest magnitude as bits of fp32.  For 16-bit types the magnitudes are compared
// as they are, two at a time, and one is converted at the end.
template <int DT>
__device__ __forceinline__ uint32_t piece_peak(const rowio::Piece<DT>& p) {
  if constexpr (DT == INT8_FP32) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = p.v[i >> 2][i & 3];
      m = max(m, w & 0x7FFFFFFFu);
    }
    return m;
  } else {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = p.v[0][i] & 0x7FFF7FFFu;
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w));
    }
    const uint16_t h = m[0] > m[1] ? m[0] : m[1];
    if constexpr (DT == INT8_BF16) return static_cast<uint32_t>(h) << 16;
    // (of an infinity or a NaN the field is 255 again)
    return __builtin_bit_cast(uint32_t, nf4dev::f16_to_f32(h)) & 0x7FFFFFFFu;
  }
}

// mxfp4_quantize of checked arguments.
void quantize_launch(const void* x, int32_t dt, int64_t rows, int64_t K, uint8_t* q, uint8_t* scale,
                     hipStream_t st);

}  // namespace mxdev
