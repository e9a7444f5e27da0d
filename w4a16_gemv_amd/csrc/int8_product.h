// int8_product.h -- the int8 row encoder's arithmetic and the launchers that
// the int8 sources share (private to libnf4).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8.h"
#include "nf4_device.h"
#include "row_io.h"

namespace int8dev {

constexpr int64_t kMaxDim = 0x7FFFFFFF;
constexpr int64_t kMaxK = 131071;  // K * 128 * 128 < 2^31

// 64-byte rows: 16-byte loads at every K, and a row's padding fills one matrix
// instruction's depth at most.
inline int64_t pitch_of(int64_t K) { return K > 0 ? (K + 63) / 64 * 64 : 0; }

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), d)));
  return v;
}

// Largest magnitude as bits: without the sign, the order of the bits is that of
// the values, infinity above every number and NaN above infinity.
template <int DT>
__device__ __forceinline__ uint32_t piece_peak(const rowio::Piece<DT>& p) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    m = max(m, __builtin_bit_cast(uint32_t, rowio::element<DT>(p, i)) & 0x7FFFFFFFu);
  return m;
}

struct RowScale {
  float scale, inverse;
};

// Of a row's largest magnitude; NaN and 0 for a row that is not finite, whose
// codes are then all zero.  Both by products with a rounded reciprocal: what the
// tensor expressions a / 127 and 127 / a compute on this device, so that a program
// that encodes with those gets the same codes, ties such as a / 2 included.  The price
// is an inverse up to 1.5 ulp from 127 / a instead of 0.5, and a scale up to 0.56 from a
// / 127: 2^-16 of a step in the codes.  (1 / a is subnormal for a > 2^126, where the
// inverse is within 2^-21: 2^-14 of a step.)
__device__ __forceinline__ RowScale row_scale(uint32_t peak) {
  const float a = fmaxf(__builtin_bit_cast(float, peak), 0x1p-100f);
  RowScale s = {a * (1.0f / 127.0f), 127.0f * (1.0f / a)};
  if (peak >= 0x7F800000u) s = {__builtin_nanf(""), 0.0f};
  return s;
}

// Eight codes.  A row that is not finite has inverse 0, and its infinities and
// NaN give NaN here, whose low byte is no code: they are cut off by hand.
template <int DT>
__device__ __forceinline__ uint2 encode_piece(const rowio::Piece<DT>& p, const RowScale& s) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = __builtin_bit_cast(uint32_t, fmaf(rowio::element<DT>(p, i), s.inverse, 0x1.8p23f)) & 0xFFu;
  uint2 r = make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                       c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
  if (s.inverse == 0.0f) r = make_uint2(0u, 0u);
  return r;
}

// int8_quantize of checked arguments.
void quantize_launch(const void* x, int32_t dt, int64_t rows, int64_t K, int8_t* q, float* scale,
                     hipStream_t st);

}  // namespace int8dev
