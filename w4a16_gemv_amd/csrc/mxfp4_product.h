// mxfp4_product.h -- what the kernels of the products of 4-bit microscaled floats
// share (private to libnf4).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxfp4.h"
#include "mxfp4_format.h"
#include "product_tiles.h"

namespace mxdev {

using tiledev::i32x4;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct Product {
  const uint8_t* xq;
  const uint8_t* xs;
  const uint8_t* wq;
  const uint8_t* ws;
  void* y;
  int64_t M, N;      // rows of y and channels (of one expert)
  int64_t pitch;     // bytes of a row of codes
  int64_t steps;     // tiles of scales along K
  // grouped only
  const int32_t* order;
  const int32_t* offsets;
  int64_t x_rows;
  int top_k, experts;
  // K split over `splits` workgroups of a tile: fp32 sums to planes of
  // M x sums_pitch at `sums` instead of y (dense only)
  float* sums;
  int64_t sums_pitch;
  int splits;
  uint32_t cus;  // compute units
};

constexpr int kFp4 = 4;    // the operands' format in the matrix instructions
constexpr int kCodes = 3;  // the tokens' type where they are encoded already (else an int8_dtype)

// Four of the eight registers that the instruction has room for.
__device__ __forceinline__ i32x8 four(const i32x4& a) {
  return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
}

// Keeps sums where they are computed, by all lanes.  Where only some lanes use them the
// compiler may move a matrix instruction to these lanes alone, though it reads the operands
// of all.  (No instruction is written here, so there is nothing that would have to wait for
// the sums; the compiler's own next one does.)
template <class V>
__device__ __forceinline__ void settled(V& v) {
  asm volatile("" : "+v"(v));
}

// Offset of the scales of row `row` (of the group of 128 codes g) from those of row
// `first`'s tile.
__device__ __forceinline__ uint32_t scale_from(int64_t first, int64_t row, int64_t steps, int g) {
  return static_cast<uint32_t>(((row >> 5) - (first >> 5)) * steps * 256 + g * 128 + (row & 31) * 4);
}

constexpr int kRowWaves = 8;  // of the few-row kernel

// The few-row kernel's variant: waves that share a tile's K, units of 64 bytes that a wave
// holds at a time.
struct Rows {
  int split, units;
};
// rows: tiles of 16 rows.
Rows row_plan(const Product& p, int64_t rows);

// Whether the few-row kernel takes rows of this length, 22 units to a wave at most.  (LDS for
// 16 rows of codes and the grid's second dimension set no limit: who chooses the kernel asks
// for 35 KB and 2048 tiles of rows at most.)
bool fits_rows(const Product& p);

// The few-row kernel on tokens of type xt at x, or on the product's codes (kCodes).
nf4_status launch_rows(const Product& p, bool grouped, const void* x, int32_t xt, int64_t K, int32_t y_dtype,
                       hipStream_t st);

}  // namespace mxdev
