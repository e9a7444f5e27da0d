// int8_quantize.hip -- the int8 encoder (activations per token, weights per
// output channel) and its inverse.
//
// Encoder, per row: a = max(max|x|, 2^-100), scale = a * (1 / 127) and inverse =
// 127 * (1 / a) (each step rounded: row_scale() says why), code = x * inverse rounded
// half to even.
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

// A grid may not have 2^32 threads: past this many workgroups each takes several
// turns.
constexpr int64_t kMaxGroups = 1 << 20;

uint32_t groups_for(int64_t n) { return static_cast<uint32_t>(n < kMaxGroups ? n : kMaxGroups); }

// WAVES waves per row: a whole workgroup, or each of its waves a row of its own
// where rows are short and many.  The row's values stay in registers from the
// maximum to the codes: HOLD pieces of eight to a thread (0: the row is longer and
// read a second time, from the caches).  Bound by memory: 4097 x 11008 bf16 takes
// 23.5 us (135 MB, 5.8 TB/s).
template <int DT, int WAVES, int HOLD>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const void* __restrict__ x, int64_t rows,
                                                                 int64_t K, int64_t pitch,
                                                                 int8_t* __restrict__ q,
                                                                 float* __restrict__ scale) {
  constexpr int kAtOnce = kThreads / 64 / WAVES, kWidth = 64 * WAVES;  // rows of a workgroup, threads of a row
  __shared__ uint32_t s_max[WAVES];
  const int t = threadIdx.x % kWidth;
  for (int64_t row = int64_t(blockIdx.x) * kAtOnce + threadIdx.x / kWidth; row < rows;
       row += int64_t(gridDim.x) * kAtOnce) {
    const char* xr = static_cast<const char*>(x) + row * K * dtype_bytes(DT);
    Piece<DT> held[HOLD > 0 ? HOLD : 1];
    uint32_t m = 0;
    if constexpr (HOLD > 0) {
#pragma unroll
      for (int i = 0; i < HOLD; ++i) {
        const int64_t at = 8 * (t + int64_t(i) * kWidth);
        held[i] = Piece<DT>{};
        if (at + 8 <= K)
          held[i] = whole_piece<DT, true>(xr, at);
        else if (at < K)
          held[i] = load_piece<DT>(xr, at, K);
      }
#pragma unroll
      for (int i = 0; i < HOLD; ++i) m = max(m, piece_peak<DT>(held[i]));
    } else {
      for (int64_t at = 8 * t; at < K; at += 8 * kWidth) m = max(m, piece_peak<DT>(load_piece<DT>(xr, at, K)));
    }
    m = wave_max(m);
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < WAVES; ++i) m = max(m, s_max[i]);
      __syncthreads();  // before the next row's
    }
    const RowScale s = row_scale(m);
    if (t == 0) scale[row] = s.scale;
    int8_t* qr = q + row * pitch;
    if constexpr (HOLD > 0) {
#pragma unroll
      for (int i = 0; i < HOLD; ++i) {
        const int64_t at = 8 * (t + int64_t(i) * kWidth);
        if (at < pitch) *reinterpret_cast<uint2*>(qr + at) = encode_piece<DT>(held[i], s);
      }
    } else {
      for (int64_t at = 8 * t; at < pitch; at += 8 * kWidth)
        *reinterpret_cast<uint2*>(qr + at) = encode_piece<DT>(load_piece<DT>(xr, at, K), s);
    }
  }
}

// Threads of a row as above.  Bound by memory: 4097 x 11008 to bf16 takes 21 us (6.4
// TB/s).
template <int DT, int WAVES>
__global__ __launch_bounds__(kThreads) void dequant_rows_kernel(const int8_t* __restrict__ q,
                                                                const float* __restrict__ scale, int64_t rows,
                                                                int64_t K, int64_t pitch,
                                                                void* __restrict__ out) {
  constexpr int kAtOnce = kThreads / 64 / WAVES, kWidth = 64 * WAVES;
  for (int64_t row = int64_t(blockIdx.x) * kAtOnce + threadIdx.x / kWidth; row < rows;
       row += int64_t(gridDim.x) * kAtOnce) {
    const float s = scale[row];
    char* o = static_cast<char*>(out) + row * K * dtype_bytes(DT);
    for (int64_t at = 8 * (threadIdx.x % kWidth); at < K; at += 8 * kWidth) {
      const uint2 c = *reinterpret_cast<const uint2*>(q + row * pitch + at);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        f[i] = static_cast<float>(static_cast<int8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)))) * s;
      store_piece<DT>(o, at, K, make_piece<DT>(f));
    }
  }
}

// Short rows, and so many that they fill the card as waves too: a wave each, which
// needs no barrier.  Encoder: 1024 x 512 in 3.2 us against 3.7, 16384 x 512 in 10.3
// against 20.3, 16384 x 2048 in 18.5 against 24.6; 256 x 2048 would take 3.4 against
// 2.8.  A longer row would not fit a wave's registers.
bool encode_by_waves(int64_t rows, int64_t K) { return K <= 4 * 8 * 64 && rows >= 4 * device_cus(); }

// Its inverse has no barrier to save: 16384 x 512 in 5.8 us against 7.3, 4096 x 1024
// in 4.0 against 4.2; 2048 x 2048 would take 4.6 against 4.0.
bool decode_by_waves(int64_t rows, int64_t K) { return K <= 1024 && rows > 8 * device_cus(); }

}  // namespace

namespace int8dev {

void quantize_launch(const void* x, int32_t dt, int64_t rows, int64_t K, int8_t* q, float* scale,
                     hipStream_t st) {
  with_dtype(dt, [&](auto t) {
    constexpr int DT = decltype(t)::value;
    const int64_t pitch = pitch_of(K);
#define INT8_QUANTIZE(WAVES, HOLD)                                                                     \
  hipLaunchKernelGGL((quantize_rows_kernel<DT, WAVES, HOLD>), dim3(groups_for((rows * WAVES + 3) / 4)), \
                     dim3(kThreads), 0, st, x, rows, K, pitch, q, scale)
    // Held rows: 4097 x 11008 in 23.5 us against 37.5 read twice, 4097 x 14336 in 33
    // against 47.5, 1000 x 32768 in 22.5 against 28.  A row takes the least variant that
    // holds it, since a thread's pieces past the row cost too: in four pieces instead of
    // six 1 x 4160 takes 2.6 us against 2.9, 4097 x 4160 12.5 against 15.4, 4097 x 8192
    // 18.6 against 19.6.
    if (encode_by_waves(rows, K))
      INT8_QUANTIZE(1, 4);
    else if (K <= 2 * 8 * kThreads)
      INT8_QUANTIZE(4, 2);
    else if (K <= 4 * 8 * kThreads)
      INT8_QUANTIZE(4, 4);
    else if (K <= 6 * 8 * kThreads)
      INT8_QUANTIZE(4, 6);
    else if (K <= 8 * 8 * kThreads)
      INT8_QUANTIZE(4, 8);
    else if (K <= 16 * 8 * kThreads)
      INT8_QUANTIZE(4, 16);
    else
      INT8_QUANTIZE(4, 0);
#undef INT8_QUANTIZE
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
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  with_dtype(out_dtype, [&](auto t) {
    constexpr int DT = decltype(t)::value;
    if (decode_by_waves(rows, K))
      hipLaunchKernelGGL((dequant_rows_kernel<DT, 1>), dim3(groups_for((rows + 3) / 4)), dim3(kThreads), 0, st, q,
                         scale, rows, K, pitch_of(K), out);
    else
      hipLaunchKernelGGL((dequant_rows_kernel<DT, 4>), dim3(groups_for(rows)), dim3(kThreads), 0, st, q, scale,
                         rows, K, pitch_of(K), out);
  });
  return launch_status();
}

}  // extern "C"
