// int8_gemm.hip -- the int8 products on the matrix cores: one matrix
// (int8_gemm, int8_linear) and rows sorted by expert (int8_gemm_grouped).
//
// v_mfma_i32_32x32x32_i8 with the weights as A (32 channels n x 32 k) and the
// activations as B (32 k x 32 tokens m).  Lane l = i + 32 g holds A[i][16 g ..
// + 15] and B[16 g .. + 15][i], and of D the column i: rows 8 (c / 4) + 4 g +
// c % 4 for its 16 registers c -- so a lane's registers are runs of four
// consecutive channels of one token.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8.h"
#include "int8_product.h"
#include "nf4_device.h"
#include "row_io.h"

namespace {

using namespace nf4dev;
using namespace rowio;
using namespace int8dev;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kMaxExperts = 1024;

struct Product {
  const int8_t* xq;
  const float* xs;
  const int8_t* wq;
  const float* ws;
  void* y;
  int64_t M, N;      // rows of y and channels (of one expert)
  int64_t pitch;
  // grouped only
  const int32_t* order;
  const int32_t* offsets;
  int64_t x_rows;
  int top_k, experts;
};

template <int DT>
__device__ __forceinline__ void store_one(void* y, int64_t i, float v) {
  if constexpr (DT == INT8_FP32)
    static_cast<float*>(y)[i] = v;
  else
    static_cast<uint16_t*>(y)[i] = to_half_bits<DT>(v);
}

// Where a tile of rows lies: rows [first, end) of y, of expert `expert`
// (end <= first: no tile).
struct RowTile {
  int64_t first, end;
  int expert;
};

// The tile'th tile of BM rows over all experts, each of which starts a new
// tile: 64 experts at a time, the lanes count theirs' tiles and sum them up.
template <int BM>
__device__ __forceinline__ RowTile find_tile(const Product& p, int64_t tile) {
  const int lane = threadIdx.x & 63;
  int64_t done = 0;
  for (int base = 0; base < p.experts; base += 64) {
    const int e = base + lane;
    int64_t a = 0, b = 0;
    if (e < p.experts) {
      a = min(max(static_cast<int64_t>(p.offsets[e]), int64_t(0)), p.M);
      b = min(max(static_cast<int64_t>(p.offsets[e + 1]), a), p.M);
    }
    const int tiles = static_cast<int>((b - a + BM - 1) / BM);
    int in = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(in, d);
      if (lane >= d) in += o;
    }
    const uint64_t past = __ballot(done + in > tile);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int64_t before = done + __shfl(in - tiles, l);
      const int64_t a0 = __shfl(static_cast<int>(a), l), b0 = __shfl(static_cast<int>(b), l);
      const int64_t first = a0 + (tile - before) * BM;
      return {first, min(b0, first + BM), base + l};
    }
    done += __shfl(in, 63);
  }
  return {0, 0, 0};
}

// The row of xq that row i of y is made from, -1 if there is none.
template <bool GROUPED>
__device__ __forceinline__ int64_t source_row(const Product& p, int64_t i) {
  if constexpr (!GROUPED) return i;
  const int64_t s = p.order ? (p.order[i] < 0 ? -1 : p.order[i] / p.top_k) : i;
  return s < p.x_rows ? s : -1;
}

// 64 x 64 tile, four waves of 32 x 32, 64 bytes of K at a time through LDS.
template <int DT, bool GROUPED>
__global__ __launch_bounds__(256) void product_kernel(Product p) {
  constexpr int kRow = 80;  // 64 bytes and 16 of padding
  __shared__ __attribute__((aligned(16))) int8_t s_x[64 * kRow], s_w[64 * kRow];
  RowTile t = {static_cast<int64_t>(blockIdx.y) * 64, p.M, 0};
  t.end = min(p.M, t.first + 64);
  if constexpr (GROUPED) {
    t = find_tile<64>(p, blockIdx.y);
    if (t.end <= t.first) return;
  }
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int8_t* wq = p.wq + t.expert * p.N * p.pitch;
  const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 16;
  int64_t src = -1;
  if (t.first + r < t.end) src = source_row<GROUPED>(p, t.first + r);
  const int8_t* xr = src >= 0 ? p.xq + src * p.pitch + c : nullptr;
  const int8_t* wr = n0 + r < p.N ? wq + (n0 + r) * p.pitch + c : nullptr;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wn = (wave & 1) * 32, wm = (wave >> 1) * 32;
  i32x16 acc = {};
  for (int64_t k = 0; k < p.pitch; k += 64) {
    const i32x4 zero = {};
    const i32x4 vx = xr ? *reinterpret_cast<const i32x4*>(xr + k) : zero;
    const i32x4 vw = wr ? *reinterpret_cast<const i32x4*>(wr + k) : zero;
    __syncthreads();
    *reinterpret_cast<i32x4*>(s_x + r * kRow + c) = vx;
    *reinterpret_cast<i32x4*>(s_w + r * kRow + c) = vw;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = 32 * h + 16 * (lane >> 5);
      const i32x4 a = *reinterpret_cast<const i32x4*>(s_w + (wn + (lane & 31)) * kRow + at);
      const i32x4 b = *reinterpret_cast<const i32x4*>(s_x + (wm + (lane & 31)) * kRow + at);
      acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, acc, 0, 0, 0);
    }
  }
  const int64_t m = t.first + wm + (lane & 31);
  if (m >= t.end) return;
  const int64_t s = source_row<GROUPED>(p, m);
  const float xs = s >= 0 ? p.xs[s] : 0.0f;
  const float* ws = p.ws + t.expert * p.N;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t n = n0 + wn + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
    if (n < p.N) store_one<DT>(p.y, m * p.N + n, static_cast<float>(acc[i]) * xs * ws[n]);
  }
}

template <bool GROUPED>
nf4_status launch(const Product& p, int32_t y_dtype, int64_t row_tiles, hipStream_t st) {
  const int64_t gx = (p.N + 63) / 64;
  if (row_tiles > 65535 || gx * 256 >= (int64_t(1) << 32)) return NF4_EUNSUPPORTED;
  with_dtype(y_dtype, [&](auto d) {
    hipLaunchKernelGGL((product_kernel<decltype(d)::value, GROUPED>),
                       dim3(static_cast<uint32_t>(gx), static_cast<uint32_t>(row_tiles)), dim3(256),
                       0, st, p);
  });
  return launch_status();
}

// What the products check alike (the activations apart).
nf4_status check_product(const int8_t* wq, const float* ws, int64_t N, int64_t K, const void* y,
                         int32_t y_dtype) {
  if (!y || !ws || (K > 0 && !wq)) return NF4_EINVAL;
  if (!aligned(wq, 16) || !aligned(ws, 4) || !aligned(y, dtype_bytes(y_dtype))) return NF4_EINVAL;
  if (N > kMaxDim || K > kMaxK) return NF4_EUNSUPPORTED;
  return NF4_OK;
}

size_t codes_bytes(int64_t M, int64_t K) { return static_cast<size_t>(M * pitch_of(K) + 255) / 256 * 256; }

}  // namespace

extern "C" {

size_t int8_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  (void)M, (void)N, (void)K;
  return 0;
}

nf4_status int8_gemm(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                     int64_t M, int64_t N, int64_t K, void* y, int32_t y_dtype, void* workspace,
                     size_t workspace_bytes, void* stream) {
  (void)workspace_bytes;
  if (M < 0 || N < 0 || K < 0 || !known_dtype(y_dtype) || !aligned(workspace, 256))
    return NF4_EINVAL;
  if (M == 0 || N == 0) return NF4_OK;
  if (!xs || (K > 0 && !xq) || !aligned(xq, 16) || !aligned(xs, 4)) return NF4_EINVAL;
  if (const nf4_status st = check_product(wq, ws, N, K, y, y_dtype)) return st;
  if (M > kMaxDim) return NF4_EUNSUPPORTED;
  const Product p = {xq, xs, wq, ws, y, M, N, pitch_of(K), nullptr, nullptr, M, 1, 1};
  return launch<false>(p, y_dtype, (M + 63) / 64, reinterpret_cast<hipStream_t>(stream));
}

size_t int8_linear_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxK) return 0;
  return codes_bytes(M, K) + (static_cast<size_t>(M) * 4 + 255) / 256 * 256 +
         int8_gemm_workspace_size(M, N, K);
}

nf4_status int8_linear(const void* x, int32_t x_dtype, const int8_t* wq, const float* ws,
                       int64_t M, int64_t N, int64_t K, void* y, int32_t y_dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || !known_dtype(x_dtype) || !known_dtype(y_dtype) ||
      !aligned(workspace, 256))
    return NF4_EINVAL;
  if (M == 0 || N == 0) return NF4_OK;
  if ((K > 0 && !x) || !aligned(x, dtype_bytes(x_dtype))) return NF4_EINVAL;
  if (const nf4_status st = check_product(wq, ws, N, K, y, y_dtype)) return st;
  if (M > kMaxDim) return NF4_EUNSUPPORTED;
  if (!workspace || workspace_bytes < int8_linear_workspace_size(M, N, K)) return NF4_EINVAL;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  int8_t* xq = static_cast<int8_t*>(workspace);
  float* xs = reinterpret_cast<float*>(xq + codes_bytes(M, K));
  quantize_launch(x, x_dtype, M, K, xq, xs, st);
  const Product p = {xq, xs, wq, ws, y, M, N, pitch_of(K), nullptr, nullptr, M, 1, 1};
  return launch<false>(p, y_dtype, (M + 63) / 64, st);
}

nf4_status int8_gemm_grouped(const int8_t* xq, const float* xs, int64_t x_rows,
                             const int32_t* order, int32_t top_k, const int8_t* wq,
                             const float* ws, const int32_t* offsets, int32_t experts,
                             int64_t rows, int64_t N, int64_t K, void* y, int32_t y_dtype,
                             void* stream) {
  if (x_rows < 0 || rows < 0 || N < 0 || K < 0 || experts < 0 || (order && top_k < 1) ||
      !known_dtype(y_dtype))
    return NF4_EINVAL;
  if (experts == 0 || rows == 0 || N == 0) return NF4_OK;
  if (!offsets || !aligned(offsets, 4) || !aligned(order, 4)) return NF4_EINVAL;
  if (x_rows > 0 && (!xs || (K > 0 && !xq))) return NF4_EINVAL;
  if (!aligned(xq, 16) || !aligned(xs, 4)) return NF4_EINVAL;
  if (const nf4_status st = check_product(wq, ws, N, K, y, y_dtype)) return st;
  if (experts > kMaxExperts || rows > kMaxDim || x_rows > kMaxDim) return NF4_EUNSUPPORTED;
  const Product p = {xq, xs, wq, ws, y, rows, N, pitch_of(K), order, offsets, x_rows,
                     order ? top_k : 1, experts};
  // every expert ends in at most one tile that is not full
  const int64_t tiles = rows / 64 + (rows < experts ? rows : experts);
  return launch<true>(p, y_dtype, tiles, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
