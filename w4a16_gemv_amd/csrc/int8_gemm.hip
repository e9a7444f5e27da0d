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
      const int first = __builtin_amdgcn_readfirstlane(static_cast<int>(a0 + (tile - before) * BM));
      const int end = __builtin_amdgcn_readfirstlane(static_cast<int>(min(b0, int64_t(first) + BM)));
      return {first, end, base + l};
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

// Tiles in an order whose neighbours share rows and channels, for the workgroup
// that the hardware starts as number b: it deals workgroups out to the eight
// dies in turn, so each die gets a range of its own, and within it bands of
// kBand row tiles.  False past the last tile.
constexpr uint32_t kDies = 8;
constexpr uint32_t kBand = 8;

__device__ __forceinline__ bool place_tile(uint32_t b, uint32_t tiles_m, uint32_t tiles_n,
                                           uint32_t& tm, uint32_t& tn) {
  const uint32_t all = tiles_m * tiles_n;  // < 2^24, by the grid's limit
  const uint32_t each = (all + kDies - 1) / kDies;
  const uint32_t at = b / kDies, i = b % kDies * each + at;
  if (at >= each || i >= all) return false;
  const uint32_t band = i / (kBand * tiles_n), in = i % (kBand * tiles_n);
  const uint32_t high = min(uint32_t(kBand), tiles_m - band * kBand);
  // the divisions run on the vector unit: back to scalars, so that what follows
  // from them (buffer resources among it) is one value per wave
  tm = __builtin_amdgcn_readfirstlane(band * kBand + in % high);
  tn = __builtin_amdgcn_readfirstlane(in / high);
  return true;
}

// Row tiles over all experts.
template <int BM>
__device__ __forceinline__ uint32_t count_tiles(const Product& p) {
  const int lane = threadIdx.x & 63;
  int sum = 0;
  for (int e = lane; e < p.experts; e += 64) {
    const int64_t a = min(max(static_cast<int64_t>(p.offsets[e]), int64_t(0)), p.M);
    const int64_t b = min(max(static_cast<int64_t>(p.offsets[e + 1]), a), p.M);
    sum += static_cast<int>((b - a + BM - 1) / BM);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
  return __builtin_amdgcn_readfirstlane(sum);
}

// ---------------------------------------------------------------------------
// Tiles through LDS.  Four waves, 2 x 2, share a tile of BN channels x BM
// tokens; each holds its quarter in int32 accumulators.  128 bytes of K at a
// time (a step): the tile's rows go from memory to registers one step ahead,
// into one of two LDS buffers, and from there to the matrix cores, 32 bytes of
// K at a time (a part) with the next 32 being read.  One barrier per step: it
// stands before the last part, whose operands are in registers by then, so
// that the other buffer's first operands are read while the matrix cores still
// work.  The order of the instructions is given by hand (sched_group_barrier):
// left alone the compiler reads operands right before their use.
//
// LDS: two rows of eight 16-byte chunks fill the 64 banks; chunk c of row r is
// stored at c ^ (r / 2 % 8), so that the sixteen lanes that are served at a
// time, 16 rows of one chunk (reads) or two whole rows (writes), lie in all
// banks once.
//
// Rows past the tile's end are zeros or whatever row is at hand (their outputs
// are not stored); bytes past a row's pitch are zeros on the weights' side.
// The step past the last is loaded too: zeros that nothing uses.
//
// Out: 32 tokens at a time through LDS, so that whole lines of y are written.
// ---------------------------------------------------------------------------
constexpr int kTileThreads = 256;
constexpr int kDepth = 128;  // bytes of K per step
constexpr uint32_t kNever = 0x80000000u;

// In the order of the program: one vector-memory load or LDS instruction
// (kind), then `count` matrix instructions.
constexpr int kSchedMfma = 0x8, kSchedLoad = 0x20, kSchedRead = 0x100, kSchedWrite = 0x200;

template <int DT, int BM, int BN>
constexpr int tile_lds() {
  constexpr int in = 2 * (BM + BN) * kDepth;
  constexpr int out = 4 * 32 * (BN / 2 * dtype_bytes(DT) + 16);
  return in > out ? in : out;
}

template <int DT, bool GROUPED, int BM, int BN>
__global__ __launch_bounds__(kTileThreads, BM* BN >= 256 * 256 ? 1 : 2) void tile_kernel(Product p) {
  constexpr int TM = BM / 64, TN = BN / 64;          // 32 x 32 tiles of a wave
  constexpr int LM = BM / 32, LN = BN / 32;          // 16-byte loads of a thread per step
  __shared__ __attribute__((aligned(16))) int8_t s_mem[tile_lds<DT, BM, BN>()];

  // --- which tile
  const uint32_t tiles_n = static_cast<uint32_t>((p.N + BN - 1) / BN);
  uint32_t tiles_m = static_cast<uint32_t>((p.M + BM - 1) / BM);
  if constexpr (GROUPED) tiles_m = count_tiles<BM>(p);
  uint32_t tm, tn;
  if (!place_tile(blockIdx.x, tiles_m, tiles_n, tm, tn)) return;
  RowTile t = {static_cast<int64_t>(tm) * BM, min(p.M, static_cast<int64_t>(tm) * BM + BM), 0};
  if constexpr (GROUPED) t = find_tile<BM>(p, tm);
  const int64_t n0 = static_cast<int64_t>(tn) * BN;

  // --- memory to registers: eight threads a row
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int row = threadIdx.x >> 3, chunk = (threadIdx.x & 7) * 16;
  const int pitch = static_cast<int>(p.pitch);
  const int8_t* w0 = p.wq + (t.expert * p.N + n0) * p.pitch;
  const auto rw = rsrc(w0, static_cast<uint32_t>(min(int64_t(BN), p.N - n0) * p.pitch));
  const auto rx = rsrc(GROUPED ? nullptr : p.xq + t.first * p.pitch,
                       static_cast<uint32_t>((t.end - t.first) * p.pitch));
  const uint32_t voff = static_cast<uint32_t>(row * pitch + chunk);
  const int8_t* xrow[GROUPED ? LM : 1];
  if constexpr (GROUPED) {
#pragma unroll
    for (int i = 0; i < LM; ++i) {
      const int64_t m = t.first + row + 32 * i;
      const int64_t src = m < t.end ? source_row<true>(p, m) : -1;
      xrow[i] = src >= 0 ? p.xq + src * p.pitch : w0;  // any row that may be read
    }
  }
  i32x4 g[LN + LM];
  auto load = [&](int i, int k) {
    const bool in = k + chunk < pitch;
    const uint32_t v = in ? voff + k : kNever;
    if (i < LN)
      g[i] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, v, 32 * i * pitch, 0));
    else if constexpr (GROUPED)
      g[i] = *reinterpret_cast<const i32x4*>(xrow[GROUPED ? i - LN : 0] + (in ? k + chunk : 0));
    else
      g[i] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, v, 32 * (i - LN) * pitch, 0));
  };

  // --- registers to LDS: the weights' rows first, then the tokens'
  constexpr int kBuffer = (BM + BN) * kDepth;
  const int put = row * kDepth + (chunk ^ ((row >> 1 & 7) * 16));
  auto store = [&](int i, int buf) {
    *reinterpret_cast<i32x4*>(s_mem + buf * kBuffer + put + 32 * i * kDepth) = g[i];
  };

  // --- LDS to the matrix cores
  const int wn = (wave & 1) * (BN / 2), wm = (wave >> 1) * (BM / 2);
  i32x4 fw[2][TN], fx[2][TM];
  auto fetch = [&](int set, int buf, int part) {
    const int at = buf * kBuffer + (lane & 31) * kDepth + (((2 * part + (lane >> 5)) ^ (lane >> 1 & 7)) * 16);
#pragma unroll
    for (int i = 0; i < TN; ++i)
      fw[set][i] = *reinterpret_cast<const i32x4*>(s_mem + (wn + 32 * i) * kDepth + at);
#pragma unroll
    for (int i = 0; i < TM; ++i)
      fx[set][i] = *reinterpret_cast<const i32x4*>(s_mem + (BN + wm + 32 * i) * kDepth + at);
  };
  i32x16 acc[TN][TM] = {};
  auto multiply = [&](int set) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[set][i], fx[set][j], acc[i][j], 0, 0, 0);
  };

  const int steps = (pitch + kDepth - 1) / kDepth;
  if (steps > 0) {
#pragma unroll
    for (int i = 0; i < LN + LM; ++i) load(i, 0);
#pragma unroll
    for (int i = 0; i < LN + LM; ++i) {
      store(i, 0);
      load(i, kDepth);
    }
    __syncthreads();
    fetch(0, 0, 0);
    for (int k = 0; k < steps; ++k) {
      const int buf = k & 1;
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        fetch((part + 1) & 1, buf, part + 1);
        constexpr int kAll = LN + LM, kThird = (kAll + 2) / 3;
        const int moves = part < 2 ? kThird : kAll - 2 * kThird;
#pragma unroll
        for (int i = part * kThird; i < part * kThird + moves; ++i) {
          store(i, buf ^ 1);
          load(i, (k + 2) * kDepth);
        }
        multiply(part & 1);
        // operand reads first, one to a matrix instruction, then the moves
#pragma unroll
        for (int i = 0; i < TN + TM; ++i) {
          __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
          __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
        }
#pragma unroll
        for (int i = 0; i < moves; ++i) {
          __builtin_amdgcn_sched_group_barrier(kSchedWrite, 1, 0);
          __builtin_amdgcn_sched_group_barrier(kSchedLoad, 1, 0);
          __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();
      fetch(0, buf ^ 1, 0);
      multiply(1);
#pragma unroll
      for (int i = 0; i < TN + TM; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
  }

  // --- out: each wave has an LDS region of its own, 32 tokens of its channels
  constexpr int kB = dtype_bytes(DT);
  constexpr int kRow = BN / 2 * kB + 16;  // 16 bytes of padding
  int8_t* mine = s_mem + wave * 32 * kRow;
  const float* ws = p.ws + t.expert * p.N;
  const int64_t n1 = n0 + wn;  // the wave's first channel
  const int64_t wide = min(p.N - n1, int64_t(BN / 2));
  float wscale[TN][16];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const int64_t n = n1 + 32 * i + 8 * (c >> 2) + 4 * (lane >> 5) + (c & 3);
      wscale[i][c] = n < p.N ? ws[n] : 0.0f;
    }
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t m0 = t.first + wm + 32 * j;
    const int64_t m = m0 + (lane & 31);
    const int64_t src = m < t.end ? source_row<GROUPED>(p, m) : -1;
    const float xs = src >= 0 ? p.xs[src] : 0.0f;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int c = 0; c < 16; c += 4) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = static_cast<float>(acc[i][j][c + e]) * xs * wscale[i][c + e];
        int8_t* to = mine + (lane & 31) * kRow + (32 * i + 2 * c + 4 * (lane >> 5)) * kB;
        if constexpr (DT == INT8_FP32)
          *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
        else
          *reinterpret_cast<uint2*>(to) = make_uint2(pack_pair<DT>(f[0], f[1]), pack_pair<DT>(f[2], f[3]));
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    constexpr int kPieces = BN / 2 / 8;  // of eight channels, to a row
#pragma unroll
    for (int i = lane; i < 32 * kPieces; i += 64) {
      const int r = i / kPieces, at = i % kPieces * 8;
      if (m0 + r >= t.end || at >= wide) continue;
      Piece<DT> v;
      v.v[0] = *reinterpret_cast<const u32x4*>(mine + r * kRow + at * kB);
      if constexpr (DT == INT8_FP32) v.v[1] = *reinterpret_cast<const u32x4*>(mine + r * kRow + at * kB + 16);
      store_piece<DT>(static_cast<char*>(p.y) + ((m0 + r) * p.N + n1) * kB, at, wide, v);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

template <bool GROUPED, int BM, int BN>
nf4_status launch_tiles(const Product& p, int32_t y_dtype, int64_t tiles_m, hipStream_t st) {
  const int64_t all = tiles_m * ((p.N + BN - 1) / BN);
  const int64_t groups = (all + kDies - 1) / kDies * kDies;
  if (groups * kTileThreads >= (int64_t(1) << 32)) return NF4_EUNSUPPORTED;
  with_dtype(y_dtype, [&](auto d) {
    hipLaunchKernelGGL((tile_kernel<decltype(d)::value, GROUPED, BM, BN>),
                       dim3(static_cast<uint32_t>(groups)), dim3(kTileThreads), 0, st, p);
  });
  return launch_status();
}

// Tiles of BM rows that p.M rows need at most: every expert ends in at most one
// tile that is not full.
template <bool GROUPED>
int64_t row_tiles(const Product& p, int64_t BM) {
  if constexpr (GROUPED) return p.M / BM + (p.M < p.experts ? p.M : p.experts);
  return (p.M + BM - 1) / BM;
}

template <bool GROUPED>
nf4_status launch(const Product& p, int32_t y_dtype, hipStream_t st) {
  const int64_t rows = GROUPED ? p.M / p.experts : p.M;
  if (rows > 128) return launch_tiles<GROUPED, 256, 256>(p, y_dtype, row_tiles<GROUPED>(p, 256), st);
  if (rows > 64) return launch_tiles<GROUPED, 128, 128>(p, y_dtype, row_tiles<GROUPED>(p, 128), st);
  return launch_tiles<GROUPED, 64, 64>(p, y_dtype, row_tiles<GROUPED>(p, 64), st);
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
  return launch<false>(p, y_dtype, reinterpret_cast<hipStream_t>(stream));
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
  return launch<false>(p, y_dtype, st);
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
  return launch<true>(p, y_dtype, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
