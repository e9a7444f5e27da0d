// mxfp4_few.hip -- the products of 4-bit microscaled floats for few rows.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mxfp4.h"
#include "mxfp4_format.h"
#include "mxfp4_product.h"
#include "nf4_device.h"
#include "product_tiles.h"
#include "row_io.h"

namespace {

using namespace nf4dev;
using namespace rowio;
using namespace tiledev;
using namespace mxdev;

constexpr int kRowThreads = 64 * kRowWaves;

// Bytes in LDS from one token's codes to the next, and dwords from its scales to the
// next's: such that a chunk of 16 rows lies in different banks.
__device__ __host__ __forceinline__ int lds_pitch(int pitch) { return pitch + 16; }
__device__ __host__ __forceinline__ int lds_groups(int pitch) { return pitch / 64 | 1; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true));
}

// ---------------------------------------------------------------------------
// Up to 16 tokens, whose codes and scales a workgroup keeps in LDS.  It goes through its
// channels in tiles of 16, 8 / SPLIT at a time, each with SPLIT waves that share K: the
// weights go from memory through registers to the matrix cores
// (v_mfma_scale_f32_16x16x128_f8f6f4: lane i + 16 g holds the codes 32 g .. + 31 of row i
// of A, B likewise with i the column, and D[4 g .. + 3][i]), each byte read once, the next tile's asked for as soon as the
// registers are free.  The waves' sums meet in LDS and are added in the waves' order.  More
// rows than 16 go to more workgroups.
//
// Tokens that are not codes yet (XT other than kCodes) are encoded on the way to LDS,
// after the workgroup's first weights have been asked for.
//
// Bound by the weights' stream and a start of 2 us: 1 x 4096 x 4096 with encoding 4.7 us
// (9 MB, a plain read of as much 3.0), 16 tokens' 4 of 64 experts of 1024 x 2048 9.4 us (46 MB,
// 8.3).  Four lanes to a row's 64 bytes and a turn by ds_bpermute: the operands' own layout,
// 16 rows' 16 bytes a load, reads at 60-90% of the rate.
// ---------------------------------------------------------------------------
template <int XT, int DT, bool GROUPED, int SPLIT, int UNITS>
__global__ __launch_bounds__(kRowThreads, UNITS > 8 ? 2 : 4) void mx_row_kernel(Product p, const void* x, int64_t K) {
  __shared__ f32x4 s_sum[2][kRowWaves][64];
  extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];
  constexpr uint32_t kGroup = kRowWaves / SPLIT;  // tiles at a time
  const uint32_t tiles = static_cast<uint32_t>((p.N + 15) / 16), groups_n = (tiles + kGroup - 1) / kGroup;
  RowTile t = {int64_t(16) * blockIdx.y, min(p.M, int64_t(16) * blockIdx.y + 16), 0};
  if constexpr (GROUPED) t = find_tile<16>(p, blockIdx.y);
  if (t.end <= t.first) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int pitch = static_cast<int>(p.pitch), rows = static_cast<int>(t.end - t.first);
  const int share = wave % SPLIT;  // of K
  // a unit as it is loaded: lane 4 i + g has 16 bytes g of row i, so that four lanes
  // read 64 bytes in a row; turned() hands them to lane i + 16 g
  const int row = lane >> 2, inside = (lane & 3) * 16, g = lane >> 4;
  auto turned = [&](const i32x4& v) {
    const int from = 4 * (4 * (lane & 15) + g);  // a lane's number times 4
    i32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = __builtin_amdgcn_ds_bpermute(from, v[e]);
    return r;
  };
  // the wave's units of 64 bytes: pairs, so that two loads read whole lines
  const int units = pitch / 64;
  auto unit = [&](int u) { return 2 * share + 2 * SPLIT * (u >> 1) + (u & 1); };
  const uint32_t voff = static_cast<uint32_t>(row * pitch + inside);
  const uint8_t* w0 = p.wq + t.expert * p.N * p.pitch;
  i32x4 w[UNITS];
  uint32_t ws[UNITS];
  struct Tile {
    __amdgpu_buffer_rsrc_t codes, scales;
    uint32_t at;  // of the lane's row's scales
  };
  auto range = [&](uint32_t group) {
    const uint32_t tile = group * kGroup + wave / SPLIT;
    const int64_t n0 = static_cast<int64_t>(min(tile, tiles - 1)) * 16, c0 = t.expert * p.N + n0;
    const int64_t wide = tile < tiles ? min(int64_t(16), p.N - n0) : 0;  // no rows: zeros
    return Tile{rsrc(w0 + n0 * p.pitch, static_cast<uint32_t>(wide * p.pitch)),
                rsrc(p.ws + (c0 >> 5) * p.steps * 256,
                     static_cast<uint32_t>(wide > 0 ? (((c0 + wide + 31) >> 5) - (c0 >> 5)) * p.steps * 256 : 0)),
                scale_from(c0, c0 + (lane & 15), p.steps, 0)};
  };
  auto load = [&](const Tile& r, int u) {
    const bool in = unit(u) < units;
    w[u] = __builtin_bit_cast(
        i32x4, __builtin_amdgcn_raw_buffer_load_b128(r.codes, in ? voff + 64 * unit(u) : kNever, 0, 0));
    ws[u] = __builtin_amdgcn_raw_buffer_load_b32(r.scales, in ? r.at + 128 * unit(u) : kNever, 0, 0);
  };
  const Tile first = range(blockIdx.x);
#pragma unroll
  for (int u = 0; u < UNITS; ++u) load(first, u);

  // --- the tokens' codes and scales
  const int wide = lds_pitch(pitch), groups = lds_groups(pitch);
  uint32_t* s_scale = reinterpret_cast<uint32_t*>(s_x + rows * wide);
  if constexpr (XT == kCodes) {
    // a row of codes after the other to the threads, 16 bytes each, and of scales
    const int pieces = pitch / 16;
    for (int i = threadIdx.x; i < rows * pieces; i += kRowThreads) {
      const int r = i / pieces, at = 16 * (i - r * pieces);
      const int64_t src = source_row<GROUPED>(p, t.first + r);
      const uint8_t* q = src >= 0 ? p.xq + src * p.pitch : w0;  // any row that may be read
      *reinterpret_cast<i32x4*>(s_x + r * wide + at) = *reinterpret_cast<const i32x4*>(q + at);
    }
    for (int i = threadIdx.x; i < rows * units; i += kRowThreads) {
      const int r = i / units, u = i - r * units;
      const int64_t src = source_row<GROUPED>(p, t.first + r);
      s_scale[r * groups + u] = src >= 0 ? *reinterpret_cast<const uint32_t*>(p.xs + scale_at(src, p.steps, u)) : 0u;
    }
  } else {
    // sixteen lanes take a group of 128 elements of a row, several groups' loads at a time
    constexpr int kAtOnce = XT == INT8_FP32 ? 4 : 8;
    const int eights = pitch / 4, all = rows * eights;
    for (int i0 = threadIdx.x; i0 < all; i0 += kAtOnce * kRowThreads) {
      Piece<XT> v[kAtOnce];
      int r[kAtOnce], at[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int i = i0 + k * kRowThreads;
        r[k] = i / eights, at[k] = 8 * (i - r[k] * eights);
        v[k] = Piece<XT>{};
        if (i < all && at[k] < K)
          v[k] = load_piece<XT>(static_cast<const char*>(x) + (t.first + r[k]) * K * dtype_bytes(XT), at[k], K);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (i0 + k * kRowThreads >= all) break;
        uint32_t m = piece_peak<XT>(v[k]);
        m = max(m, dpp<0xB1>(m));  // the neighbour
        m = max(m, dpp<0x4E>(m));  // the other pair of the four, a block
        const uint32_t e = block_scale(m);
        *reinterpret_cast<uint32_t*>(s_x + r[k] * wide + at[k] / 2) = encode_piece<XT>(v[k], e);
        uint32_t s = e | dpp<0x104>(e) << 8;  // four blocks' in the first of sixteen lanes
        s |= dpp<0x108>(s) << 16;
        if ((lane & 15) == 0) s_scale[r[k] * groups + at[k] / 128] = s;
      }
    }
  }
  __syncthreads();

  const int64_t m = t.first + (lane & 15);
  const int mine = min(lane & 15, rows - 1);
  const uint32_t keep = keep_mask<GROUPED>(source_row<GROUPED>(p, t.first + mine));
  const uint8_t* xc = s_x + mine * wide + 16 * g;
  const uint32_t* xs = s_scale + mine * groups;
  int turn = 0;
  for (uint32_t group = blockIdx.x; group < groups_n; group += gridDim.x, ++turn) {
    const Tile next = range(group + gridDim.x);
    f32x4 acc = {};
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int at = unit(u) < units ? unit(u) : 0;  // past the row the weights are zeros, and their scales
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          four(turned(w[u])), four(*reinterpret_cast<const i32x4*>(xc + 64 * at)), acc, kFp4, kFp4, 0,
          static_cast<int>(ws[u] >> (8 * g)), 0, static_cast<int>(xs[at] >> (8 * g)));
      // the products first, then the loads into the registers that they free: the
      // other way round the compiler takes twice the registers
      if (u & 1) {
        __builtin_amdgcn_sched_barrier(0);
        load(next, u - 1);
        load(next, u);
      }
    }
    const uint32_t tile = group * kGroup + wave / SPLIT;
    settled(acc);
    f32x4 sum = acc;
    if constexpr (SPLIT > 1) {
      s_sum[turn & 1][wave][lane] = acc;
      __syncthreads();
      // one of a tile's waves a turn adds up; its buffer is written again two turns later,
      // after a barrier that this wave reaches when it is through
      if (share != (turn & (SPLIT - 1))) continue;
      sum = s_sum[turn & 1][wave - share][lane];
#pragma unroll
      for (int v = 1; v < SPLIT; ++v) sum += s_sum[turn & 1][wave - share + v][lane];
    }
    const int64_t n = static_cast<int64_t>(tile) * 16 + 4 * g;
    const int left = static_cast<int>(min(p.N - n, int64_t(4)));
    if (m >= t.end || left <= 0) continue;
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = sum[e];
      f[e] = masked(v, keep);
    }
    store_four<DT>(p.y, m * p.N + n, left, f);
  }
}

int64_t lds_bytes(int64_t pitch, int64_t rows) {
  return rows * (lds_pitch(static_cast<int>(pitch)) + 4 * lds_groups(static_cast<int>(pitch)));
}

template <int XT, bool GROUPED>
nf4_status launch_typed(const Product& p, const void* x, int64_t K, int32_t y_dtype, hipStream_t st) {
  const int64_t rows = row_tiles<GROUPED>(p, 16);
  const Rows r = row_plan(p, rows);
  // two workgroups fit a compute unit
  const int64_t groups = ((p.N + 15) / 16 * r.split + kRowWaves - 1) / kRowWaves;
  const int64_t most = 2 * device_cus(), share = (most + rows - 1) / rows;
  const dim3 grid(static_cast<uint32_t>(groups < share ? groups : share), static_cast<uint32_t>(rows));
  const uint32_t lds = static_cast<uint32_t>(lds_bytes(p.pitch, p.M < 16 ? p.M : 16));
  bool known = true;
  with_dtype(y_dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    auto run = [&](auto split, auto units) {
      hipLaunchKernelGGL((mx_row_kernel<XT, DT, GROUPED, decltype(split)::value, decltype(units)::value>), grid,
                         dim3(kRowThreads), lds, st, p, x, K);
    };
    using std::integral_constant;
    const int variant = r.split == kRowWaves ? r.units : -r.split;
    if constexpr (!GROUPED) {  // experts' rows take four waves or fewer
      if (variant == 4) return run(integral_constant<int, 8>{}, integral_constant<int, 4>{});
      if constexpr (XT != kCodes) {  // codes come in short rows and few tiles
        if (variant == 8) return run(integral_constant<int, 8>{}, integral_constant<int, 8>{});
        if (variant == 12) return run(integral_constant<int, 8>{}, integral_constant<int, 12>{});
        if (variant == 22) return run(integral_constant<int, 8>{}, integral_constant<int, 22>{});
      }
    }
    if constexpr (GROUPED || XT != kCodes) {
      if (variant == -4) return run(integral_constant<int, 4>{}, integral_constant<int, 4>{});
      if (variant == -2) return run(integral_constant<int, 2>{}, integral_constant<int, 4>{});
      if (variant == -1) return run(integral_constant<int, 1>{}, integral_constant<int, 4>{});
    }
    known = false;
  });
  if (!known) return NF4_EUNSUPPORTED;
  return launch_status();
}

}  // namespace

namespace mxdev {

Rows row_plan(const Product& p, int64_t rows) {
  const int64_t units = p.pitch / 64, tiles = rows * ((p.N + 15) / 16);
  Rows r = {kRowWaves, 0};
  // four units to a wave where that leaves each compute unit two workgroups: a tile's waves
  // meet at its end
  while (r.split > 1 && 4 * (r.split / 2) >= units && tiles * (r.split / 2) >= int64_t(2 * kRowWaves) * device_cus())
    r.split /= 2;
  const int64_t each = (units + r.split - 1) / r.split;
  r.units = each <= 4 ? 4 : each <= 8 ? 8 : each <= 12 ? 12 : 22;
  return r;
}

bool fits_rows(const Product& p) { return p.pitch > 0 && p.pitch <= 22 * 64 * kRowWaves; }

nf4_status launch_rows(const Product& p, bool grouped, const void* x, int32_t xt, int64_t K, int32_t y_dtype,
                       hipStream_t st) {
  if (grouped) return launch_typed<kCodes, true>(p, nullptr, 0, y_dtype, st);
  switch (xt) {
    case INT8_BF16: return launch_typed<INT8_BF16, false>(p, x, K, y_dtype, st);
    case INT8_FP16: return launch_typed<INT8_FP16, false>(p, x, K, y_dtype, st);
    case INT8_FP32: return launch_typed<INT8_FP32, false>(p, x, K, y_dtype, st);
    default: return launch_typed<kCodes, false>(p, nullptr, 0, y_dtype, st);
  }
}

}  // namespace mxdev
