// mxfp4_gemv.hip -- activations as they are times 4-bit microscaled weights: up to
// 16 rows (mxfp4_gemv), and the expert layer of a few tokens (mxfp4_moe_mlp).
//
// v_mfma_f32_16x16x32_bf16 with the weights as A: lane i + 16 g holds A[i][8 g .. + 7],
// B likewise with i the column, and D[4 g .. + 3][i].  Every value of the format below
// 2^128 is a bf16 number, so the weights are converted on the way (two codes and their scale an
// instruction) and a lane's block of 32 codes is four matrix instructions' operands; which
// codes of a row a lane has is free as long as both sides agree.  Activations are split
// into bf16 numbers whose sum they are (parts): one for bf16, two for fp16 (8 + 3 bits),
// three for fp32 (8 + 8 + 8).  So each product is exact.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxfp4.h"
#include "mxfp4_format.h"
#include "mxfp4_product.h"
#include "nf4_device.h"
#include "nf4_probe.h"
#include "product_tiles.h"
#include "row_io.h"

namespace {

using namespace nf4dev;
using namespace rowio;
using namespace tiledev;
using namespace mxdev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kUnit = 128;  // elements of K that a wave takes at a time

__device__ __host__ constexpr int parts_of(int dt) { return dt == INT8_BF16 ? 1 : dt == INT8_FP16 ? 2 : 3; }

// A number as bf16 numbers: the upper half of its bits, of what is left, and of what is
// left then, each difference exact.  What is not finite is its own upper half, a NaN a
// quiet one.
__device__ __forceinline__ void split(float f, float (&part)[3]) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, f);
  const bool finite = (bits & 0x7F800000u) != 0x7F800000u;
  part[0] = f != f ? __builtin_nanf("") : __builtin_bit_cast(float, bits & 0xFFFF0000u);
  const float rest = finite ? f - part[0] : 0.0f;
  part[1] = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, rest) & 0xFFFF0000u);
  part[2] = rest - part[1];
}

__device__ __forceinline__ uint32_t upper_halves(float even, float odd) {
  return __builtin_bit_cast(uint32_t, even) >> 16 | (__builtin_bit_cast(uint32_t, odd) & 0xFFFF0000u);
}

// Eight activations to the parts' eight bf16 numbers each.  fp16: without the last three
// bits, and these, both exact in fp16 and in bf16.  An infinity less itself is a NaN: what
// is not finite shows in the sum of what is left of the eight, and is seen to apart (tests
// of every element took as long as the rest: 7 x 4096 x 11008 fp16 16.9 us).
template <int DT>
__device__ __forceinline__ void split_piece(const Piece<DT>& p, u32x4 (&out)[parts_of(DT)]) {
  if constexpr (DT == INT8_BF16) {
    out[0] = p.v[0];
  } else if constexpr (DT == INT8_FP16) {
    f16x2 left = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = p.v[0][i], high = w & 0xFFF8FFF8u;
      const f16x2 h = __builtin_bit_cast(f16x2, high), low = __builtin_bit_cast(f16x2, w) - h;
      left += low;
      out[0][i] = upper_halves(static_cast<float>(h[0]), static_cast<float>(h[1]));
      out[1][i] = upper_halves(static_cast<float>(low[0]), static_cast<float>(low[1]));
    }
    const _Float16 sum = left[0] + left[1];
    if (sum != sum) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = p.v[0][i];
        if ((w & 0x7C00u) == 0x7C00u) {  // a NaN may have its bits among the last three
          out[0][i] |= (w & 0x7FFFu) > 0x7C00u ? 0x0040u : 0u;
          out[1][i] &= 0xFFFF0000u;
        }
        if ((w & 0x7C000000u) == 0x7C000000u) {
          out[0][i] |= (w & 0x7FFF0000u) > 0x7C000000u ? 0x00400000u : 0u;
          out[1][i] &= 0x0000FFFFu;
        }
      }
    }
  } else {
    float left = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float part[2][3];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float f = element<DT>(p, i + k);
        part[k][0] = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, f) & 0xFFFF0000u);
        const float rest = f - part[k][0];
        part[k][1] = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, rest) & 0xFFFF0000u);
        part[k][2] = rest - part[k][1];
        left += part[k][2];
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) out[q][i / 2] = upper_halves(part[0][q], part[1][q]);
    }
    if (left != left) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float a[3], b[3];
        split(element<DT>(p, i), a);
        split(element<DT>(p, i + 1), b);
#pragma unroll
        for (int q = 0; q < 3; ++q) out[q][i / 2] = upper_halves(a[q], b[q]);
      }
    }
  }
}

// Eight codes of a block whose scale is s.
__device__ __forceinline__ bf16x8 weights8(uint32_t c, float s) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// Sixteen channels of weights, for a wave: codes as they are loaded, lane 4 i + g 16 bytes
// g of row i's 64, so that four lanes read them in a row.
struct Channels {
  __amdgpu_buffer_rsrc_t codes, scales;
  uint32_t code_at, scale_at;
};

// Channels c0 .. c0 + wide - 1 (16 at most, none for wide <= 0: zeros) of the rows of
// codes at q.
__device__ __forceinline__ Channels channels(const uint8_t* q, const uint8_t* s, int64_t c0, int64_t wide, int64_t pitch,
                                             int64_t steps) {
  const int lane = threadIdx.x & 63;
  const int64_t n = min(wide, int64_t(16));
  return Channels{rsrc(q + c0 * pitch, static_cast<uint32_t>(n > 0 ? n * pitch : 0)),
                  rsrc(s + (c0 >> 5) * steps * 256,
                       static_cast<uint32_t>(n > 0 ? (((c0 + n + 31) >> 5) - (c0 >> 5)) * steps * 256 : 0)),
                  static_cast<uint32_t>((lane >> 2) * pitch + (lane & 3) * 16),
                  scale_from(c0, c0 + (lane & 15), steps, 0)};
}

template <int CT>
struct Tiles {
  Channels ch[CT];
};

struct Loaded {
  i32x4 codes;
  uint32_t scales;
};

__device__ __forceinline__ Loaded load_unit(const Channels& c, int unit, bool in) {
  return {__builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(c.codes, in ? c.code_at + 64 * unit : kNever, 0, 0)),
          __builtin_amdgcn_raw_buffer_load_b32(c.scales, in ? c.scale_at + 128 * unit : kNever, 0, 0)};
}

// The lane's block of a unit: 32 codes to lane i + 16 g, as four operands.  EIGHT: of a
// pair of eight channels, the second unit's as rows 8 to 15.
template <bool EIGHT = false>
__device__ __forceinline__ void operands(const Loaded& l, bf16x8 (&a)[4]) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int from = 4 * (EIGHT ? 8 * (lane & 7) + 4 * (lane >> 3 & 1) + g : 4 * (lane & 15) + g);  // a lane's number times 4
  const float s = scale_value(l.scales >> (8 * g) & 255);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int w = l.codes[e];
    a[e] = weights8(static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(from, w)), s);
  }
}

// ---------------------------------------------------------------------------
// Rows in LDS (gemv and up): a workgroup keeps `rows` rows' parts, `width` elements of
// them at a time, for its waves' products: [part][row][width + 8] bf16 numbers, the
// eight so that a chunk of 16 rows lies in different banks.
// ---------------------------------------------------------------------------
__device__ __host__ __forceinline__ int lds_row(int width) { return 2 * width + 16; }

// Elements first .. first + width - 1 of rows row(0), row(1), ... of K each (zeros from K
// on), by all threads of the workgroup, several loads of each in flight (as many as the
// registers beside CT tiles' weights leave).
template <int XT, int CT, class Row>
__device__ __forceinline__ void stage_rows(uint8_t* lds, int rows, int64_t first, int width, int64_t K, Row&& row) {
  constexpr int kParts = parts_of(XT), kAtOnce = XT == INT8_FP32 ? (CT > 1 ? 2 : 3) : XT == INT8_FP16 ? (CT > 1 ? 4 : 6) : (CT > 1 ? 4 : 8);
  const int pieces = width / 8, all = rows * pieces, pitch = lds_row(width);
  for (int i0 = threadIdx.x; i0 < all; i0 += kAtOnce * kThreads) {
    Piece<XT> v[kAtOnce];
    int to[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * kThreads;
      v[k] = Piece<XT>{};
      if (i >= all) continue;
      const int r = i / pieces, c = i - r * pieces;
      to[k] = r * pitch + 16 * c;
      const int64_t at = first + 8 * c;
      if (at < K) v[k] = load_piece<XT>(row(r), at, K);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (i0 + k * kThreads >= all) break;
      u32x4 part[kParts];
      split_piece<XT>(v[k], part);
#pragma unroll
      for (int q = 0; q < kParts; ++q) *reinterpret_cast<u32x4*>(lds + q * rows * pitch + to[k]) = part[q];
    }
  }
}

// The units of a wave in its own order: it starts `turn` units after the first, so that
// waves of other channels read other memory channels than it (a power of two from one
// row to the next leads a unit's 16 rows to few of them).
struct Order {
  int from, count, turn;
  __device__ __forceinline__ int operator()(int i) const {
    const int u = i + turn;
    return from + (u < count ? u : u - count);
  }
};

// Eight channels for a wave, as Channels: a pair of units at a time, lane 8 i + j 16 bytes j
// of row i's 128.
__device__ __forceinline__ Channels eight_channels(const uint8_t* q, const uint8_t* s, int64_t c0, int64_t wide,
                                                   int64_t pitch, int64_t steps) {
  const int lane = threadIdx.x & 63;
  const int64_t n = min(wide, int64_t(8));
  return Channels{rsrc(q + c0 * pitch, static_cast<uint32_t>(n > 0 ? n * pitch : 0)),
                  rsrc(s + (c0 >> 5) * steps * 256,
                       static_cast<uint32_t>(n > 0 ? (((c0 + n + 31) >> 5) - (c0 >> 5)) * steps * 256 : 0)),
                  static_cast<uint32_t>((lane >> 3) * pitch + (lane & 7) * 16),
                  scale_from(c0, c0 + (lane & 7), steps, 0)};
}

// units: of a row; the second of the last pair may lie past it, and is zeros.
__device__ __forceinline__ Loaded load_pair(const Channels& c, int pair, int units, bool in) {
  const int lane = threadIdx.x & 63, unit = 2 * pair + (lane >> 3 & 1);
  const bool codes = in && 2 * pair + (lane >> 2 & 1) < units;
  return {__builtin_bit_cast(i32x4,
                             __builtin_amdgcn_raw_buffer_load_b128(c.codes, codes ? c.code_at + 128 * pair : kNever, 0, 0)),
          __builtin_amdgcn_raw_buffer_load_b32(c.scales, in && unit < units ? c.scale_at + 128 * unit : kNever, 0, 0)};
}

// Adds to the rows' columns those of their other parts, where these stand beside them.
template <int PARTS, int CT>
__device__ __forceinline__ void join_parts(f32x4 (&v)[CT], bool together, int rows) {
  if constexpr (PARTS > 1) {
    if (!together) return;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const float each[4] = {v[c][0], v[c][1], v[c][2], v[c][3]};
#pragma unroll
      for (int k = 1; k < PARTS; ++k) {
        const int from = (threadIdx.x & 63) + k * rows;
        v[c] += f32x4{__shfl(each[0], from), __shfl(each[1], from), __shfl(each[2], from), __shfl(each[3], from)};
      }
    }
  }
}

// Streams tiles of 16 channels (CT of each, which share the rows) through a workgroup,
// kWaves / SPLIT of them at a time, whose SPLIT waves share K: a step is UNITS units of
// each wave, neighbouring waves' next to each other, so that the workgroup reads its rows
// of weights in a row.  While a step is multiplied the next one's weights, of the next tile
// at a tile's end, are asked for.
//
//  tiles, first, apart : the workgroup takes the groups of tiles first, first + apart, ...
//                        below tiles
//  tile(t)             : the channels of tile t
//  rows_at(unit)       : has the rows' elements from this unit on put into LDS (between
//                        barriers), `width` of them (whole steps), zeros past K
//  done(t, acc)        : takes a tile's sums, in one wave (t < tiles)
template <int PARTS, int CT, int SPLIT, int UNITS, class Tile, class RowsAt, class Done>
__device__ __forceinline__ void stream_tiles(int units, int64_t tiles, int64_t first, int64_t apart, const uint8_t* lds,
                                             int rows, int width, f32x4 (&sums)[2][kWaves][CT][64], Tile&& tile,
                                             RowsAt&& rows_at, Done&& done) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  constexpr int kStep = SPLIT * UNITS, kGroup = kWaves / SPLIT;
  const int part = wave % SPLIT;
  const int steps = max(1, (units + kStep - 1) / kStep), held = width / kUnit;
  // a wave's units of a step: from `mine` on, apart_of(u) further
  const int mine = UNITS == 1 ? part : 2 * part;
  auto apart_of = [](int u) { return 2 * SPLIT * (u >> 1) + (u & 1); };
  Loaded w[UNITS][CT];
  auto load = [&](const Channels (&ch)[CT], int u, int step, bool in) {
    const int at = kStep * step + mine + apart_of(u);
#pragma unroll
    for (int c = 0; c < CT; ++c) w[u][c] = load_unit(ch[c], at, in && at < units);
  };
  // t: the wave's tile; the workgroup goes on while the group's first is one
  int64_t t = first * kGroup + wave / SPLIT;
  auto some = [&](int64_t at) { return at - wave / SPLIT < tiles; };
  Tiles<CT> next = tile(t);
#pragma unroll
  for (int u = 0; u < UNITS; ++u) load(next.ch, u, 0, true);
  // the rows' parts are columns of one product each where there are 16 at most; else each
  // part is multiplied by itself
  const int pitch = lds_row(width), columns = PARTS * rows <= 16 ? PARTS * rows : rows;
  const bool together = PARTS > 1 && columns > rows;
  const uint8_t* x = lds + min(lane & 15, columns - 1) * pitch + 64 * (lane >> 4) + 2 * kUnit * mine;
  f32x4 acc[CT] = {};
  int step = 0, turn = 0, base = -1;
  while (some(t)) {
    if (kStep * step - base >= held || kStep * step < base || base < 0) {  // (once where all are held)
      base = kStep * step;
      rows_at(base);
    }
    const bool last = step + 1 == steps;
    const int64_t next_t = last ? t + apart * kGroup : t;
    if (last) next = tile(next_t);
    const uint8_t* xs = x + 2 * kUnit * (kStep * step - base);
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      bf16x8 a[CT][4];
#pragma unroll
      for (int c = 0; c < CT; ++c) operands(w[u][c], a[c]);
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        if (k == 0 || !together) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bf16x8 b = *reinterpret_cast<const bf16x8*>(xs + k * rows * pitch + 2 * kUnit * apart_of(u) + 16 * e);
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[c][e], b, acc[c], 0, 0, 0);
          }
        }
      }
      // the products first, then the loads into the registers that they free: the
      // other way round the compiler takes twice the registers
      __builtin_amdgcn_sched_barrier(0);
      load(next.ch, u, last ? 0 : step + 1, some(next_t));
    }
    if (!last) {
      ++step;
      continue;
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) settled(acc[c]);
    if constexpr (SPLIT == 1) {
      join_parts<PARTS>(acc, together, rows);
      if (t < tiles) done(t, acc);
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[c] = f32x4{};
    } else {
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        sums[turn & 1][wave][c][lane] = acc[c];
        acc[c] = f32x4{};
      }
      __syncthreads();
      // one of a tile's waves a turn adds up, in the waves' order; its buffer is written
      // again two turns later, after a barrier that this wave reaches when it is through
      if (part == (turn & (SPLIT - 1)) && t < tiles) {
        f32x4 sum[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          sum[c] = sums[turn & 1][wave - part][c][lane];
#pragma unroll
          for (int v = 1; v < SPLIT; ++v) sum[c] += sums[turn & 1][wave - part + v][c][lane];
        }
        join_parts<PARTS>(sum, together, rows);
        done(t, sum);
      }
    }
    t = next_t;
    step = 0;
    ++turn;
  }
}

// ---------------------------------------------------------------------------
// Up to 16 rows that fit LDS as a whole.  Bound by the weights' stream: 1 x 11008 x 4096
// bf16 7.9 us (24 MB, a plain read of as much 5.2), 1 x 44032 x 4096 19.9 (95.5 MB, 15.8).
// ---------------------------------------------------------------------------
struct Gemv {
  const void* x;
  const uint8_t* wq;
  const uint8_t* ws;
  void* y;
  int64_t M, N, K, pitch, steps;
  int width;
};

template <int XT, int DT, int SPLIT, int UNITS>
__global__ __launch_bounds__(kThreads, 4) void mx_gemv_kernel(Gemv p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];
  __shared__ f32x4 s_sum[2][kWaves][1][64];
  const int lane = threadIdx.x & 63, rows = static_cast<int>(p.M);
  stream_tiles<parts_of(XT), 1, SPLIT, UNITS>(
      static_cast<int>(p.pitch / 64), (p.N + 15) / 16, blockIdx.x, gridDim.x, s_x, rows, p.width, s_sum,
      [&](int64_t t) { return Tiles<1>{{channels(p.wq, p.ws, 16 * t, p.N - 16 * t, p.pitch, p.steps)}}; },
      [&](int unit) {
        __syncthreads();  // every wave is through with the rows before
        stage_rows<XT, 1>(s_x, rows, int64_t(kUnit) * unit, p.width, p.K,
                       [&](int r) { return static_cast<const char*>(p.x) + r * p.K * dtype_bytes(XT); });
        __syncthreads();
      },
      [&](int64_t t, const f32x4 (&sum)[1]) {
        const int64_t n = 16 * t + 4 * (lane >> 4);
        const int left = static_cast<int>(min(p.N - n, int64_t(4)));
        if ((lane & 15) >= rows || left <= 0) return;
        const float f[4] = {sum[0][0], sum[0][1], sum[0][2], sum[0][3]};
        store_four<DT>(p.y, (lane & 15) * p.N + n, left, f);
      });
}

// A wave's piece of LDS: rows of a unit at a pitch of 272 bytes (so that a chunk of 16
// rows lies in different banks), the parts one after the other.
constexpr int kLdsRow = 2 * kUnit + 16;

// Rows that do not fit LDS as a whole: a workgroup goes through its tiles of 16 channels with
// K shared by its waves, two units each in turn, and every wave brings the rows of its units
// itself, through registers and a piece of LDS of its own: no wave waits for another's rows
// (in LDS a stretch at a time, between barriers, 16 x 11008 x 4096 bf16 took 17.2 us and 7
// x 4096 x 11008 fp16 16.6; here 14.4 and 13.7, of which half is splitting the rows again in
// every workgroup; to split them once takes a launch of its own and a workspace, which the
// call has not).  Rows that do fit are split once for all of a workgroup's tiles: 8
// x 11008 x 4096 bf16 9.1 us and here 12.2.  RU: loads of a lane for a unit's rows (four
// rows each).
template <int XT, int RU>
constexpr int wide_waves() {
  return RU * (XT == INT8_FP32 ? 2 : 1) > 2 ? 8 : 16;
}

template <int XT, int DT, int RU>
__global__ __launch_bounds__((64 * wide_waves<XT, RU>()), (wide_waves<XT, RU>() / 4)) void mx_gemv_wide_kernel(Gemv p) {
  constexpr int kParts = parts_of(XT), kRows = 4 * RU, kWide = wide_waves<XT, RU>(), kAhead = 2;
  constexpr bool kTogether = kParts * kRows <= 16;  // a row's parts as columns of one product
  __shared__ __attribute__((aligned(16))) uint8_t s_x[kWide][kParts * kRows * kLdsRow];
  __shared__ f32x4 s_sum[2][kWide][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int rows = static_cast<int>(p.M), units = static_cast<int>(p.pitch / 64), pairs = (units + 1) / 2;
  const int each = (pairs + kWide - 1) / kWide;  // pairs of a wave in a tile, some past the row
  const int64_t tiles = (p.N + 15) / 16;
  const int turns = static_cast<int>((tiles - blockIdx.x + gridDim.x - 1) / gridDim.x), all = turns * each;
  const char* row[RU];
#pragma unroll
  for (int j = 0; j < RU; ++j)
    row[j] = static_cast<const char*>(p.x) + min(4 * j + (lane >> 4), rows - 1) * p.K * dtype_bytes(XT);
  auto tile = [&](int64_t t) {
    const int64_t at = min(t, tiles - 1);
    return channels(p.wq, p.ws, 16 * at, t < tiles ? p.N - 16 * at : 0, p.pitch, p.steps);
  };
  Loaded w[kAhead][2];
  Piece<XT> x[kAhead][2][RU];
  int64_t t = blockIdx.x, next_t = t;
  int step = 0, next_step = 0, turn = 0;
  Channels next = tile(t);
  auto load = [&](int d) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int unit = 2 * (wave + kWide * next_step) + i;
      const bool in = next_t < tiles && unit < units;
      w[d][i] = load_unit(next, unit, in);
      const int64_t at = kUnit * unit + 8 * (lane & 15);
#pragma unroll
      for (int j = 0; j < RU; ++j) {
        x[d][i][j] = Piece<XT>{};
        if (in && 4 * j < rows && at < p.K) x[d][i][j] = load_piece<XT>(row[j], at, p.K);
      }
    }
    if (++next_step == each) {
      next_step = 0;
      next_t += gridDim.x;
      next = tile(next_t);
    }
  };
  f32x4 acc = {};
  auto take = [&](int d) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (2 * (wave + kWide * step) + i >= units) break;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int j = 0; j < RU; ++j) {
        if (4 * j >= rows) break;
        u32x4 part[kParts];
        split_piece<XT>(x[d][i][j], part);
#pragma unroll
        for (int k = 0; k < kParts; ++k)
          *reinterpret_cast<u32x4*>(s_x[wave] + (k * kRows + 4 * j + (lane >> 4)) * kLdsRow + (lane & 15) * 16) = part[k];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      bf16x8 a[4];
      operands(w[d][i], a);
      constexpr int kColumns = kTogether ? kParts * kRows : kRows;
      const uint8_t* h = s_x[wave] + min(lane & 15, kColumns - 1) * kLdsRow + 64 * (lane >> 4);
#pragma unroll
      for (int k = 0; k < (kTogether ? 1 : kParts); ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              a[e], *reinterpret_cast<const bf16x8*>(h + k * kRows * kLdsRow + 16 * e), acc, 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto advance = [&] {
    if (++step < each) return;
    settled(acc);
    s_sum[turn & 1][wave][lane] = acc;
    acc = f32x4{};
    __syncthreads();
    // one of the waves a turn adds up, in the waves' order; its buffer is written again two
    // turns later, after a barrier that this wave reaches when it is through
    if (wave == turn % kWide) {
      f32x4 sum[1] = {s_sum[turn & 1][0][lane]};
#pragma unroll 3
      for (int v = 1; v < kWide; ++v) sum[0] += s_sum[turn & 1][v][lane];
      join_parts<kParts>(sum, kTogether, kRows);
      const int64_t n = 16 * t + 4 * (lane >> 4);
      const int left = static_cast<int>(min(p.N - n, int64_t(4)));
      const float f[4] = {sum[0][0], sum[0][1], sum[0][2], sum[0][3]};
      if ((lane & 15) < rows && left > 0) store_four<DT>(p.y, (lane & 15) * p.N + n, left, f);
    }
    step = 0;
    t += gridDim.x;
    ++turn;
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) load(d);
  // (the last ones apart: with a way out in the middle of the loop the compiler has each
  // turn of it wait for all loads)
  int i = 0;
  for (; i + kAhead - 1 < all; i += kAhead) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      take(d);
      load(d);
      advance();
    }
  }
#pragma unroll
  for (int d = 0; d < kAhead - 1; ++d)
    if (i + d < all) {
      take(d);
      advance();
    }
}

// ---------------------------------------------------------------------------
// The expert layer.  Both kernels first see from the ids which tokens go to which
// expert: a mask of tokens to each.  The experts that have any are numbered in their
// order, and their (expert, token) pairs too: these are the rows of what lies between the
// two products (h).
//
//  up:    a workgroup takes tiles of an expert's 16 channels (of the gate and of the
//         others) and its tokens, as the kernel above.  act(v) times the router's weight
//         goes to h as parts.
//  down:  a workgroup takes 16 or 8 channels of y.  Its waves share the experts' F, one expert
//         after the other without a pause in their weights' stream, and add each's sums
//         to those of the tokens that it has.
//
// Bound by the weights' streams: 1 token, 2 of 8 experts of 4096 x 11008, gated: up 24.4 us
// (95.5 MB, a plain read 15.8), down 16.1 (48 MB, 8.5); 16 tokens, 4 of 64 experts of 2048
// x 1024: 20.1 and 15.7 (92 and 46 MB).  With K of the way down shared by workgroups and
// joined in a third launch that took 14.5 + 4.6 us (64 tokens 83 in all, here 92), with a
// join by the last workgroup to arrive 80.
// ---------------------------------------------------------------------------
constexpr int kMaxTokens = 64, kMaxTopK = 32;

struct Mlp {
  const void* x;
  const uint8_t* w1q;
  const uint8_t* w1s;
  const uint8_t* w2q;
  const uint8_t* w2s;
  const void* ids;
  const float* weights;
  void* y;
  uint16_t* h;  // [rows][parts][h_width]
  int64_t H, F, h_width;
  int64_t pitch1, steps1, pitch2, steps2;
  int T, top_k, experts, id_bytes, gated;
  int rows, lds;  // of up: rows at a time (16 at most), bytes for them
};

// What h is kept in: 16 bits of each number, or all of fp32.  16 bits are off by 2^-17 of a
// number at most, where the output's own rounding is off by 2^-9 (bf16) or 2^-12 (fp16): one
// token's 2 of 8 experts of 4096 x 11008 in bf16 differ by 1.6e-4 of their norm from fp32 all the
// way, flips of last bits, and both are 1.7e-3 from the exact outputs.  Two parts of four rows
// stand side by side in eight columns; three would not.
__device__ __host__ constexpr int h_parts(int dt) { return dt == INT8_FP32 ? 3 : 2; }

struct Routing {
  uint32_t masks[kMaxExperts][2];  // of an expert's tokens
};

__device__ __forceinline__ int64_t id_of(const Mlp& p, int slot) {
  return p.id_bytes == 8 ? static_cast<const int64_t*>(p.ids)[slot] : static_cast<const int32_t*>(p.ids)[slot];
}

// Fills the masks; past it every wave may read them.
__device__ __forceinline__ void read_routing(const Mlp& p, Routing& r) {
  // (the ids are asked for first: the kernel can do nothing without them)
  const int slots = p.T * p.top_k;
  int64_t e = threadIdx.x < slots ? id_of(p, threadIdx.x) : -1;
  for (int i = threadIdx.x; i < p.experts; i += blockDim.x) r.masks[i][0] = r.masks[i][1] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < slots; s += blockDim.x) {
    if (s != threadIdx.x) e = id_of(p, s);
    const int t = s / p.top_k;
    if (e >= 0 && e < p.experts) atomicOr(&r.masks[e][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
}

__device__ __forceinline__ uint64_t mask_of(const Routing& r, int e) {
  return static_cast<uint64_t>(r.masks[e][1]) << 32 | r.masks[e][0];
}

// The experts' tokens in segments of ROWS at most, in order: the expert, the segment's
// first row among the expert's, and that row's place in h.
template <int ROWS>
struct Segments {
  static constexpr int kMost = kMaxExperts + (ROWS < kMaxTokens ? kMaxTokens * kMaxTopK / ROWS : 0);
  uint16_t expert[kMost], first[kMost], place[kMost];
  int count;
};

// Past it every wave may read the masks and the segments.
template <int ROWS>
__device__ __forceinline__ void read_segments(const Mlp& p, Routing& r, Segments<ROWS>& s) {
  read_routing(p, r);
  const int lane = threadIdx.x;
  if (lane < 64) {
    int segments = 0, rows = 0;
    for (int base = 0; base < p.experts; base += 64) {
      const int mine = base + lane < p.experts ? __builtin_popcountll(mask_of(r, base + lane)) : 0;
      const int own = (mine + ROWS - 1) / ROWS;
      int in = own << 16 | mine;  // (2048 pairs at most)
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(in, d);
        if (lane >= d) in += o;
      }
      for (int i = 0; i < own; ++i) {
        const int at = segments + (in >> 16) - own + i;
        s.expert[at] = static_cast<uint16_t>(base + lane);
        s.first[at] = static_cast<uint16_t>(ROWS * i);
        s.place[at] = static_cast<uint16_t>(rows + (in & 0xFFFF) - mine + ROWS * i);
      }
      const int all = __shfl(in, 63);
      segments += all >> 16;
      rows += all & 0xFFFF;
    }
    if (lane == 0) s.count = segments;
  }
  __syncthreads();
}

template <int DT, bool GATED, int SPLIT, int UNITS>
__global__ __launch_bounds__(kThreads, 4) void mx_up_kernel(Mlp p) {
  constexpr int CT = GATED ? 2 : 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];
  __shared__ f32x4 s_sum[2][kWaves][CT][64];
  __shared__ Routing s_routing;
  __shared__ int s_token[kMaxTokens];     // the expert's
  __shared__ float s_weight[kMaxTokens];  // the router's, of these
  read_routing(p, s_routing);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  // the blockIdx.y'th expert that has tokens, and the pairs before it
  int expert = -1, pairs = 0;
  {
    int seen = 0;
    for (int base = 0; base < p.experts && expert < 0; base += 64) {
      const uint64_t mine = base + lane < p.experts ? mask_of(s_routing, base + lane) : 0;
      uint64_t live = __ballot(mine != 0);
      const int n = __builtin_popcountll(live), want = static_cast<int>(blockIdx.y) - seen;
      int count = __builtin_popcountll(mine);
      if (want < n) {
        for (int i = 0; i < want; ++i) live &= live - 1;
        const int at = __builtin_ctzll(live);
        expert = base + at;
        if (lane >= at) count = 0;
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) count += __shfl_xor(count, d);
      pairs += count;
      seen += n;
    }
  }
  if (expert < 0) return;
  expert = __builtin_amdgcn_readfirstlane(expert);
  pairs = __builtin_amdgcn_readfirstlane(pairs);
  const uint64_t mask = mask_of(s_routing, expert);
  const int tokens = __builtin_amdgcn_readfirstlane(__builtin_popcountll(mask));
  if (wave == 0 && (mask >> lane & 1)) s_token[__builtin_popcountll(mask & ((uint64_t(1) << lane) - 1))] = lane;
  __syncthreads();

  const int units = static_cast<int>(p.pitch1 / 64);
  for (int t0 = 0; t0 < tokens; t0 += p.rows) {
    const int rows = min(tokens - t0, p.rows);
    // as many steps of the rows as there are and have room
    constexpr int kStep = SPLIT * UNITS;
    const int room = (p.lds / (rows * parts_of(DT)) - 16) / (2 * kUnit) / kStep, steps = (units + kStep - 1) / kStep;
    const int width = kUnit * kStep * min(room, steps);
    if (t0 > 0) __syncthreads();  // the sums before have been read
    stream_tiles<parts_of(DT), CT, SPLIT, UNITS>(
        units, p.h_width / 16, blockIdx.x, gridDim.x, s_x, rows, width, s_sum,
        [&](int64_t t) {
          Tiles<CT> r;
#pragma unroll
          for (int c = 0; c < CT; ++c)
            r.ch[c] = channels(p.w1q, p.w1s, expert * (CT * p.F) + c * p.F + 16 * t, p.F - 16 * t, p.pitch1, p.steps1);
          return r;
        },
        [&](int unit) {
          __syncthreads();  // every wave is through with the rows before
          if (unit == 0 && t0 == 0 && threadIdx.x < tokens) {
            // a few loads one after the other, while the first weights are on their way
            float weight = 0.0f;
            for (int j = 0; j < p.top_k; ++j) {
              const int s = s_token[threadIdx.x] * p.top_k + j;
              if (id_of(p, s) == expert) weight += p.weights ? p.weights[s] : 1.0f;
            }
            s_weight[threadIdx.x] = weight;
          }
          stage_rows<DT, CT>(s_x, rows, int64_t(kUnit) * unit, width, p.H, [&](int r) {
            return static_cast<const char*>(p.x) + s_token[t0 + r] * p.H * dtype_bytes(DT);
          });
          __syncthreads();
        },
        [&](int64_t t, const f32x4 (&sum)[CT]) {
          if ((lane & 15) >= rows) return;
          const float weight = s_weight[t0 + (lane & 15)];
          constexpr int kParts = h_parts(DT);
          uint32_t out[kParts][2];
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            float part[2][3];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float gate = sum[0][e + i], other = sum[CT - 1][e + i];
              const float a = gate / (1.0f + expf(-gate));
              split((GATED ? a * other : a) * weight, part[i]);
              // the last of the parts that are kept is rounded
              if constexpr (kParts == 2) part[i][1] = part[i][1] + part[i][2];
            }
#pragma unroll
            for (int k = 0; k < kParts; ++k)
              out[k][e / 2] =
                  k + 1 < kParts ? upper_halves(part[0][k], part[1][k]) : pack_pair<NF4_BF16>(part[0][k], part[1][k]);
          }
          uint16_t* to = p.h + (pairs + t0 + (lane & 15)) * (kParts * p.h_width) + 16 * t + 4 * (lane >> 4);
#pragma unroll
          for (int k = 0; k < kParts; ++k)
            *reinterpret_cast<uint2*>(to + k * p.h_width) = make_uint2(out[k][0], out[k][1]);
          // Past F the codes are zeros, but their scales are those of the rows behind, the other
          // half's, the next expert's or none's, and may be NaN; and the router's weight may not
          // be finite.  So zeros are written over what came of it.  (By choosing every value,
          // in every tile, up took 0.2-0.8 us longer; to set the zeros before the store takes
          // registers that fp32 with a gate does not have.)
          if (p.F - 16 * t < 16) {
            const int left = static_cast<int>(p.F - 16 * t) - 4 * (lane >> 4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (e >= left)
#pragma unroll
                for (int k = 0; k < kParts; ++k) to[k * p.h_width + e] = 0;
          }
        });
  }
}

// A wave's piece of LDS in down.
template <int DT, int RU>
constexpr int wave_lds() {
  return h_parts(DT) * 4 * RU * kLdsRow;
}

// An expert's rows of h, 4 RU at most, and its channels.
struct Segment {
  Channels ch[1];
  const uint16_t* h;
  int count;
};

// WAVES: of a workgroup; RU: loads of a lane for a unit's rows (four rows each); TT: tiles
// of 16 tokens.  EIGHT: channels of a workgroup, two units of which stand side by side in
// a product: rows and columns 8 to 15 are the second unit's, and of the sums only those
// where both sides are of one unit count.
template <int DT, int WAVES, int RU, int TT, bool EIGHT>
__global__ __launch_bounds__(64 * WAVES, WAVES / 4) void mx_down_kernel(Mlp p) {
  constexpr int kParts = h_parts(DT), kRows = 4 * RU;
  // pairs of units in flight, as registers allow
  constexpr int kAhead = kParts * RU > 8 ? 1 : EIGHT ? 3 : 2;
  constexpr int kChannels = EIGHT ? 8 : 16;
  static_assert(!EIGHT || (RU == 1 && TT == 1 && kParts == 2));
  constexpr int kSumBytes = WAVES * TT * 64 * 16, kWaveLds = (EIGHT ? 2 : 1) * wave_lds<DT, RU>();
  constexpr int kHBytes = WAVES * kWaveLds;
  __shared__ __attribute__((aligned(16))) uint8_t s_h[kHBytes > kSumBytes ? kHBytes : kSumBytes];
  __shared__ Routing s_routing;
  __shared__ Segments<kRows> s_segments;
  read_segments(p, s_routing, s_segments);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int units = static_cast<int>(p.pitch2 / 64), pairs = (units + 1) / 2;
  const int64_t n0 = int64_t(kChannels) * blockIdx.x;
  auto segment = [&](int j) {
    const int expert = __builtin_amdgcn_readfirstlane(s_segments.expert[j]), first = __builtin_amdgcn_readfirstlane(s_segments.first[j]);
    const int tokens = __builtin_amdgcn_readfirstlane(__builtin_popcountll(mask_of(s_routing, expert)));
    const int64_t place = __builtin_amdgcn_readfirstlane(s_segments.place[j]);
    return Segment{{EIGHT ? eight_channels(p.w2q, p.w2s, expert * p.H + n0, p.H - n0, p.pitch2, p.steps2)
                          : channels(p.w2q, p.w2s, expert * p.H + n0, p.H - n0, p.pitch2, p.steps2)},
                   p.h + place * (kParts * p.h_width), min(tokens - first, kRows)};
  };
  // the wave's pairs of units (whole lines) of all segments'
  const int all = s_segments.count * pairs, each = (all + WAVES - 1) / WAVES;
  int at = min(all, wave * each);
  const int end = min(all, at + each);
  uint8_t* lds = s_h + wave * kWaveLds;
  f32x4 total[TT] = {};
  if (at < end) {
    Loaded w[kAhead][EIGHT ? 1 : 2];
    u32x4 x[kAhead][2][RU][kParts];
    int seg = at / pairs, pair = at - seg * pairs;
    int ahead = at, next_seg = seg, next_pair = pair;
    Segment next = segment(seg);
    int count = next.count;
    auto load = [&](int d) {
      if constexpr (EIGHT) w[d][0] = load_pair(next.ch[0], next_pair, units, ahead < end);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int unit = 2 * next_pair + i;
        const bool in = ahead < end && unit < units;
        if constexpr (EIGHT) {
          if (!in) x[d][i][0][0] = x[d][i][0][1] = u32x4{};  // (zeros are multiplied with them)
        } else {
          w[d][i] = load_unit(next.ch[0], unit, in);
        }
#pragma unroll
        for (int j = 0; j < RU; ++j) {
          if (!in || 4 * j >= next.count) continue;
          const uint16_t* h =
              next.h + min(4 * j + (lane >> 4), next.count - 1) * (kParts * p.h_width) + kUnit * unit + 8 * (lane & 15);
#pragma unroll
          for (int k = 0; k < kParts; ++k) x[d][i][j][k] = *reinterpret_cast<const u32x4*>(h + k * p.h_width);
        }
      }
      ++ahead;
      if (++next_pair == pairs && ahead < end) {
        next_pair = 0;
        next = segment(++next_seg);
      }
    };
#pragma unroll
    for (int d = 0; d < kAhead; ++d) load(d);
    f32x4 acc = {};
    auto take = [&](int d) {
      if constexpr (EIGHT) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < kParts; ++k)
            *reinterpret_cast<u32x4*>(lds + (8 * i + 4 * k + (lane >> 4)) * kLdsRow + (lane & 15) * 16) = x[d][i][0][k];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        bf16x8 a[4];
        operands<true>(w[d][0], a);
        const uint8_t* h = lds + (lane & 15) * kLdsRow + 64 * (lane >> 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[e], *reinterpret_cast<const bf16x8*>(h + 16 * e), acc, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        return;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (2 * pair + i >= units) break;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int j = 0; j < RU; ++j) {
          if (4 * j >= count) break;
#pragma unroll
          for (int k = 0; k < kParts; ++k)
            *reinterpret_cast<u32x4*>(lds + (k * kRows + 4 * j + (lane >> 4)) * kLdsRow + (lane & 15) * 16) = x[d][i][j][k];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        bf16x8 a[4];
        operands(w[d][EIGHT ? 0 : i], a);
        // four rows' parts are columns of one product (what the others hold nobody asks for)
        constexpr int kColumns = RU == 1 ? kParts * kRows : kRows;
        const uint8_t* h = lds + min(lane & 15, kColumns - 1) * kLdsRow + 64 * (lane >> 4);
#pragma unroll
        for (int k = 0; k < (RU == 1 ? 1 : kParts); ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                a[e], *reinterpret_cast<const bf16x8*>(h + k * kRows * kLdsRow + 16 * e), acc, 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // After a pair: at the segment's end its sums go to the tokens' columns; the others
    // keep theirs (not by adding zeros: a channel whose weights are NaN leaves the tokens
    // of other experts alone).
    auto advance = [&] {
      ++at;
      if (++pair < pairs && at < end) return;
      const uint64_t mask = mask_of(s_routing, s_segments.expert[seg]);
      const int first = s_segments.first[seg];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int token = 16 * t + (lane & 15);
        const int column = __builtin_popcountll(mask & ((uint64_t(1) << token) - 1)) - first;
        const bool has = (mask >> token & 1) && column >= 0 && column < kRows;
        // (of eight channels, those of the lanes from 32 on are the second unit's)
        const int from = (has ? column : 0) + (lane & (EIGHT ? 16 : 48));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = acc[e];
          float o = __shfl(v, from);
          if constexpr (EIGHT) {
            o += __shfl(v, from + 4);
            o += __shfl(v, from + 40) + __shfl(v, from + 44);
          } else if constexpr (RU == 1) {
#pragma unroll
            for (int k = 1; k < kParts; ++k) o += __shfl(v, from + k * kRows);
          }
          if (has) total[t][e] += o;
        }
      }
      acc = f32x4{};
      if (at >= end) return;
      pair = 0;
      ++seg;
      count = min(__builtin_popcountll(mask_of(s_routing, s_segments.expert[seg])) - s_segments.first[seg], kRows);
      count = __builtin_amdgcn_readfirstlane(count);
    };
    // (the last ones apart: with a way out in the middle of the loop the compiler has each
    // turn of it wait for all loads)
    while (at + kAhead - 1 < end) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        take(d);
        load(d);
        advance();
      }
    }
#pragma unroll
    for (int d = 0; d < kAhead - 1; ++d)
      if (at < end) {
        take(d);
        advance();
      }
  }
  __syncthreads();  // every wave is through with its rows
  f32x4* s_sum = reinterpret_cast<f32x4*>(s_h);  // [wave][token tile][lane]
#pragma unroll
  for (int t = 0; t < TT; ++t) s_sum[(wave * TT + t) * 64 + lane] = total[t];
  __syncthreads();
  const int token = 16 * wave + (lane & 15);
  const int64_t n = n0 + 4 * (lane >> 4);
  const int left = static_cast<int>(min(p.H - n, int64_t(4)));
  if (wave >= TT || token >= p.T || left <= 0 || (EIGHT && lane >= 32)) return;
  f32x4 sum = s_sum[wave * 64 + lane];
#pragma unroll
  for (int v = 1; v < WAVES; ++v) sum += s_sum[(v * TT + wave) * 64 + lane];
  const float f[4] = {sum[0], sum[1], sum[2], sum[3]};
  store_four<DT>(p.y, token * p.H + n, left, f);
}

// How a workgroup takes its tiles: `split` waves share K, a step is `units` units of each;
// the rows lie in LDS `width` elements (whole steps) at a time.  Whole rows if they have
// room, so that every tile finds them there, if need be with one workgroup to a compute
// unit instead of two.
struct Held {
  int split, units, width;
  int64_t bytes, groups;  // of LDS; of tiles
  bool two;               // workgroups to a compute unit
};
constexpr int64_t kWholeLds = 112 << 10, kHalfLds = 36 << 10;

// tiles: of 16 channels, of all experts that may have tokens.
Held hold(int64_t units, int64_t rows, int64_t tiles) {
  Held h = {};
  auto bytes = [&](int64_t step) { return rows * lds_row(static_cast<int>(kUnit * step)); };
  // four units of each wave to a step, and as many waves to a tile as that leaves work
  // (a tile's waves meet at its end); more where there are few tiles
  h.split = units >= 32 ? 8 : units >= 16 ? 4 : units >= 8 ? 2 : 1;
  while (h.split < kWaves && units > h.split && tiles * h.split < int64_t(kWaves) * device_cus()) h.split *= 2;
  auto per_wave = [&] { return (units + h.split - 1) / h.split; };
  // four or fewer waves take four units each and no others (with_split): where a step of that
  // has no room, eight waves do
  if (bytes(units) > kWholeLds || bytes(4 * h.split) > kWholeLds) h.split = kWaves;
  h.units = h.split < 8 || per_wave() > 2 ? 4 : per_wave() > 1 ? 2 : 1;
  while (h.units > 1 && bytes(h.split * h.units) > kWholeLds) h.units /= 2;
  const int64_t step = h.split * h.units, all = units > 0 ? (units + step - 1) / step : 1;
  const int64_t room = kWholeLds / bytes(step);  // (48 rows' step of 8 units is 97 KiB)
  h.width = static_cast<int>(kUnit * step * (all < room ? all : room));
  h.bytes = bytes(h.width / kUnit);
  h.groups = (tiles + kWaves / h.split - 1) / (kWaves / h.split);
  h.two = h.bytes <= kHalfLds;
  return h;
}

template <class F>
void with_split(const Held& h, F&& f) {
  auto run = [&](auto split, auto units) { f(split, units); };
  if (h.split == 8 && h.units == 1)
    run(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  else if (h.split == 8 && h.units == 2)
    run(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
  else if (h.split == 8)
    run(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
  else if (h.split == 4)
    run(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
  else if (h.split == 2)
    run(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
  else
    run(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
}

// Whether the rows of mxfp4_gemv lie in LDS whole; else each wave brings its own.
bool whole_rows(const Held& h, int64_t units) { return h.width / kUnit >= units; }

int64_t h_width(int64_t F) { return (F + kUnit - 1) / kUnit * kUnit; }

bool known_mlp(int64_t T, int32_t top_k, int32_t experts, int64_t H, int64_t F, int32_t dtype) {
  return T >= 0 && T <= kMaxTokens && top_k >= 1 && top_k <= kMaxTopK && experts >= 0 && experts <= kMaxExperts &&
         H >= 0 && H <= kMaxK && F >= 0 && F <= kMaxK && known_dtype(dtype);
}

size_t h_bytes(int64_t T, int32_t top_k, int64_t F, int32_t dtype) {
  return static_cast<size_t>(T * top_k * h_parts(dtype) * h_width(F) * 2 + 255) / 256 * 256;
}

// The variants of the way down: eight channels to a workgroup; four rows of an expert at a
// time, or sixteen, for up to 16 tokens and for more.
enum Down { kEight, kFourOfFew, kFour, kSixteenOfFew, kSixteen };

struct MlpPlan {
  Held held;            // of up
  int64_t live, tiles;  // experts that may have tokens, tiles of 16 channels of each
  int rows;             // of up, at a time
  Down down;
};

MlpPlan plan_mlp(int64_t T, int32_t top_k, int32_t experts, int64_t H, int64_t F, int32_t dtype) {
  MlpPlan m = {};
  const int64_t slots = T * top_k;
  m.live = experts < slots ? experts : slots;
  m.tiles = h_width(F) / 16;
  // rows at a time: twice as many as an expert has on average, eight at least
  const int64_t often = m.live > 0 ? 2 * ((slots + m.live - 1) / m.live) : 0, some = often < 8 ? 8 : often < 16 ? often : 16;
  m.rows = static_cast<int>(T < some ? T : some);
  m.held = hold(pitch_of(H) / 64, m.rows * parts_of(dtype), m.tiles * m.live);
  // few rows to an expert: four at a time
  const bool four = T <= 4 || slots <= 2 * m.live;
  // eight channels to a workgroup where sixteen would leave half of the compute units without
  // any, for twice the reads of h: 16 tokens' 4 of 64 experts of 2048 x 1024 15.7 us, with
  // sixteen 18.0; one token's 2 of 8 of 2048 x 5632 both launches 21.9 and 21.8
  const bool eight = four && T <= 16 && dtype != INT8_FP32 && (H + 7) / 8 <= device_cus();
  m.down = eight ? kEight : four ? (T <= 16 ? kFourOfFew : kFour) : T <= 16 ? kSixteenOfFew : kSixteen;
  return m;
}

}  // namespace

extern "C" {

nf4_status nf4_probe_mxfp4_rows(int64_t T, int32_t top_k, int32_t experts, int64_t H, int64_t F, int32_t dtype,
                                int32_t* plan) {
  if (!plan || T < 1 || top_k < 1 || experts < 0 || H < 0 || F < 0 || !known_dtype(dtype)) return NF4_EINVAL;
  Held h = {};
  if (experts == 0) {
    if (T > 16) return NF4_EINVAL;
    if (F > kMaxDim || H > kMaxK) return NF4_EUNSUPPORTED;
    h = hold(pitch_of(H) / 64, T * parts_of(dtype), (F + 15) / 16);
    plan[2] = whole_rows(h, pitch_of(H) / 64) ? h.width : 0;
    plan[3] = static_cast<int32_t>(T);
    plan[4] = -1;
  } else {
    if (!known_mlp(T, top_k, experts, H, F, dtype)) return NF4_EUNSUPPORTED;
    const MlpPlan m = plan_mlp(T, top_k, experts, H, F, dtype);
    h = m.held;
    plan[2] = h.width, plan[3] = m.rows, plan[4] = m.down;
  }
  plan[0] = h.split, plan[1] = h.units;
  return NF4_OK;
}

nf4_status mxfp4_gemv(const void* x, int32_t x_dtype, const uint8_t* wq, const uint8_t* ws, int64_t M,
                      int64_t N, int64_t K, void* y, int32_t y_dtype, void* stream) {
  if (M < 0 || M > 16 || N < 0 || K < 0 || !known_dtype(x_dtype) || !known_dtype(y_dtype)) return NF4_EINVAL;
  if (M == 0 || N == 0) return NF4_OK;
  if (!y || (K > 0 && (!x || !wq || !ws))) return NF4_EINVAL;
  if (!aligned(x, dtype_bytes(x_dtype)) || !aligned(wq, 16) || !aligned(ws, 16) || !aligned(y, dtype_bytes(y_dtype)))
    return NF4_EINVAL;
  if (N > kMaxDim || K > kMaxK) return NF4_EUNSUPPORTED;
  const int64_t tiles = (N + 15) / 16, units = pitch_of(K) / 64;
  Gemv p = {x, wq, ws, y, M, N, K, pitch_of(K), steps_of(K), 0};
  const Held held = hold(units, M * parts_of(x_dtype), tiles);
  p.width = held.width;
  if (!whole_rows(held, units)) {
    const dim3 wide(static_cast<uint32_t>(tiles < device_cus() ? tiles : device_cus()));
    with_dtype(x_dtype, [&](auto a) {
      with_dtype(y_dtype, [&](auto d) {
        auto run = [&](auto ru) {
          constexpr int XT = decltype(a)::value, RU = decltype(ru)::value;
          hipLaunchKernelGGL((mx_gemv_wide_kernel<XT, decltype(d)::value, RU>), wide, dim3(64 * wide_waves<XT, RU>()), 0,
                             reinterpret_cast<hipStream_t>(stream), p);
        };
        if (M <= 4)
          run(std::integral_constant<int, 1>{});
        else if (M <= 8)
          run(std::integral_constant<int, 2>{});
        else
          run(std::integral_constant<int, 4>{});
      });
    });
    return launch_status();
  }
  const int64_t most = (held.two ? 2 : 1) * device_cus();
  const dim3 grid(static_cast<uint32_t>(held.groups < most ? held.groups : most));
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  with_split(held, [&](auto split, auto u) {
    with_dtype(x_dtype, [&](auto a) {
      with_dtype(y_dtype, [&](auto d) {
        hipLaunchKernelGGL(
            (mx_gemv_kernel<decltype(a)::value, decltype(d)::value, decltype(split)::value, decltype(u)::value>), grid,
            dim3(kThreads), static_cast<uint32_t>(held.bytes), st, p);
      });
    });
  });
  return launch_status();
}

size_t mxfp4_moe_mlp_workspace_size(int64_t T, int32_t top_k, int32_t experts, int64_t H, int64_t F, int32_t dtype) {
  if (!known_mlp(T, top_k, experts, H, F, dtype)) return 0;
  return h_bytes(T, top_k, F, dtype);
}

nf4_status mxfp4_moe_mlp(const void* x, int32_t dtype, const uint8_t* w1q, const uint8_t* w1s,
                         const uint8_t* w2q, const uint8_t* w2s, const void* ids, int32_t id_bytes,
                         const float* weights, int64_t T, int32_t top_k, int32_t experts, int64_t H,
                         int64_t F, int32_t gated, void* y, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (T < 0 || top_k < 1 || experts < 0 || H < 0 || F < 0 || !known_dtype(dtype) ||
      (id_bytes != 4 && id_bytes != 8) || !aligned(workspace, 256))
    return NF4_EINVAL;
  if (T == 0 || H == 0) return NF4_OK;
  if (!x || !y || !ids || !aligned(x, dtype_bytes(dtype)) || !aligned(y, dtype_bytes(dtype)) ||
      !aligned(ids, id_bytes) || !aligned(weights, 4))
    return NF4_EINVAL;
  if (experts > 0 && F > 0 && (!w1q || !w1s || !w2q || !w2s)) return NF4_EINVAL;
  if (!aligned(w1q, 16) || !aligned(w1s, 16) || !aligned(w2q, 16) || !aligned(w2s, 16)) return NF4_EINVAL;
  if (!known_mlp(T, top_k, experts, H, F, dtype) || experts * H > kMaxDim || experts * F * (gated ? 2 : 1) > kMaxDim)
    return NF4_EUNSUPPORTED;
  const size_t need = h_bytes(T, top_k, F, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return NF4_EINVAL;
  Mlp p = {};
  p.x = x, p.w1q = w1q, p.w1s = w1s, p.w2q = w2q, p.w2s = w2s, p.ids = ids, p.weights = weights, p.y = y;
  p.h = static_cast<uint16_t*>(workspace);
  p.H = H, p.F = F, p.h_width = h_width(F);
  p.pitch1 = pitch_of(H), p.steps1 = steps_of(H), p.pitch2 = pitch_of(F), p.steps2 = steps_of(F);
  p.T = static_cast<int>(T), p.top_k = top_k, p.experts = F > 0 ? experts : 0, p.id_bytes = id_bytes, p.gated = gated;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const MlpPlan m = plan_mlp(T, top_k, experts, H, F, dtype);
  const Held& held = m.held;
  p.rows = m.rows, p.lds = static_cast<int>(held.bytes);
  const dim3 grid(static_cast<uint32_t>(m.down == kEight ? (H + 7) / 8 : (H + 15) / 16));
  with_dtype(dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    if (p.experts > 0) {
      const int64_t share = ((held.two ? 2 : 1) * device_cus() + m.live - 1) / m.live;
      const int64_t groups = (m.tiles + kWaves / held.split - 1) / (kWaves / held.split);
      const dim3 up(static_cast<uint32_t>(groups < share ? groups : share), static_cast<uint32_t>(m.live));
      with_split(held, [&](auto split, auto u) {
        constexpr int SPLIT = decltype(split)::value, UNITS = decltype(u)::value;
        if (gated)
          hipLaunchKernelGGL((mx_up_kernel<DT, true, SPLIT, UNITS>), up, dim3(kThreads), static_cast<uint32_t>(p.lds), st,
                             p);
        else
          hipLaunchKernelGGL((mx_up_kernel<DT, false, SPLIT, UNITS>), up, dim3(kThreads), static_cast<uint32_t>(p.lds),
                             st, p);
      });
    }
    switch (m.down) {
      case kEight:
        if constexpr (DT != INT8_FP32) hipLaunchKernelGGL((mx_down_kernel<DT, 16, 1, 1, true>), grid, dim3(1024), 0, st, p);
        break;
      case kFourOfFew: hipLaunchKernelGGL((mx_down_kernel<DT, 16, 1, 1, false>), grid, dim3(1024), 0, st, p); break;
      case kFour: hipLaunchKernelGGL((mx_down_kernel<DT, 8, 1, 4, false>), grid, dim3(512), 0, st, p); break;
      case kSixteenOfFew: hipLaunchKernelGGL((mx_down_kernel<DT, 8, 4, 1, false>), grid, dim3(512), 0, st, p); break;
      case kSixteen: hipLaunchKernelGGL((mx_down_kernel<DT, 8, 4, 4, false>), grid, dim3(512), 0, st, p); break;
    }
  });
  return launch_status();
}

}  // extern "C"
