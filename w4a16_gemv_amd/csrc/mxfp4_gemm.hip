// mxfp4_gemm.hip -- the products of two matrices of 4-bit microscaled floats on the
// scaled matrix cores: one matrix (mxfp4_gemm, mxfp4_linear) and rows sorted by
// expert (mxfp4_gemm_grouped).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 with the weights as A (32 channels n x 64 k) and
// the activations as B (64 k x 32 tokens m).  Lane l = i + 32 g holds 32 codes of row
// i of A, 16 bytes, and of B, their scales in a byte of one register each, and of D the
// column i: rows 8 (c / 4) + 4 g + c % 4 for its 16 registers c.  The instruction sums
// over all of its k, so which 32 codes of a row a lane has is free as long as both
// sides agree: here lane group g takes the codes 128 g + 32 p of 256 in the p'th of
// four instructions, so that the four scales that it needs are one dword.
//
// Products of codes and scales are exact; on this device a sum of one instruction was
// within 2^-24 of the exact one, relative to the sum of the magnitudes.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <type_traits>

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

// BYTE: of the scales' dwords.
template <int BYTE>
__device__ __forceinline__ f32x16 mfma32(const i32x4& a, uint32_t sa, const i32x4& b, uint32_t sb, const f32x16& c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(four(a), four(b), c, kFp4, kFp4, BYTE,
                                                         static_cast<int>(sa), BYTE, static_cast<int>(sb));
}
__device__ __forceinline__ f32x16 mfma32(int byte, const i32x4& a, uint32_t sa, const i32x4& b, uint32_t sb,
                                         const f32x16& c) {
  switch (byte) {  // a constant where this is inlined
    case 0: return mfma32<0>(a, sa, b, sb, c);
    case 1: return mfma32<1>(a, sa, b, sb, c);
    case 2: return mfma32<2>(a, sa, b, sb, c);
    default: return mfma32<3>(a, sa, b, sb, c);
  }
}

// Writes a wave's 32 TM tokens from m0 on x 32 TN channels from n0 on, 32 tokens x
// CHANNELS at a time through an LDS region of its own, so that whole lines of y are
// written.  keep(j) is the mask of the lane's token of tile j.
template <int DT, int TM, int TN, int CHANNELS, class Keep>
__device__ __forceinline__ void write_tile(const Product& p, int64_t end, int64_t n0, int64_t m0,
                                           const f32x16 (&acc)[TN][TM], int8_t* lds, Keep&& keep) {
  constexpr int kB = dtype_bytes(DT), kRow = CHANNELS * kB, kTiles = CHANNELS / 32;
  constexpr int kPieces = CHANNELS / 8;          // of eight channels, to a row
  constexpr int kChunks = kRow / 16;             // of 16 bytes, to a row
  // 256 / kRow rows fill the banks; a row's chunks lie at chunk ^ swap(row), so
  // that neither side meets in a bank
  auto swap = [](int r) { return r / (16 / kChunks) & (kChunks - 1); };
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i0 = 0; i0 < TN; i0 += kTiles) {
    const int64_t n1 = n0 + 32 * i0;
    const int64_t wide = min(p.N - n1, int64_t(CHANNELS));
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t m1 = m0 + 32 * j;
      const uint32_t k = keep(j);
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const f32x16& v = acc[i0 + i][j];
          const float f[4] = {v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]};
          const int at = (32 * i + 8 * c + 4 * (lane >> 5)) * kB;
          int8_t* to = lds + (lane & 31) * kRow + (((at >> 4) ^ swap(lane & 31)) << 4) + (at & 15);
          if constexpr (DT == INT8_FP32)
            *reinterpret_cast<float4*>(to) =
                make_float4(masked(f[0], k), masked(f[1], k), masked(f[2], k), masked(f[3], k));
          else
            *reinterpret_cast<uint2*>(to) = make_uint2(pack_pair<DT>(f[0], f[1]) & k, pack_pair<DT>(f[2], f[3]) & k);
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = lane; i < 32 * kPieces; i += 64) {
        const int r = i / kPieces, at = i % kPieces;
        if (m1 + r >= end || 8 * at >= wide) continue;
        Piece<DT> v;
#pragma unroll
        for (int h = 0; h < kB / 2; ++h)
          v.v[h] = *reinterpret_cast<const u32x4*>(lds + r * kRow + (((at * (kB / 2) + h) ^ swap(r)) << 4));
        store_piece<DT>(static_cast<char*>(p.y) + ((m1 + r) * p.N + n1) * kB, 8 * at, wide, v);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
}

// ---------------------------------------------------------------------------
// Large tiles: 256 channels x 256 tokens (or 128).  Four waves, 2 x 2, each with 128
// x 128 outputs in accumulators, which takes all of a compute unit's registers and
// LDS.
//
// 128 bytes of K at a time (a step, 256 codes): the tile's rows and their scales go
// from memory straight to one of two LDS buffers, and from there to the matrix cores,
// a quarter of the step at a time (a part) with the next being read.  One barrier per
// step: it stands before the last part, whose operands are in registers by then, so
// that the other buffer's first operands are read while the matrix cores still work.
// The order of the instructions is given by hand (sched_group_barrier): left alone
// the compiler reads operands right before their use.
//
// LDS: two rows of eight 16-byte chunks fill the 64 banks; chunk c of row r is
// stored at c ^ (r / 2 % 8), so that the sixteen lanes that are served at a
// time, 16 rows of one chunk (reads) or two whole rows (writes), lie in all
// banks once.  The scales follow, a tile of 256 bytes (32 rows) after the other.
//
// Rows past the tile's end are zeros or whatever row is at hand (their outputs
// are not stored); bytes past a row's pitch are zeros on the weights' side, and the
// scales of a step past the last are 2^-127 there.  The steps past the last are loaded
// too: zeros that nothing uses.
// ---------------------------------------------------------------------------
constexpr int kTile = 256;
constexpr int kTileThreads = 256;
constexpr int kDepth = 128;     // bytes of K per step
constexpr int kScaleDepth = 8;  // bytes of a row's scales per step

constexpr int kOutBytes = 4 * 32 * 128;  // LDS that the outputs go through
// A buffer: the codes of the channels and of BM tokens, and the scales behind them.
__device__ __host__ constexpr int tile_codes(int BM) { return (kTile + BM) * kDepth; }
constexpr int kBufferBytes = 2 * kTile * (kDepth + kScaleDepth);

// One tile, or half of one; group: of those that do this share.  s_a, s_b: two buffers
// that the compiler can tell apart: reads of one do not wait for the loads into the other.
template <int DT, bool GROUPED, Share SHARE>
__device__ __forceinline__ void compute_tile(const Product& p, uint32_t group, int8_t* s_a, int8_t* s_b, int8_t* s_out,
                                             uint32_t* s_keep) {
  constexpr int TN = kTile / 64, TM = SHARE == kHalves ? TN / 2 : TN;  // 32 x 32 tiles of a wave
  constexpr int BM = 64 * TM;                      // tokens
  constexpr int LN = kTile / 32, LM = BM / 32;     // 16-byte loads of a thread per step
  constexpr int SN = LN / 4, SM = LM / 4;          // its loads of four scales
  constexpr int kCodes = tile_codes(BM);

  const uint32_t tiles_n = static_cast<uint32_t>((p.N + kTile - 1) / kTile);
  uint32_t tiles_m = static_cast<uint32_t>((p.M + kTile - 1) / kTile);
  if constexpr (GROUPED) tiles_m = count_tiles<kTile>(p);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int row = 8 * wave + (lane >> 3);
  const int chunk = ((lane & 7) ^ (row >> 1 & 7)) * 16;
  const int pitch = static_cast<int>(p.pitch), steps = static_cast<int>(p.steps);
  const uint32_t voff = static_cast<uint32_t>(row * pitch + chunk);

  uint32_t index, half = 0, tm, tn;
  const uint32_t all = tiles_m * tiles_n, whole = whole_tiles(all, p.cus);
  if constexpr (SHARE == kHalves) {
    if (in_quarters(all - whole, p.cus) || !tile_of_group(group, 2 * (all - whole), index)) return;
    half = index & 1;
    index = whole + index / 2;
  } else {
    if (!tile_of_group(group, whole, index)) return;
  }
  locate_tile(index, tiles_m, tiles_n, tm, tn);
  RowTile t = {static_cast<int64_t>(tm) * kTile, min(p.M, static_cast<int64_t>(tm) * kTile + kTile), 0};
  if constexpr (GROUPED) t = find_tile<kTile>(p, tm);
  if constexpr (SHARE == kHalves) {
    t.first += half * BM;
    t.end = min(t.end, t.first + BM);
    if (t.end <= t.first) return;
  }
  const int64_t n0 = static_cast<int64_t>(tn) * kTile, c0 = t.expert * p.N + n0;  // channel of all experts'
  const int64_t wide = min(int64_t(kTile), p.N - n0);
  const uint8_t* w0 = p.wq + c0 * p.pitch;
  const auto rw = rsrc(w0, static_cast<uint32_t>(wide * p.pitch));
  const auto rx = rsrc(GROUPED ? nullptr : p.xq + t.first * p.pitch,
                       static_cast<uint32_t>((t.end - t.first) * p.pitch));
  // (a range that ends with the tile of the last row: c0 may lie anywhere in one)
  const auto rws = rsrc(p.ws + (c0 >> 5) * p.steps * 256,
                        static_cast<uint32_t>((((c0 + wide + 31) >> 5) - (c0 >> 5)) * p.steps * 256));
  const auto rxs = rsrc(GROUPED ? nullptr : p.xs + (t.first >> 5) * p.steps * 256,
                        static_cast<uint32_t>((((t.end + 31) >> 5) - (t.first >> 5)) * p.steps * 256));
  const uint8_t* xrow[GROUPED ? LM : 1];
  const uint8_t* xscale[GROUPED ? SM : 1];
  if constexpr (GROUPED) {
#pragma unroll
    for (int i = 0; i < LM; ++i) {
      const int64_t m = t.first + row + 32 * i;
      const int64_t src = m < t.end ? source_row<true>(p, m) : -1;
      xrow[i] = src >= 0 ? p.xq + src * p.pitch : w0;  // any row that may be read
    }
#pragma unroll
    for (int i = 0; i < SM; ++i) {
      const int64_t m = t.first + 32 * (4 * i + wave) + (lane & 31);
      const int64_t src = m < t.end ? source_row<true>(p, m) : -1;
      xscale[i] = (src >= 0 ? p.xs + scale_at(src, p.steps, 0) : p.ws) + 128 * (lane >> 5);
    }
  }
  uint32_t sw_at[SN];
#pragma unroll
  for (int i = 0; i < SN; ++i) sw_at[i] = scale_from(c0, c0 + 32 * (4 * i + wave) + (lane & 31), p.steps, lane >> 5);
  const uint32_t sx_at = scale_from(0, 32 * wave + (lane & 31), p.steps, lane >> 5);

  // --- memory to LDS: a wave fills eight rows at a time, the channels' first, or 32
  // rows' scales
  auto load = [&](int8_t* buf, int i, int k) {
    if (i >= LN + LM) {
      const int s = i - LN - LM;
      const LdsPtr to = (LdsPtr)(buf + kCodes + (4 * s + wave) * 256);
      const bool in = k < kDepth * steps;
      if (s < SN)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rws, to, 4, in ? sw_at[s < SN ? s : 0] + 2 * k : kNever, 0, 0, 0);
      else if constexpr (GROUPED)
        __builtin_amdgcn_global_load_lds((GlobalPtr)(xscale[GROUPED ? s - SN : 0] + (in ? 2 * k : 0)), to, 4, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rxs, to, 4, in ? sx_at + 2 * k + 4 * (s - SN) * steps * 256 : kNever, 0, 0, 0);
      return;
    }
    const bool in = k + chunk < pitch;
    const uint32_t v = in ? voff + k : kNever;
    const LdsPtr to = (LdsPtr)(buf + (32 * i + 8 * wave) * kDepth);
    if (i < LN)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, to, 16, v + 32 * i * pitch, 0, 0, 0);
    else if constexpr (GROUPED)
      __builtin_amdgcn_global_load_lds((GlobalPtr)(xrow[GROUPED ? i - LN : 0] + (in ? k + chunk : 0)), to, 16, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, to, 16, v + 32 * (i - LN) * pitch, 0, 0, 0);
  };

  // --- LDS to the matrix cores
  const int wn = (wave & 1) * (kTile / 2), wm = (wave >> 1) * (BM / 2);
  i32x4 fw[2][TN], fx[2][TM];
  uint32_t sw[2][TN], sx[2][TM];
  auto fetch = [&](int set, const int8_t* buf, int part) {
    const int at = (lane & 31) * kDepth + (((part + 4 * (lane >> 5)) ^ (lane >> 1 & 7)) * 16);
#pragma unroll
    for (int i = 0; i < TN; ++i)
      fw[set][i] = *reinterpret_cast<const i32x4*>(buf + (wn + 32 * i) * kDepth + at);
#pragma unroll
    for (int i = 0; i < TM; ++i)
      fx[set][i] = *reinterpret_cast<const i32x4*>(buf + (kTile + wm + 32 * i) * kDepth + at);
  };
  auto fetch_scales = [&](int set, const int8_t* buf) {
    const int8_t* at = buf + kCodes + 4 * lane;
#pragma unroll
    for (int i = 0; i < TN; ++i) sw[set][i] = *reinterpret_cast<const uint32_t*>(at + (wn + 32 * i) * kScaleDepth);
#pragma unroll
    for (int i = 0; i < TM; ++i)
      sx[set][i] = *reinterpret_cast<const uint32_t*>(at + (kTile + wm + 32 * i) * kScaleDepth);
  };
  f32x16 acc[TN][TM] = {};
  auto multiply = [&](int set, int scales, int part) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
        acc[i][j] = mfma32(part, fw[set][i], sw[scales][i], fx[set][j], sx[scales][j], acc[i][j]);
  };
  // The step after the next one's loads may start when the barrier has freed its
  // buffer: they are spread over the parts 3, 0 and 1, one to two or more matrix
  // instructions, since four waves' loads in a row would hold up the issue.
  constexpr int kMoves = LN + LM + SN + SM, kThree = (kMoves + 2) / 3, kZero = (kMoves - kThree + 1) / 2;
  constexpr int kOne = kMoves - kThree - kZero;
  auto order = [&](int loads, auto reads) {
#pragma unroll
    for (int i = 0; i < TN + TM; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedRead, decltype(reads)::value, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      if (i < loads) __builtin_amdgcn_sched_group_barrier(kSchedLoad, 1, 0);
      if (i < TN * TM - TN - TM) __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // one step: `now` holds this step's rows, `next` the next one's; `scales` is the set
  // of this step's
  auto step = [&](int8_t* now, int8_t* next, int scales, int k) {
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      fetch((part + 1) & 1, now, part + 1);
      if (part == 0) {
#pragma unroll
        for (int i = kThree; i < kThree + kZero; ++i) load(next, i, (k + 1) * kDepth);
      }
      if (part == 1) {
#pragma unroll
        for (int i = kThree + kZero; i < kMoves; ++i) load(next, i, (k + 1) * kDepth);
      }
      multiply(part & 1, scales, part);
      order(part == 0 ? kZero : part == 1 ? kOne : 0, std::integral_constant<int, 1>{});
    }
    __syncthreads();
    fetch(0, next, 0);
    fetch_scales(scales ^ 1, next);
#pragma unroll
    for (int i = 0; i < kThree; ++i) load(now, i, (k + 2) * kDepth);
    multiply(1, scales, 3);
    order(kThree, std::integral_constant<int, 2>{});  // with the scales
  };

  if (steps > 0) {
#pragma unroll
    for (int i = 0; i < kMoves; ++i) load(s_a, i, 0);
#pragma unroll
    for (int i = 0; i < kThree; ++i) load(s_b, i, kDepth);
    __syncthreads();
    fetch(0, s_a, 0);
    fetch_scales(0, s_a);
    for (int k = 0; k < steps; k += 2) {  // with an odd number the last step is one of zeros
      step(s_a, s_b, 0, k);
      step(s_b, s_a, 1, k + 1);
    }
  }
  if constexpr (GROUPED) {
    const int64_t m = t.first + threadIdx.x;
    s_keep[threadIdx.x] = keep_mask<true>(m < t.end ? source_row<true>(p, m) : -1);
  }
  __syncthreads();
  write_tile<DT, TM, TN, 128 / dtype_bytes(DT)>(
      p, t.end, n0 + wn, t.first + wm, acc, s_out + wave * 32 * 128,
      [&](int j) { return GROUPED ? s_keep[GROUPED ? wm + 32 * j + (lane & 31) : 0] : ~0u; });
}

// The first `halves` workgroups take the halves of a last turn's tiles, the others whole
// tiles.  Halves first: compute units that start with one are out of step with the others,
// so that not all write their outputs at the same time (33 MB a turn), and no launch of
// their own has to wait for the last tile (8192 x 11008 x 4096 bf16: 199.9 us, with a launch
// for each 201.3, in turn on one card).  For rows sorted by expert a turn of workgroups stands
// in front, which are empty where the last turn goes in quarters or whole: 4096 tokens' 2 of 8
// experts of 4096 x 4096 take 109.0 us, with a launch for each 109.8.
//
// Bound by the matrix cores' clock under load and by a turn's start and outputs: a
// turn of 256 tiles takes 1.5 us for 256 of K (5.6 PF, where the instructions alone reach
// 6.2 on random codes) and 11.4 us besides, of which 6 are the outputs at a copy's rate.
// 8192 x 8192 x 8192 takes 244 us (4.5 PF).
template <int DT, bool GROUPED>
__global__ __launch_bounds__(kTileThreads, 1) void mx_tile_kernel(Product p, uint32_t halves) {
  __shared__ __attribute__((aligned(256))) int8_t s_a[kBufferBytes];
  __shared__ __attribute__((aligned(256))) int8_t s_b[kBufferBytes];
  __shared__ __attribute__((aligned(256))) int8_t s_out[kOutBytes];
  __shared__ uint32_t s_keep[GROUPED ? kTile : 1];  // the tokens' masks
  if (blockIdx.x < halves)
    compute_tile<DT, GROUPED, kHalves>(p, blockIdx.x, s_a, s_b, s_out, s_keep);
  else
    compute_tile<DT, GROUPED, kWhole>(p, blockIdx.x - halves, s_a, s_b, s_out, s_keep);
}

// ---------------------------------------------------------------------------
// Small tiles: WM x WN x WK waves, each with TM x TN tiles of 32 x 32; the WK
// waves of a tile share each step's K, 128 / WK bytes each.  Few steps are long
// enough to hide anything, so the chain of a step is kept short: STAGES buffers in
// LDS, each asked for STAGES steps ahead; operands read from LDS a step ahead of
// the matrix instructions that use them; one barrier, at which a wave waits for
// the next step's rows only.  LDS is laid out as for the large tiles.  Bound by the loads
// into a compute unit: a step of 64 x 64 takes 0.15 us for 17 KB (256 x 4096 x 4096: 7.3 us,
// of which 3.2 are a launch's).
// ---------------------------------------------------------------------------
template <int DT, bool GROUPED, int WM, int WN, int WK, int TM, int TN, int STAGES, bool QUARTERS = false>
__global__ __launch_bounds__(64 * WM* WN* WK) void mx_stream_kernel(Product p) {
  constexpr int kWaves = WM * WN * WK, kThreads = 64 * kWaves;
  constexpr int BM = 32 * WM * TM, BN = 32 * WN * TN;
  constexpr int kRows = kThreads / 8;                         // rows that a load of all threads fills
  constexpr int kScaleTiles = (BM + BN) / 32;
  constexpr int LM = BM / kRows, LN = BN / kRows, LS = (kScaleTiles + kWaves - 1) / kWaves;
  constexpr int kLoads = LM + LN + LS;
  static_assert(LM * kRows == BM && LN * kRows == BN);
  constexpr int kB = dtype_bytes(DT);
  constexpr int kCodeBytes = (BM + BN) * kDepth, kStage = kCodeBytes + (BM + BN) * kScaleDepth;
  static_assert(WK == 1 || (TM == 1 && TN == 1));
  __shared__ __attribute__((aligned(256))) int8_t s_rows[STAGES][kStage];
  static_assert(WM * WN * 32 * 32 * TN * kB <= STAGES * kStage);
  int8_t* const s_out = s_rows[0];  // at the end
  __shared__ __attribute__((aligned(256))) f32x4 s_meet[WK > 1 ? (WK - 1) * WM * WN * 256 : 1];

  // tiles of its own, or quarters of the large ones
  constexpr int kM = QUARTERS ? 2 * BM : BM, kN = QUARTERS ? 2 * BN : BN;
  static_assert(!QUARTERS || (kM == kTile && kN == kTile));
  const uint32_t tiles_n = static_cast<uint32_t>((p.N + kN - 1) / kN);
  uint32_t tiles_m = static_cast<uint32_t>((p.M + kM - 1) / kM);
  if constexpr (GROUPED) tiles_m = count_tiles<kM>(p);
  uint32_t index, quarter = 0, tm, tn;
  const uint32_t all = tiles_m * tiles_n;
  if constexpr (QUARTERS) {
    const uint32_t whole = whole_tiles(all, p.cus);
    if (!in_quarters(all - whole, p.cus) || !tile_of_group(blockIdx.x, 4 * (all - whole), index)) return;
    quarter = index & 3;
    index = whole + index / 4;
  } else {
    if (!tile_of_group(blockIdx.x, all, index)) return;
  }
  locate_tile(index, tiles_m, tiles_n, tm, tn);
  RowTile t = {static_cast<int64_t>(tm) * kM, min(p.M, static_cast<int64_t>(tm) * kM + kM), 0};
  if constexpr (GROUPED) t = find_tile<kM>(p, tm);
  const int64_t n0 = static_cast<int64_t>(tn) * kN + (quarter & 1) * BN;
  if constexpr (QUARTERS) {
    t.first += (quarter >> 1) * BM;
    t.end = min(t.end, t.first + BM);
    if (t.end <= t.first || n0 >= p.N) return;
  }

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int row = 8 * wave + (lane >> 3);
  const int chunk = ((lane & 7) ^ (row >> 1 & 7)) * 16;
  const int pitch = static_cast<int>(p.pitch);
  // this workgroup's range of K, in bytes of a row
  int begin = 0, end = pitch;
  if constexpr (!GROUPED) {
    const int each = ((pitch + kDepth - 1) / kDepth + p.splits - 1) / p.splits * kDepth;
    begin = min(pitch, static_cast<int>(blockIdx.y) * each);
    end = min(pitch, begin + each);
  }
  const int64_t c0 = t.expert * p.N + n0;
  const uint8_t* w0 = p.wq + c0 * p.pitch;
  i32x4 rw = range_words(w0, static_cast<uint32_t>(min(int64_t(BN), p.N - n0) * p.pitch));
  i32x4 rx = range_words(GROUPED ? nullptr : p.xq + t.first * p.pitch,
                         static_cast<uint32_t>((t.end - t.first) * p.pitch));
  // scalars that the vector unit has written (range_words) may be read by a load
  // five instructions later; the compiler sees to that for its own loads only
  asm volatile("s_nop 4" : "+s"(rw), "+s"(rx));
  const uint32_t voff = static_cast<uint32_t>(row * pitch + chunk);
  const uint8_t* xrow[GROUPED ? LM : 1];
  if constexpr (GROUPED) {
#pragma unroll
    for (int i = 0; i < LM; ++i) {
      const int64_t m = t.first + row + kRows * i;
      const int64_t src = m < t.end ? source_row<true>(p, m) : -1;
      xrow[i] = src >= 0 ? p.xq + src * p.pitch : w0;  // any row that may be read
    }
  }
  // the lane's row of each tile of scales that its wave loads: the channels' tiles
  // first; waves past the last tile load that one again.  Rows past the end: the last.
  const uint8_t* srow[LS];
  auto scale_tile = [&](int i) { return min(i * kWaves + wave, kScaleTiles - 1); };
#pragma unroll
  for (int i = 0; i < LS; ++i) {
    const int s = scale_tile(i), r = 32 * s + (lane & 31);
    if (s < BN / 32) {
      srow[i] = p.ws + scale_at(min(c0 + r, (t.expert + 1) * p.N - 1), p.steps, 0);
    } else {
      const int64_t src = source_row<GROUPED>(p, min(t.first + r - BN, t.end - 1));
      srow[i] = src >= 0 ? p.xs + scale_at(src, p.steps, 0) : p.ws;
    }
    srow[i] += 128 * (lane >> 5);
  }
  const uint32_t lds0 = lds_address(s_rows[0]);
  // load i of a thread for step k / 128: the channels' rows first, scales last
  auto load = [&](int stage, int i, int k) {
    if (i >= LN + LM) {
      const int s = i - LN - LM;
      lds_load_dword(lds0 + stage * kStage + kCodeBytes + scale_tile(s) * 256, srow[s < 0 ? 0 : s] + (k < end ? 2 * k : 0));
      return;
    }
    const bool in = k + chunk < end;
    const uint32_t v = in ? voff + k : kNever, to = lds0 + stage * kStage + (8 * wave + kRows * i) * kDepth;
    if (i < LN)
      lds_load(to, rw, v + kRows * i * pitch);
    else if constexpr (GROUPED)
      lds_load(to, reinterpret_cast<const int8_t*>(xrow[GROUPED ? i - LN : 0] + (in ? k + chunk : 0)));
    else
      lds_load(to, rx, v + kRows * (i - LN) * pitch);
  };

  const int wk = wave % WK, wn = wave / WK % WN * (32 * TN), wm = wave / (WK * WN) * (32 * TM);
  constexpr int kParts = 4 / WK;
  f32x16 acc[TN][TM] = {};
  constexpr int kReads = (kParts + 1) * (TN + TM), kProducts = kParts * TN * TM;
  i32x4 operand[2][kParts][TN + TM];
  uint32_t scale[2][TN + TM];
  // read i of a step: the scales of the channels and of the tokens, then of each part
  // the channels' operands and the tokens'
  auto fetch = [&](int set, int stage, int i) {
    const int part = i / (TN + TM) - 1, q = i % (TN + TM);
    const int first = q < TN ? wn + 32 * q : BN + wm + 32 * (q - TN);
    if (part < 0) {
      const int8_t* at = s_rows[stage] + kCodeBytes + first * kScaleDepth + 4 * lane;
      scale[set][q] = *reinterpret_cast<const uint32_t*>(at) >> (8 * kParts * wk);
      return;
    }
    const int at = (lane & 31) * kDepth + (((wk * kParts + part + 4 * (lane >> 5)) ^ (lane >> 1 & 7)) * 16);
    operand[set][part < 0 ? 0 : part][q] = *reinterpret_cast<const i32x4*>(s_rows[stage] + first * kDepth + at);
  };
  // Waits until this wave's operands have been read and its loads of the next
  // stage have landed; past the barrier both hold for all waves.
  auto arrive = [] {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0), in a form that the compiler counts with
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((STAGES - 2) * kLoads) : "memory");
  };
  auto step = [&](int set, int stage, int k) {
    arrive();
    // this step's products with the next one's reads and a later one's loads in
    // between: in a row, four waves' reads would hold up the issue of the products
    constexpr int kOthers = kReads + kLoads;
#pragma unroll
    for (int m = 0; m < kProducts; ++m) {
      const int part = m / (TN * TM), i = m / TM % TN, j = m % TM;
      acc[i][j] = mfma32(part, operand[set][part][i], scale[set][i], operand[set][part][TN + j], scale[set][TN + j],
                         acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int o = m * kOthers / kProducts; o < (m + 1) * kOthers / kProducts; ++o) {
        if (o < kReads)
          fetch(set ^ 1, (stage + 1) % STAGES, o);
        else
          load(stage, o - kReads, k + STAGES * kDepth);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(STAGES % 2 == 0, "the operand sets alternate with the stages");
  if (begin < end) {
#pragma unroll
    for (int q = 0; q < STAGES - 1; ++q)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load(q, i, begin + q * kDepth);
    arrive();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load(STAGES - 1, i, begin + (STAGES - 1) * kDepth);
#pragma unroll
    for (int i = 0; i < kReads; ++i) fetch(0, 0, i);
    for (int k = begin; k < end;) {
      // the rows of a step past the last are zeros
#pragma unroll
      for (int i = 0; i < STAGES; ++i) {
        step(i & 1, i, k);
        if ((k += kDepth) >= end) break;
      }
    }
    // nothing may be on its way to LDS when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  }
  if constexpr (WK > 1) {
    // the tile's other waves hand their sums to the first; past the barrier every wave
    // is through with the stages
    const int slot = (wave / WK) * (WK - 1) - 1;
    if (wk > 0)
#pragma unroll
      for (int c = 0; c < 16; c += 4)
        s_meet[((slot + wk) * 4 + c / 4) * 64 + lane] = f32x4{acc[0][0][c], acc[0][0][c + 1], acc[0][0][c + 2], acc[0][0][c + 3]};
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int v = 1; v < WK; ++v)
#pragma unroll
      for (int c = 0; c < 16; c += 4) {
        const f32x4 o = s_meet[((slot + v) * 4 + c / 4) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][0][c + e] += o[e];
      }
  }
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) settled(acc[i][j]);
  if constexpr (WK == 1) __syncthreads();  // every wave is through with the stages
  if constexpr (!GROUPED) {
    if (p.splits > 1) {
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int64_t m = t.first + wm + 32 * j + (lane & 31);
        if (m >= t.end) continue;
        float* to = p.sums + (blockIdx.y * p.M + m) * p.sums_pitch;
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const int64_t n = n0 + wn + 32 * i + 2 * c + 4 * (lane >> 5);
            if (n < p.sums_pitch)
              *reinterpret_cast<f32x4*>(to + n) =
                  f32x4{acc[i][j][c], acc[i][j][c + 1], acc[i][j][c + 2], acc[i][j][c + 3]};
          }
      }
      return;
    }
  }
  write_tile<DT, TM, TN, 32 * TN>(p, t.end, n0 + wn, t.first + wm, acc, s_out + wave / WK * (32 * 32 * TN * kB),
                                  [&](int j) {
                                    const int64_t m = t.first + wm + 32 * j + (lane & 31);
                                    return keep_mask<GROUPED>(m < t.end ? source_row<GROUPED>(p, m) : -1);
                                  });
}

// The sums of a product whose K was split, four channels of a token to a thread.
template <int DT>
__global__ __launch_bounds__(256) void mx_join_kernel(Product p) {
  const int64_t fours = p.sums_pitch / 4, all = p.M * fours;
  for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < all; i += gridDim.x * int64_t(256)) {
    const int64_t m = i / fours, n = i % fours * 4;
    f32x4 sum = {};
    for (int v = 0; v < p.splits; ++v)
      sum += *reinterpret_cast<const f32x4*>(p.sums + (v * p.M + m) * p.sums_pitch + n);
    const float f[4] = {sum[0], sum[1], sum[2], sum[3]};
    store_four<DT>(p.y, m * p.N + n, static_cast<int>(min(p.N - n, int64_t(4))), f);
  }
}

// Tiles of 256 x 256.  A last turn of the compute units that is half full at most is
// computed in halves of 128 tokens, by the same launch, and one that is a quarter full
// at most in quarters, by the kernel for smaller tiles.
template <bool GROUPED>
nf4_status launch_tiles(const Product& p, int32_t y_dtype, hipStream_t st) {
  const uint32_t groups = tile_groups<GROUPED>(p, kTile, kTile, kTileThreads);
  const uint32_t turn = (p.cus + kDies - 1) / kDies * kDies;
  if (groups == 0 || (int64_t(groups) + turn) * kTileThreads >= int64_t(1) << 32) return NF4_EUNSUPPORTED;
  // how many tiles experts' rows make only the GPU knows: the workgroups find out
  const int64_t all = row_tiles<GROUPED>(p, kTile) * ((p.N + kTile - 1) / kTile);
  const uint32_t whole = whole_tiles(static_cast<uint32_t>(all), p.cus), rest = static_cast<uint32_t>(all) - whole;
  const bool quarters = GROUPED || (rest > 0 && in_quarters(rest, p.cus));
  const uint32_t halves = GROUPED || (rest > 0 && !quarters) ? turn : 0;
  const uint32_t grid = halves + (GROUPED || whole > 0 ? groups : 0);
  with_dtype(y_dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    if (grid > 0)
      hipLaunchKernelGGL((mx_tile_kernel<DT, GROUPED>), dim3(grid), dim3(kTileThreads), 0, st, p, halves);
    if (quarters)
      hipLaunchKernelGGL((mx_stream_kernel<DT, GROUPED, 2, 2, 1, 2, 2, 4, true>), dim3(turn), dim3(256), 0, st, p);
  });
  return launch_status();
}

template <bool GROUPED, int WM, int WN, int WK, int TM, int TN, int STAGES>
nf4_status launch_stream(const Product& p, int32_t y_dtype, hipStream_t st) {
  constexpr int kThreads = 64 * WM * WN * WK;
  const uint32_t groups = tile_groups<GROUPED>(p, 32 * WM * TM, 32 * WN * TN, kThreads);
  if (groups == 0) return NF4_EUNSUPPORTED;
  with_dtype(y_dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    hipLaunchKernelGGL((mx_stream_kernel<DT, GROUPED, WM, WN, WK, TM, TN, STAGES>),
                       dim3(groups, static_cast<uint32_t>(p.splits)), dim3(kThreads), 0, st, p);
    if (p.splits > 1) {
      const int64_t blocks = (p.M * (p.sums_pitch / 4) + 255) / 256;
      hipLaunchKernelGGL((mx_join_kernel<DT>), dim3(static_cast<uint32_t>(blocks < 4096 ? blocks : 4096)), dim3(256),
                         0, st, p);
    }
  });
  return launch_status();
}

// The tiled kernels, and what their steps of 128 bytes of K take (us): with a tile on
// few compute units, and for each of a compute unit's tiles where all have one or more (the
// memory behind them is busier then).  The figures are fitted to 1 to 2048 rows of
// 4096 x 4096, 11008 x 4096, 4096 x 11008, 2048 x 2048 and 1024 x 11008 in every tiling:
// what they pick is within 5% of the best of these.  Largest tiles load the least per
// product, but leave compute units idle and take the longest for themselves: 512 x
// 4096 x 4096 takes 23.6 / 20.7 / 10.7 / 10.6 / 13.2 / 13.1 us from the smallest tiles to
// the largest, 64 x 4096 x 4096 6.1 / 6.8 / 6.9 / 9.1 / 12.3 / 12.1, 1024 x 11008 x 4096
// - / - / 44 / 49 / 40 / 32.
struct Tiling {
  int BM, BN;         // tokens, channels
  double alone, each; // us a step
  double fixed;       // us a turn that no step hides
};
constexpr Tiling kTilings[] = {{32, 32, 0.086, 0.12, 0.8},  {64, 32, 0.09, 0.158, 1.3},
                               {64, 64, 0.152, 0.21, 0.63}, {128, 64, 0.23, 0.376, 1.2},
                               {128, 128, 0.376, 0.61, 2.2}, {256, 256, 1.49, 1.49, 11.4}};
constexpr int kLargest = 5;
// A last turn of the largest in halves and in quarters.
constexpr double kHalfStep = 1.03, kHalfFixed = 4.5, kQuarterStep = 0.41, kQuarterFixed = 2.3;
constexpr double kLaunchUs = 3.2, kJoinUs = 4.5, kSumUs = 8.0 / 3e6;  // a sum there and back
// Rows sorted by expert: finding a tile, a stream of weights that counts, two launches.
constexpr double kFindUs = 1.3, kLonger = 1.45, kLaunchesUs = 3.4;
constexpr int kMaxSplits = 16;

struct Plan {
  int tiling, splits;
};

// The tiling with the least time by the figures above, with K split over workgroups
// where that leaves compute units without a tile and the workspace has room for the sums,
// unless writing and reading the sums costs as much (17 x 1024 x 11008: 8.3 us in one
// piece, 8.1 in four; 128 x 4096 x 11008 11.8 and 13.7 in two).  The model orders the
// tilings; it is no time of long weights from memory, which it does not know.
//
// Rows sorted by expert: every expert with rows ends in a tile that is half full.  Tiles
// of 64 x 32 and 128 x 64 were the best nowhere (8 to 128 experts with 16 to 8192
// rows), and those of 32 x 32 only where a compute unit has one at most.
template <bool GROUPED>
Plan plan(const Product& p, size_t room) {
  const int64_t cus = device_cus();
  const double steps = static_cast<double>((p.pitch + kDepth - 1) / kDepth);
  Plan best = {0, 1};
  double least = 1e30;
  for (int i = 0; i <= kLargest; ++i) {
    const Tiling& t = kTilings[i];
    double rows = static_cast<double>((p.M + t.BM - 1) / t.BM);
    if (GROUPED)
      rows = p.M >= int64_t(p.experts) * t.BM / 2 ? static_cast<double>(p.M) / t.BM + 0.5 * p.experts
                                                  : static_cast<double>(p.M < p.experts ? p.M : p.experts);
    const double tiles = rows * static_cast<double>((p.N + t.BN - 1) / t.BN);
    if (i < kLargest && tile_groups<GROUPED>(p, t.BM, t.BN, 256) == 0) continue;
    if (GROUPED && (i == 1 || i == 3 || (i == 0 && tiles > cus))) continue;
    const int most = GROUPED || i == kLargest ? 1 : kMaxSplits;
    for (int splits = 1; splits <= most; ++splits) {
      if (splits > 1 && (tiles * splits > cus || p.M * p.sums_pitch * 4 * splits > static_cast<int64_t>(room) ||
                         steps < 4 * splits))
        break;
      const double full = tiles * splits / cus, part = full - std::floor(full);
      double us = kLaunchUs;
      if (i == kLargest) {
        us += std::floor(full) * (t.fixed + steps * t.each) + (GROUPED ? kLaunchesUs : 0.0);
        if (part > 0.5) {  // more of the memory's rate for each
          const double s = 2 * part - 1;
          us += kHalfFixed + (t.fixed - kHalfFixed) * s + steps * (kHalfStep + (t.each - kHalfStep) * s);
        } else if (part > 0.25) {
          us += kHalfFixed + steps * kHalfStep;
        } else if (part > 0) {
          us += kQuarterFixed + steps * kQuarterStep;
        }
      } else {
        const double turns = std::ceil(full), step = full > 1 ? turns * t.each : t.alone + (t.each - t.alone) * full;
        us += turns * (t.fixed + (GROUPED ? kFindUs : 0.0)) +
              std::ceil(steps / splits) * step * (GROUPED ? kLonger : 1.0);
      }
      if (splits > 1) us += kJoinUs + p.M * p.sums_pitch * splits * kSumUs;
      if (us < least * (splits > 1 ? 0.85 : 1.0)) {
        least = us;
        best = {i, splits};
      }
    }
  }
  return best;
}

Product dense(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws, void* y, int64_t M,
              int64_t N, int64_t K) {
  Product p = {};
  p.xq = xq, p.xs = xs, p.wq = wq, p.ws = ws, p.y = y;
  p.M = M, p.N = N, p.pitch = pitch_of(K), p.steps = steps_of(K), p.x_rows = M;
  p.top_k = p.experts = p.splits = 1;
  p.sums_pitch = (N + 3) / 4 * 4;
  p.cus = static_cast<uint32_t>(device_cus());
  return p;
}

// Whether the row kernel takes the product: it reads weights once for every 16 rows.
// Its start is shorter than a tile's, so it does better where every compute unit has one
// tile of 16 x 16 at most and rows are not long (1 x 1024 x 4096: 4.0 us and 5.3 in tiles,
// 4 x 4096 x 4096 5.6 and 5.8, 32 x 2048 x 2048 4.5 and 4.7; 4 x 4096 x 11008 9.4 and 8.4,
// 4 x 11008 x 4096 7.7 and 7.0).  By expert: where the weights' stream counts and a tile
// of 64 x 64 has few steps (64 experts of 1024 x 2048 with 64 to 512 rows: 12.9-17.2 us and
// 14.9-17.8; of 2048 x 1024 with 1024 rows 22.5 and 24.6; with 16 rows of 1024 x 2048 8.4
// and 7.5, 16 experts of 2048 x 4096 with 64 rows 15.5 and 14.8).
constexpr int64_t kShortPitch = 2048, kShortestPitch = 512;

template <bool GROUPED>
bool few(const Product& p) {
  if (!fits_rows(p)) return false;
  const int64_t cus = device_cus();
  if (GROUPED) {
    const int64_t most = p.M < p.experts ? p.M : p.experts;
    return p.pitch <= kShortPitch / 2 && most * ((p.N + 15) / 16) > 8 * cus &&
           p.M <= (p.pitch <= kShortestPitch ? 16 : 8) * int64_t(p.experts);
  }
  return p.pitch <= kShortPitch && row_tiles<false>(p, 16) * ((p.N + 15) / 16) <= cus;
}

// Whether it takes the activations as they are and encodes them too, which each of its
// workgroups does again: up to 32768 elements (16 rows at a time) where every compute unit
// has one tile, 16384 where it has more.  One launch and two: 8 x 4096 x 4096 6.8 us and
// 8.1, 16 rows 9.7 and 8.3; 4 x 11008 x 4096 8.8 and 9.5, 8 rows 11.0 and 9.5; 2 x 4096 x
// 11008 10.1 and 10.9, 4 rows 12.3 and 10.9; 1 x 44032 x 4096 18.5 and 21.5.
bool encodes_rows(const Product& p) {
  if (!fits_rows(p)) return false;
  const int64_t elements = (p.M < 16 ? p.M : 16) * 2 * p.pitch;
  const bool one = row_tiles<false>(p, 16) * ((p.N + 15) / 16) <= device_cus();
  return elements <= (one ? 32768 : 16384) && (p.M <= 16 || one);
}

// What a product goes to: the few-row kernel, or tiles as planned.
constexpr int kToRows = -1;

template <bool GROUPED>
Plan choose(const Product& p, size_t room) {
  if (few<GROUPED>(p)) return {kToRows, 1};
  return plan<GROUPED>(p, room);
}

template <bool GROUPED>
nf4_status launch(Product p, int32_t y_dtype, void* workspace, size_t room, hipStream_t st) {
  const Plan plan_ = choose<GROUPED>(p, workspace ? room : 0);
  if (plan_.tiling == kToRows) return launch_rows(p, GROUPED, nullptr, kCodes, 0, y_dtype, st);
  p.splits = plan_.splits;
  p.sums = static_cast<float*>(workspace);
  switch (plan_.tiling) {
    case 0: return launch_stream<GROUPED, 1, 1, 4, 1, 1, 8>(p, y_dtype, st);
    case 1:
      if constexpr (!GROUPED) return launch_stream<false, 2, 1, 2, 1, 1, 8>(p, y_dtype, st);
      return NF4_EUNSUPPORTED;
    case 2: return launch_stream<GROUPED, 2, 2, 1, 1, 1, 4>(p, y_dtype, st);
    case 3:
      if constexpr (!GROUPED) return launch_stream<false, 2, 2, 1, 2, 1, 4>(p, y_dtype, st);
      return NF4_EUNSUPPORTED;
    case 4: return launch_stream<GROUPED, 2, 2, 1, 2, 2, 4>(p, y_dtype, st);
    default: return launch_tiles<GROUPED>(p, y_dtype, st);
  }
}

// What the products check alike (the activations apart).
nf4_status check_product(const uint8_t* wq, const uint8_t* ws, int64_t N, int64_t K, const void* y,
                         int32_t y_dtype) {
  if (!y || (K > 0 && (!wq || !ws))) return NF4_EINVAL;
  if (!aligned(wq, 16) || !aligned(ws, 16) || !aligned(y, dtype_bytes(y_dtype))) return NF4_EINVAL;
  if (N > kMaxDim || K > kMaxK) return NF4_EUNSUPPORTED;
  return NF4_OK;
}

size_t rounded(int64_t bytes) { return static_cast<size_t>(bytes + 255) / 256 * 256; }
size_t codes_bytes(int64_t M, int64_t K) { return rounded(M * pitch_of(K)); }
size_t scales_bytes(int64_t M, int64_t K) { return rounded(scale_bytes(M, K)); }

}  // namespace

extern "C" {

nf4_status nf4_probe_mxfp4_plan(int64_t M, int64_t N, int64_t K, int32_t experts, size_t room, int32_t* plan,
                                int32_t* detail) {
  if (!plan || !detail || M < 1 || N < 1 || K < 0 || experts < -1) return NF4_EINVAL;
  if (M > kMaxDim || N > kMaxDim || K > kMaxK || experts > kMaxExperts) return NF4_EUNSUPPORTED;
  Product p = dense(nullptr, nullptr, nullptr, nullptr, nullptr, M, N, K);
  if (experts > 0) p.experts = experts;
  const Plan best = experts < 0 && encodes_rows(p) ? Plan{kToRows, 1}
                    : experts > 0                  ? choose<true>(p, 0)
                                                   : choose<false>(p, room);
  *plan = best.tiling;
  if (best.tiling == kToRows) {
    const Rows r = row_plan(p, experts > 0 ? row_tiles<true>(p, 16) : row_tiles<false>(p, 16));
    *detail = r.split == kRowWaves ? r.units : -r.split;
  } else if (best.tiling < kLargest || experts > 0) {
    *detail = best.splits;
  } else {
    const uint32_t all = static_cast<uint32_t>(row_tiles<false>(p, kTile) * ((N + kTile - 1) / kTile));
    const uint32_t whole = whole_tiles(all, p.cus), rest = all - whole;
    *detail = (whole > 0 ? 1 : 0) + (rest == 0 ? 0 : in_quarters(rest, p.cus) ? 4 : 2);
  }
  return NF4_OK;
}

size_t mxfp4_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxK) return 0;
  const Product p = dense(nullptr, nullptr, nullptr, nullptr, nullptr, M, N, K);
  const Plan best = choose<false>(p, static_cast<size_t>(1) << 62);
  return best.splits > 1 ? static_cast<size_t>(M * p.sums_pitch * 4 * best.splits) : 0;
}

nf4_status mxfp4_gemm(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws,
                      int64_t M, int64_t N, int64_t K, void* y, int32_t y_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || !known_dtype(y_dtype) || !aligned(workspace, 256))
    return NF4_EINVAL;
  if (M == 0 || N == 0) return NF4_OK;
  if ((K > 0 && (!xq || !xs)) || !aligned(xq, 16) || !aligned(xs, 16)) return NF4_EINVAL;
  if (const nf4_status st = check_product(wq, ws, N, K, y, y_dtype)) return st;
  if (M > kMaxDim) return NF4_EUNSUPPORTED;
  return launch<false>(dense(xq, xs, wq, ws, y, M, N, K), y_dtype, workspace, workspace_bytes,
                       reinterpret_cast<hipStream_t>(stream));
}

size_t mxfp4_linear_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxK) return 0;
  if (encodes_rows(dense(nullptr, nullptr, nullptr, nullptr, nullptr, M, N, K))) return 0;
  return codes_bytes(M, K) + scales_bytes(M, K) + mxfp4_gemm_workspace_size(M, N, K);
}

nf4_status mxfp4_linear(const void* x, int32_t x_dtype, const uint8_t* wq, const uint8_t* ws,
                        int64_t M, int64_t N, int64_t K, void* y, int32_t y_dtype, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || !known_dtype(x_dtype) || !known_dtype(y_dtype) ||
      !aligned(workspace, 256))
    return NF4_EINVAL;
  if (M == 0 || N == 0) return NF4_OK;
  if ((K > 0 && !x) || !aligned(x, dtype_bytes(x_dtype))) return NF4_EINVAL;
  if (const nf4_status st = check_product(wq, ws, N, K, y, y_dtype)) return st;
  if (M > kMaxDim) return NF4_EUNSUPPORTED;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  Product p = dense(nullptr, nullptr, wq, ws, y, M, N, K);
  if (encodes_rows(p)) return launch_rows(p, false, x, x_dtype, K, y_dtype, st);
  if (K == 0) return launch<false>(p, y_dtype, nullptr, 0, st);
  // the codes and scales have to have room; the rest is for the sums of a split
  const size_t used = codes_bytes(M, K) + scales_bytes(M, K);
  if (!workspace || workspace_bytes < used) return NF4_EINVAL;
  uint8_t* xq = static_cast<uint8_t*>(workspace);
  uint8_t* xs = xq + codes_bytes(M, K);
  if ((K + 127) / 128 > kMaxDim / M) return NF4_EUNSUPPORTED;
  quantize_launch(x, x_dtype, M, K, xq, xs, st);
  return launch<false>(dense(xq, xs, wq, ws, y, M, N, K), y_dtype, xq + used, workspace_bytes - used, st);
}

nf4_status mxfp4_gemm_grouped(const uint8_t* xq, const uint8_t* xs, int64_t x_rows,
                              const int32_t* order, int32_t top_k, const uint8_t* wq,
                              const uint8_t* ws, const int32_t* offsets, int32_t experts,
                              int64_t rows, int64_t N, int64_t K, void* y, int32_t y_dtype,
                              void* stream) {
  if (x_rows < 0 || rows < 0 || N < 0 || K < 0 || experts < 0 || (order && top_k < 1) ||
      !known_dtype(y_dtype))
    return NF4_EINVAL;
  if (experts == 0 || rows == 0 || N == 0) return NF4_OK;
  if (!offsets || !aligned(offsets, 4) || !aligned(order, 4)) return NF4_EINVAL;
  if (x_rows > 0 && K > 0 && (!xs || !xq)) return NF4_EINVAL;
  if (!aligned(xq, 16) || !aligned(xs, 16)) return NF4_EINVAL;
  if (const nf4_status st = check_product(wq, ws, N, K, y, y_dtype)) return st;
  if (experts > kMaxExperts || rows > kMaxDim || x_rows > kMaxDim || experts * N > kMaxDim) return NF4_EUNSUPPORTED;
  Product p = dense(xq, xs, wq, ws, y, rows, N, K);
  p.order = order, p.offsets = offsets, p.x_rows = x_rows;
  p.top_k = order ? top_k : 1, p.experts = experts;
  return launch<true>(p, y_dtype, nullptr, 0, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
