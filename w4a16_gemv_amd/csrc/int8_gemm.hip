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

#include <cmath>

#include "int8.h"
#include "int8_product.h"
#include "nf4_device.h"
#include "nf4_probe.h"
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
  // K split over `splits` workgroups of a tile: int32 sums to planes of
  // M x sums_pitch at `sums` instead of y (dense only)
  int32_t* sums;
  int64_t sums_pitch;
  int splits;
  uint32_t cus;  // compute units
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

// The token of a row of y: its scale, and the mask of its outputs' bits, 0 where there
// is none.  The zero scale alone would leave the NaN of a channel whose scale is NaN or
// infinite.  (A mask, since selecting the value takes the few-row kernel 5% longer: 64
// x 2 tokens over 64 experts of 512 x 4096 22.7 us against 21.5.)
struct RowToken {
  float scale;
  uint32_t keep;
};
template <bool GROUPED>
__device__ __forceinline__ uint32_t keep_mask(int64_t src) {
  return !GROUPED || src >= 0 ? ~0u : 0u;
}
__device__ __forceinline__ float masked(float v, uint32_t keep) {
  return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & keep);
}

// The hardware deals workgroups out to the eight dies in turn; each die gets a
// range of its own of the `count` tiles.  False past the last.
constexpr uint32_t kDies = 8;

__device__ __forceinline__ bool tile_of_group(uint32_t b, uint32_t count, uint32_t& i) {
  const uint32_t each = (count + kDies - 1) / kDies, at = b / kDies;
  i = b % kDies * each + at;
  return at < each && i < count;
}

// Tiles in an order whose neighbours share rows and channels: bands of kBand row
// tiles.
constexpr uint32_t kBand = 8;

__device__ __forceinline__ void locate_tile(uint32_t i, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm,
                                            uint32_t& tn) {
  const uint32_t band = i / (kBand * tiles_n), in = i % (kBand * tiles_n);
  const uint32_t high = min(uint32_t(kBand), tiles_m - band * kBand);
  // the divisions run on the vector unit: back to scalars, so that what follows
  // from them (buffer resources among it) is one value per wave
  tm = __builtin_amdgcn_readfirstlane(band * kBand + in % high);
  tn = __builtin_amdgcn_readfirstlane(in / high);
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

// Scales a wave's 32 TM tokens from m0 on x 32 TN channels from n0 on and writes
// them, 32 tokens x CHANNELS at a time through an LDS region of its own, so that
// whole lines of y are written.  Channel(c) gives the scales of channels n0 + c ..
// n0 + c + 3 (0 past the end), token(j) the lane's token of tile j.
template <int DT, int TM, int TN, int CHANNELS, class Channel, class Token>
__device__ __forceinline__ void write_tile(const Product& p, int64_t end, int64_t n0, int64_t m0,
                                           const i32x16 (&acc)[TN][TM], int8_t* lds, Channel&& channel,
                                           Token&& token) {
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
    float4 ws[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) ws[i][c] = channel(32 * (i0 + i) + 8 * c + 4 * (lane >> 5));
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t m1 = m0 + 32 * j;
      const RowToken x = token(j);
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const i32x16& v = acc[i0 + i][j];
          const float f[4] = {static_cast<float>(v[4 * c]) * x.scale * ws[i][c].x,
                              static_cast<float>(v[4 * c + 1]) * x.scale * ws[i][c].y,
                              static_cast<float>(v[4 * c + 2]) * x.scale * ws[i][c].z,
                              static_cast<float>(v[4 * c + 3]) * x.scale * ws[i][c].w};
          const int at = (32 * i + 8 * c + 4 * (lane >> 5)) * kB;
          int8_t* to = lds + (lane & 31) * kRow + (((at >> 4) ^ swap(lane & 31)) << 4) + (at & 15);
          if constexpr (DT == INT8_FP32)
            *reinterpret_cast<float4*>(to) = make_float4(masked(f[0], x.keep), masked(f[1], x.keep),
                                                         masked(f[2], x.keep), masked(f[3], x.keep));
          else
            *reinterpret_cast<uint2*>(to) =
                make_uint2(pack_pair<DT>(f[0], f[1]) & x.keep, pack_pair<DT>(f[2], f[3]) & x.keep);
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
// x 128 outputs in int32 accumulators, which takes all of a compute unit's
// registers and LDS.
//
// Bound by the matrix pipe, the clock and the LDS together, none of them alone: 8192 x
// 8192 x 8192 takes 430 us (2560 TOP/s), a step of 64 matrix instructions a wave about
// 1.45 us where they alone take 1.08 (the clock sinks under them; on zeros the same
// program takes 1.25), with the LDS reads 1.30.  8192 x 11008 x 4096 takes 322-344 us,
// a seventh of it for the outputs' scaling and stores, with matrix instructions in 68%
// of a tile's cycles (by expert 54%).  Measured and not kept: one workgroup for several
// tiles, the next one's first loads before the stores (273 us against 246 at 8192 x
// 8192 x 4096: the loads' waits take in the stores), registers between memory and LDS
// (the same time), all of a step's loads at its barrier (6% slower).
//
// 128 bytes of K at a time (a step): the tile's rows go from memory straight to
// one of two LDS buffers, and from there to the matrix cores, 32 bytes of K at a
// time (a part) with the next 32 being read.  One barrier per step: it stands
// before the last part, whose operands are in registers by then, so that the
// other buffer's first operands are read while the matrix cores still work.  The
// order of the instructions is given by hand (sched_group_barrier): left alone
// the compiler reads operands right before their use.
//
// LDS: two rows of eight 16-byte chunks fill the 64 banks; chunk c of row r is
// stored at c ^ (r / 2 % 8), so that the sixteen lanes that are served at a
// time, 16 rows of one chunk (reads) or two whole rows (writes), lie in all
// banks once.
//
// Rows past the tile's end are zeros or whatever row is at hand (their outputs
// are not stored); bytes past a row's pitch are zeros on the weights' side.  The
// steps past the last are loaded too: zeros that nothing uses.
//
// Out: 32 tokens at a time through LDS, so that whole lines of y are written.  The
// scales are asked for at the start: at the end each would be a wait of its own.
// ---------------------------------------------------------------------------
constexpr int kTile = 256;
constexpr int kTileThreads = 256;
constexpr int kDepth = 128;  // bytes of K per step
// Offset of a load that is to give zeros: past every range, whatever row offset
// is added.  (Row offsets go into the vector offset too: the range is checked
// against that alone once a scalar offset passes it.)
constexpr uint32_t kNever = 0x80000000u;

// What sched_group_barrier names.
constexpr int kSchedMfma = 0x8, kSchedLoad = 0x20, kSchedRead = 0x100;

typedef __attribute__((address_space(3))) void* LdsPtr;
__device__ __forceinline__ uint32_t lds_address(void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((LdsPtr)p));
}
// The four words of rsrc(p, bytes), one value per wave.
__device__ __forceinline__ i32x4 range_words(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uintptr_t>(p);
  return i32x4{__builtin_amdgcn_readfirstlane(static_cast<int>(a)),
               __builtin_amdgcn_readfirstlane(static_cast<int>(a >> 32 & 0xFFFF)),
               __builtin_amdgcn_readfirstlane(static_cast<int>(p ? bytes : 0)), 0x00020000};
}
typedef const __attribute__((address_space(1))) void* GlobalPtr;

// How many of `all` tiles are computed whole where the rest, half a turn of the
// compute units at most, is computed in pieces.
__device__ __host__ __forceinline__ uint32_t whole_tiles(uint32_t all, uint32_t cus) {
  const uint32_t rest = all % cus;
  return 2 * rest <= cus ? all - rest : all;
}

// Whether that rest is computed in quarters of 128 x 128 (stream_kernel): where the
// compute units hold them in one turn.
__device__ __host__ __forceinline__ bool in_quarters(uint32_t rest, uint32_t cus) { return 4 * rest <= cus; }

// Which tiles of 256 x 256 a launch computes: those that whole_tiles() counts, or
// the others, in halves of 128 tokens or in quarters.
enum Share { kWhole, kHalves, kQuarters };

template <int DT, bool GROUPED, Share SHARE>
__global__ __launch_bounds__(kTileThreads, 1) void tile_kernel(Product p) {
  constexpr int TN = kTile / 64, TM = SHARE == kHalves ? TN / 2 : TN;  // 32 x 32 tiles of a wave
  constexpr int BM = 64 * TM;                      // tokens
  constexpr int LN = kTile / 32, LM = BM / 32;     // 16-byte loads of a thread per step
  constexpr int kB = dtype_bytes(DT);
  // two buffers that the compiler can tell apart: reads of one do not wait for
  // the loads into the other
  __shared__ __attribute__((aligned(256))) int8_t s_a[(kTile + BM) * kDepth], s_b[(kTile + BM) * kDepth];
  __shared__ __attribute__((aligned(256))) int8_t s_out[4 * 32 * 128];
  __shared__ __attribute__((aligned(256))) float s_scale[2][kTile];  // of the channels, of the tokens
  __shared__ uint32_t s_keep[GROUPED ? kTile : 1];                    // the tokens' masks

  const uint32_t tiles_n = static_cast<uint32_t>((p.N + kTile - 1) / kTile);
  uint32_t tiles_m = static_cast<uint32_t>((p.M + kTile - 1) / kTile);
  if constexpr (GROUPED) tiles_m = count_tiles<kTile>(p);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int row = 8 * wave + (lane >> 3);
  const int chunk = ((lane & 7) ^ (row >> 1 & 7)) * 16;
  const int pitch = static_cast<int>(p.pitch);
  const uint32_t voff = static_cast<uint32_t>(row * pitch + chunk);

  uint32_t index, half = 0, tm, tn;
  const uint32_t all = tiles_m * tiles_n, whole = whole_tiles(all, p.cus);
  if constexpr (SHARE == kHalves) {
    if (in_quarters(all - whole, p.cus) || !tile_of_group(blockIdx.x, 2 * (all - whole), index)) return;
    half = index & 1;
    index = whole + index / 2;
  } else {
    if (!tile_of_group(blockIdx.x, whole, index)) return;
  }
  locate_tile(index, tiles_m, tiles_n, tm, tn);
  RowTile t = {static_cast<int64_t>(tm) * kTile, min(p.M, static_cast<int64_t>(tm) * kTile + kTile), 0};
  if constexpr (GROUPED) t = find_tile<kTile>(p, tm);
  if constexpr (SHARE == kHalves) {
    t.first += half * BM;
    t.end = min(t.end, t.first + BM);
    if (t.end <= t.first) return;
  }
  const int64_t n0 = static_cast<int64_t>(tn) * kTile;
  const int8_t* w0 = p.wq + (t.expert * p.N + n0) * p.pitch;
  const auto rw = rsrc(w0, static_cast<uint32_t>(min(int64_t(kTile), p.N - n0) * p.pitch));
  const auto rx = rsrc(GROUPED ? nullptr : p.xq + t.first * p.pitch,
                       static_cast<uint32_t>((t.end - t.first) * p.pitch));
  const int8_t* xrow[GROUPED ? LM : 1];
  if constexpr (GROUPED) {
#pragma unroll
    for (int i = 0; i < LM; ++i) {
      const int64_t m = t.first + row + 32 * i;
      const int64_t src = m < t.end ? source_row<true>(p, m) : -1;
      xrow[i] = src >= 0 ? p.xq + src * p.pitch : w0;  // any row that may be read
    }
  }

  // --- memory to LDS: a wave fills eight rows at a time, the channels' first
  auto load = [&](int8_t* buf, int i, int k) {
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
  auto fetch = [&](int set, const int8_t* buf, int part) {
    const int at = (lane & 31) * kDepth + (((2 * part + (lane >> 5)) ^ (lane >> 1 & 7)) * 16);
#pragma unroll
    for (int i = 0; i < TN; ++i)
      fw[set][i] = *reinterpret_cast<const i32x4*>(buf + (wn + 32 * i) * kDepth + at);
#pragma unroll
    for (int i = 0; i < TM; ++i)
      fx[set][i] = *reinterpret_cast<const i32x4*>(buf + (kTile + wm + 32 * i) * kDepth + at);
  };
  i32x16 acc[TN][TM] = {};
  auto multiply = [&](int set) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[set][i], fx[set][j], acc[i][j], 0, 0, 0);
  };
  // The step after the next one's loads may start when the barrier has freed its
  // buffer: they are spread over the parts 3, 0 and 1, one to two or more matrix
  // instructions, since four waves' loads in a row would hold up the issue.
  constexpr int kMoves = LN + LM, kThree = (kMoves + 2) / 3, kZero = (kMoves - kThree + 1) / 2;
  constexpr int kOne = kMoves - kThree - kZero;
  auto order = [&](int loads) {
#pragma unroll
    for (int i = 0; i < TN + TM; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      if (i < loads) __builtin_amdgcn_sched_group_barrier(kSchedLoad, 1, 0);
      if (i < TN * TM - TN - TM) __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // one step: `now` holds this step's rows, `next` the next one's
  auto step = [&](int8_t* now, int8_t* next, int k) {
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
      multiply(part & 1);
      order(part == 0 ? kZero : part == 1 ? kOne : 0);
    }
    __syncthreads();
    fetch(0, next, 0);
#pragma unroll
    for (int i = 0; i < kThree; ++i) load(now, i, (k + 2) * kDepth);
    multiply(1);
    order(kThree);
  };

  const int steps = (pitch + kDepth - 1) / kDepth;
#pragma unroll
  for (int i = 0; i < kMoves; ++i) load(s_a, i, 0);
#pragma unroll
  for (int i = 0; i < kThree; ++i) load(s_b, i, kDepth);
  // the scales of channel and token threadIdx.x, for the end
  const int64_t n = n0 + threadIdx.x, m = t.first + threadIdx.x;
  const float wscale = n < p.N ? p.ws[t.expert * p.N + n] : 0.0f;
  const int64_t src = m < t.end ? source_row<GROUPED>(p, m) : -1;
  const float xscale = src >= 0 ? p.xs[src] : 0.0f;  // (BM < 256: of tokens past the tile too, unused)
  __syncthreads();
  fetch(0, s_a, 0);
  for (int k = 0; k < steps; k += 2) {  // with an odd number the last step is one of zeros
    step(s_a, s_b, k);
    step(s_b, s_a, k + 1);
  }
  s_scale[0][threadIdx.x] = wscale;
  s_scale[1][threadIdx.x] = xscale;
  if constexpr (GROUPED) s_keep[threadIdx.x] = keep_mask<true>(src);
  __syncthreads();
  write_tile<DT, TM, TN, 128 / kB>(
      p, t.end, n0 + wn, t.first + wm, acc, s_out + wave * 32 * 128,
      [&](int c) { return *reinterpret_cast<const float4*>(&s_scale[0][wn + c]); },
      [&](int j) {
        const int at = wm + 32 * j + (lane & 31);
        return RowToken{s_scale[1][at], GROUPED ? s_keep[GROUPED ? at : 0] : ~0u};
      });
}

template <int DT>
__device__ __forceinline__ void store_four(void* y, int64_t i, int left, const float (&f)[4]) {
  if (left >= 4) {
    if constexpr (DT == INT8_FP32) {
      const u32x4 v = {__builtin_bit_cast(uint32_t, f[0]), __builtin_bit_cast(uint32_t, f[1]),
                       __builtin_bit_cast(uint32_t, f[2]), __builtin_bit_cast(uint32_t, f[3])};
      *reinterpret_cast<u32x4_a4*>(static_cast<float*>(y) + i) = v;
    } else {
      const u32x2 v = {pack_pair<DT>(f[0], f[1]), pack_pair<DT>(f[2], f[3])};
      *reinterpret_cast<u32x2_a2*>(static_cast<uint16_t*>(y) + i) = v;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < left) store_one<DT>(y, i + e, f[e]);
}

// ---------------------------------------------------------------------------
// Single tokens: one or two.  No matrix instructions: a wave takes whole rows of
// weights, two at a time, 1024 contiguous bytes to a load, and multiplies them
// by the tokens' codes, which its workgroup keeps in LDS, with v_dot4_i32_i8;
// the lanes' sums are added at a row's end.  The weights of the next two rows
// are asked for as soon as the registers are free.  Bound by the weights' stream and
// a start of about 2 us: quantization included, 1 x 4096 x 4096 takes 6.6 us and 1 x
// 11008 x 4096 11.1 (a plain read of those weights 4.6 and 8.8), two launches 8.9 and
// 14.0.
//
// XT is the tokens' type.  Codes (kCodes) are copied to LDS; tokens of other
// types are quantized on the way there, after the workgroup's first weights have
// been asked for.
// ---------------------------------------------------------------------------
constexpr int kDotWaves = 8;
constexpr int kDotThreads = 64 * kDotWaves;
constexpr int kDotRows = 2 * kDotWaves;  // of weights, of a workgroup at a time
constexpr int kCodes = 3;

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}

// The sum over the 64 lanes, in all of them.
__device__ __forceinline__ int wave_total(int v) {
  v += dpp<0xB1>(v);   // the neighbour (quad permutation 1 0 3 2)
  v += dpp<0x4E>(v);   // the other pair of the four (2 3 0 1)
  v += dpp<0x141>(v);  // the other four of the eight (half mirror)
  v += dpp<0x140>(v);  // the other eight of the sixteen (mirror)
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = a[0] + a[1];
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return b[0] + b[1];
}

// BLOCKS: 1024-byte blocks of a row, most; MT: tokens, most.
template <int XT, int DT, int MT, int BLOCKS>
__global__ __launch_bounds__(kDotThreads, 4) void dot_kernel(Product p, const void* x, int K) {
  constexpr int kLds = BLOCKS * 1024;  // of a token's codes
  __shared__ __attribute__((aligned(16))) int8_t s_x[MT * kLds];
  __shared__ uint32_t s_peak[kDotWaves][MT];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int pitch = static_cast<int>(p.pitch), M = static_cast<int>(p.M);
  const int blocks = (pitch + 1023) / 1024;
  const uint32_t tiles = static_cast<uint32_t>((p.N + kDotRows - 1) / kDotRows);
  i32x4 w[2][BLOCKS];
  auto range = [&](uint32_t tile) {
    const int64_t n0 = static_cast<int64_t>(tile) * kDotRows;
    const int64_t rows = tile < tiles ? min(int64_t(kDotRows), p.N - n0) : 0;  // no rows: zeros
    return rsrc(p.wq + n0 * p.pitch, static_cast<uint32_t>(rows * p.pitch));
  };
  const uint32_t row0 = static_cast<uint32_t>(2 * wave * pitch + 16 * lane);
  auto load = [&](__amdgpu_buffer_rsrc_t rw, int b) {
    // a row's last block ends in the next row, against zeros in LDS
    const uint32_t at = b < blocks ? row0 + 1024 * b : kNever;
#pragma unroll
    for (int r = 0; r < 2; ++r)
      w[r][b] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, at + r * pitch, 0, 0));
  };
  const auto first = range(blockIdx.x);
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) load(first, b);

  float xs[MT];
  if constexpr (XT == kCodes) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m >= M) continue;
      xs[m] = p.xs[m];
      for (int at = 16 * threadIdx.x; at < 1024 * blocks; at += 16 * kDotThreads) {
        i32x4 v = {};
        if (at < pitch) v = *reinterpret_cast<const i32x4*>(p.xq + m * p.pitch + at);
        // bytes past K may hold anything where the weights' are zero, but those
        // past the pitch meet the next row's weights
        *reinterpret_cast<i32x4*>(s_x + m * kLds + at) = v;
      }
    }
  } else {
    constexpr int kPieces = (BLOCKS * 128 + kDotThreads - 1) / kDotThreads;  // of a thread, to a row
    auto row = [&](int m) { return static_cast<const char*>(x) + static_cast<int64_t>(m) * K * dtype_bytes(XT); };
    uint32_t peak[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      peak[m] = 0;
      if (m >= M) continue;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = 8 * (threadIdx.x + i * kDotThreads);
        if (at < K) peak[m] = max(peak[m], piece_peak<XT>(load_piece<XT>(row(m), at, K)));
      }
      peak[m] = wave_max(peak[m]);
      if (lane == 0) s_peak[wave][m] = peak[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m >= M) continue;
#pragma unroll
      for (int v = 0; v < kDotWaves; ++v) peak[m] = max(peak[m], s_peak[v][m]);
      const RowScale scale = row_scale(peak[m]);
      xs[m] = scale.scale;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = 8 * (threadIdx.x + i * kDotThreads);
        if (at < 1024 * blocks)
          *reinterpret_cast<uint2*>(s_x + m * kLds + at) =
              at < K ? encode_piece<XT>(load_piece<XT>(row(m), at, K), scale) : make_uint2(0u, 0u);
      }
    }
  }
  __syncthreads();

  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    int acc[2][MT] = {};
    // few codes may stay in registers from tile to tile; more would spill
    if constexpr (MT * BLOCKS > 8) asm volatile("" ::: "memory");
    const auto next = range(tile + gridDim.x);
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
      // blocks past the row: zeros against whatever LDS holds
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const i32x4 c = *reinterpret_cast<const i32x4*>(s_x + m * kLds + 1024 * b + 16 * lane);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][m] = __builtin_amdgcn_sdot4(w[r][b][e], c[e], acc[r][m], false);
      }
      // the products first, then the load into the registers that they free: the
      // other way round the compiler takes twice the registers
#pragma unroll
      for (int m = 0; m < MT; ++m) asm volatile("" : "+v"(acc[0][m]), "+v"(acc[1][m]));
      __builtin_amdgcn_sched_barrier(0);
      load(next, b);
    }
    const int64_t n = static_cast<int64_t>(tile) * kDotRows + 2 * wave;
    const float ws0 = n < p.N ? p.ws[n] : 0.0f, ws1 = n + 1 < p.N ? p.ws[n + 1] : 0.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float f0 = static_cast<float>(wave_total(acc[0][m])) * xs[m] * ws0;
      const float f1 = static_cast<float>(wave_total(acc[1][m])) * xs[m] * ws1;
      if (m < M && lane < 2 && n + lane < p.N) store_one<DT>(p.y, m * p.N + n + lane, lane ? f1 : f0);
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows: up to 16 tokens.  The eight waves of a workgroup share K, and each
// holds the codes of its share, of all the tokens, in registers while the
// workgroup goes through its channels, 16 at a time: the weights go from memory
// through registers to the matrix cores (v_mfma_i32_16x16x64_i8: lane i + 16 g
// holds A[i][16 g .. + 15], B likewise with i the column, and D[4 g .. + 3][i]),
// each byte read once, a whole tile of them in flight while the one before is
// used.  The waves' int32 sums meet in LDS.  More rows than 16 go to more workgroups.
//
// Bound by the weights' stream: 13 x 11008 x 4096 takes 11.6 us (45 MB, a plain
// read of which takes 8.8), or 13.0 with each lane loading what it multiplies,
// where four lanes read four rows; 16 tokens' 41 of 64 experts of 1024 x 2048 take 25
// from memory (86 MB).  Measured and not kept: two tiles of weights in flight (the
// same times), the experts' tiles in equal shares over the workgroups (22 us for those
// 41, but 37 against 28 for eight of 4096 x 4096: the turns between experts), three
// to eight workgroups a compute unit (up to a third slower).  The one- and two-token kernel at more tokens
// is slower from four on (12.0 against 11.1 us at 4 x 11008 x 4096).
// ---------------------------------------------------------------------------
constexpr int kRowWaves = 8;
constexpr int kRowThreads = 64 * kRowWaves;

template <int DT, bool GROUPED, int UNITS>
__global__ __launch_bounds__(kRowThreads, UNITS > 8 ? 2 : 4) void row_kernel(Product p) {
  __shared__ i32x4 s_sum[2][kRowWaves][64];
  const uint32_t tiles = static_cast<uint32_t>((p.N + 15) / 16);
  RowTile t = {int64_t(16) * blockIdx.y, min(p.M, int64_t(16) * blockIdx.y + 16), 0};
  if constexpr (GROUPED) t = find_tile<16>(p, blockIdx.y);
  if (t.end <= t.first) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int pitch = static_cast<int>(p.pitch);
  // a unit as it is loaded: lane 4 i + g has 16 bytes g of row i, so that four lanes
  // read 64 bytes in a row; turned() hands them to lane i + 16 g
  const int row = lane >> 2, inside = (lane & 3) * 16;
  auto turned = [&](const i32x4& v) {
    const int from = 4 * (4 * (lane & 15) + (lane >> 4));  // a lane's number times 4
    i32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = __builtin_amdgcn_ds_bpermute(from, v[e]);
    return r;
  };
  // the wave's units of 64 bytes: pairs, so that two loads read whole lines
  const int units = pitch / 64;
  auto unit = [&](int u) { return 2 * wave + 2 * kRowWaves * (u >> 1) + (u & 1); };
  const uint32_t voff = static_cast<uint32_t>(row * pitch + inside);
  const int8_t* w0 = p.wq + t.expert * p.N * p.pitch;
  i32x4 w[UNITS];
  auto load = [&](uint32_t tile) {
    const int64_t n0 = static_cast<int64_t>(tile) * 16;
    const auto rw = rsrc(w0 + n0 * p.pitch, static_cast<uint32_t>(min(int64_t(16), p.N - n0) * p.pitch));
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
      w[u] = __builtin_bit_cast(
          i32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, unit(u) < units ? voff + 64 * unit(u) : kNever, 0, 0));
  };
  load(blockIdx.x);

  const int64_t m = t.first + (lane & 15);
  const int64_t src = source_row<GROUPED>(p, min(m, t.end - 1));
  const float xs = src >= 0 ? p.xs[src] : 0.0f;
  const uint32_t keep = keep_mask<GROUPED>(src);
  const int64_t from = source_row<GROUPED>(p, min(t.first + row, t.end - 1));
  const int8_t* xr = (from >= 0 ? p.xq + from * p.pitch : w0) + inside;  // any row that may be read
  i32x4 codes[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u)  // past the row the weights are zeros
    codes[u] = *reinterpret_cast<const i32x4*>(xr + (unit(u) < units ? 64 * unit(u) : 0));
#pragma unroll
  for (int u = 0; u < UNITS; ++u) codes[u] = turned(codes[u]);

  int turn = 0;
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++turn) {
    i32x4 acc = {};
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(turned(w[u]), codes[u], acc, 0, 0, 0);
    if (tile + gridDim.x < tiles) load(tile + gridDim.x);
    s_sum[turn & 1][wave][lane] = acc;
    __syncthreads();
    // one wave a turn adds up; its buffer is written again two turns later, after
    // a barrier that this wave reaches when it is through
    if (wave != (turn & (kRowWaves - 1))) continue;
    i32x4 sum = {};
#pragma unroll
    for (int v = 0; v < kRowWaves; ++v) sum += s_sum[turn & 1][v][lane];
    const int64_t n = static_cast<int64_t>(tile) * 16 + 4 * (lane >> 4);
    const int left = static_cast<int>(min(p.N - n, int64_t(4)));
    if (m >= t.end || left <= 0) continue;
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[e] = masked(static_cast<float>(sum[e]) * xs * p.ws[t.expert * p.N + n + min(e, left - 1)], keep);
    store_four<DT>(p.y, m * p.N + n, left, f);
  }
}

// ---------------------------------------------------------------------------
// Small tiles: WM x WN x WK waves, each with TM x TN tiles of 32 x 32; the WK
// waves of a tile share each step's K, 128 / WK bytes each.  Few steps are long
// enough to hide anything, so the chain of a step is kept short: STAGES buffers in
// LDS, each asked for STAGES steps ahead; operands read from LDS a step ahead of
// the matrix instructions that use them; one barrier, at which a wave waits for
// the next step's rows only.  LDS is laid out as for the large tiles.
//
// What bounds them is how fast a compute unit gets its rows: 50-60 KB/us, against
// 85-95 for the same loads alone, and 140 for loads that hit the L2 (64 x 64 tiles:
// 16 KB and 0.28 us a step).  Measured and not kept: 64 bytes a step with twice the
// stages (128 x 128 tiles, 512 x 4096 x 4096: 28 us against 23), and asking for the
// lines that a die's workgroups share ahead of time (no change).
// ---------------------------------------------------------------------------
// Loads of 16 bytes a lane from memory to LDS, lane l's to byte 16 l from `to` on
// (one address per wave).  The builtins for these would do, but for the waits: the
// compiler puts one for all of them before a loop's first LDS read, every time
// round.  Nothing lands in a register, and arrive() in stream_kernel does all the
// waiting.  m0 holds the LDS address.  It stands among the clobbers, so that the compiler
// carries no value of its own in it across a load; the warning put off here says that
// it does not save m0 around the statement either, which nothing asks for.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_load(uint32_t to, i32x4 range, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(at), "s"(range)
               : "m0", "memory");
}
__device__ __forceinline__ void lds_load(uint32_t to, const int8_t* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "m0", "memory");
}
#pragma clang diagnostic pop

template <int DT, bool GROUPED, int WM, int WN, int WK, int TM, int TN, int STAGES, bool QUARTERS = false>
__global__ __launch_bounds__(64 * WM* WN* WK) void stream_kernel(Product p) {
  constexpr int kWaves = WM * WN * WK, kThreads = 64 * kWaves;
  constexpr int BM = 32 * WM * TM, BN = 32 * WN * TN;
  constexpr int kRows = kThreads / 8;                         // rows that a load of all threads fills
  constexpr int LM = BM / kRows, LN = BN / kRows, kLoads = LM + LN;
  static_assert(LM * kRows == BM && LN * kRows == BN);
  constexpr int kB = dtype_bytes(DT);
  constexpr int kStage = (BM + BN) * kDepth;
  static_assert(WK == 1 || (TM == 1 && TN == 1));
  __shared__ __attribute__((aligned(256))) int8_t s_rows[STAGES][kStage];
  __shared__ __attribute__((aligned(256))) int8_t s_out[WM * WN * 32 * 32 * TN * kB];
  __shared__ __attribute__((aligned(256))) i32x4 s_meet[WK > 1 ? (WK - 1) * WM * WN * 256 : 1];

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
  const int8_t* w0 = p.wq + (t.expert * p.N + n0) * p.pitch;
  i32x4 rw = range_words(w0, static_cast<uint32_t>(min(int64_t(BN), p.N - n0) * p.pitch));
  i32x4 rx = range_words(GROUPED ? nullptr : p.xq + t.first * p.pitch,
                         static_cast<uint32_t>((t.end - t.first) * p.pitch));
  // scalars that the vector unit has written (range_words) may be read by a load
  // five instructions later; the compiler sees to that for its own loads only
  asm volatile("s_nop 4" : "+s"(rw), "+s"(rx));
  const uint32_t voff = static_cast<uint32_t>(row * pitch + chunk);
  const int8_t* xrow[GROUPED ? LM : 1];
  if constexpr (GROUPED) {
#pragma unroll
    for (int i = 0; i < LM; ++i) {
      const int64_t m = t.first + row + kRows * i;
      const int64_t src = m < t.end ? source_row<true>(p, m) : -1;
      xrow[i] = src >= 0 ? p.xq + src * p.pitch : w0;  // any row that may be read
    }
  }
  const uint32_t lds0 = lds_address(s_rows[0]) + 8 * wave * kDepth;
  // load i of a thread for step k / 128: the channels' rows first
  auto load = [&](int stage, int i, int k) {
    const bool in = k + chunk < end;
    const uint32_t v = in ? voff + k : kNever, to = lds0 + stage * kStage + kRows * i * kDepth;
    if (i < LN)
      lds_load(to, rw, v + kRows * i * pitch);
    else if constexpr (GROUPED)
      lds_load(to, xrow[GROUPED ? i - LN : 0] + (in ? k + chunk : 0));
    else
      lds_load(to, rx, v + kRows * (i - LN) * pitch);
  };

  const int wk = wave % WK, wn = wave / WK % WN * (32 * TN), wm = wave / (WK * WN) * (32 * TM);
  constexpr int kParts = 4 / WK;
  i32x16 acc[TN][TM] = {};
  constexpr int kReads = kParts * (TN + TM), kProducts = kParts * TN * TM;
  i32x4 operand[2][kParts][TN + TM];
  // read i of a step: of each part the channels' operands, then the tokens'
  auto fetch = [&](int set, int stage, int i) {
    const int part = i / (TN + TM), q = i % (TN + TM);
    const int at = (lane & 31) * kDepth + (((2 * (wk * kParts + part) + (lane >> 5)) ^ (lane >> 1 & 7)) * 16);
    const int first = q < TN ? wn + 32 * q : BN + wm + 32 * (q - TN);
    operand[set][part][q] = *reinterpret_cast<const i32x4*>(s_rows[stage] + first * kDepth + at);
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
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(operand[set][part][i], operand[set][part][TN + j],
                                                        acc[i][j], 0, 0, 0);
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
    // the tile's other waves hand their sums to the first
    const int slot = (wave / WK) * (WK - 1) - 1;
    if (wk > 0)
#pragma unroll
      for (int c = 0; c < 16; c += 4)
        s_meet[((slot + wk) * 4 + c / 4) * 64 + lane] = i32x4{acc[0][0][c], acc[0][0][c + 1], acc[0][0][c + 2], acc[0][0][c + 3]};
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int v = 1; v < WK; ++v)
#pragma unroll
      for (int c = 0; c < 16; c += 4) {
        const i32x4 o = s_meet[((slot + v) * 4 + c / 4) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][0][c + e] += o[e];
      }
  }
  if constexpr (!GROUPED) {
    if (p.splits > 1) {
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int64_t m = t.first + wm + 32 * j + (lane & 31);
        if (m >= t.end) continue;
        int32_t* to = p.sums + (blockIdx.y * p.M + m) * p.sums_pitch;
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const int64_t n = n0 + wn + 32 * i + 2 * c + 4 * (lane >> 5);
            if (n < p.sums_pitch)
              *reinterpret_cast<i32x4*>(to + n) =
                  i32x4{acc[i][j][c], acc[i][j][c + 1], acc[i][j][c + 2], acc[i][j][c + 3]};
          }
      }
      return;
    }
  }
  const float* ws = p.ws + t.expert * p.N;
  write_tile<DT, TM, TN, 32 * TN>(
      p, t.end, n0 + wn, t.first + wm, acc, s_out + wave / WK * (32 * 32 * TN * kB),
      [&](int c) {
        const int64_t n = n0 + wn + c;
        return make_float4(n < p.N ? ws[n] : 0.0f, n + 1 < p.N ? ws[n + 1] : 0.0f, n + 2 < p.N ? ws[n + 2] : 0.0f,
                           n + 3 < p.N ? ws[n + 3] : 0.0f);
      },
      [&](int j) {
        const int64_t m = t.first + wm + 32 * j + (lane & 31);
        const int64_t src = m < t.end ? source_row<GROUPED>(p, m) : -1;
        return RowToken{src >= 0 ? p.xs[src] : 0.0f, keep_mask<GROUPED>(src)};
      });
}

// The sums of a product whose K was split, four channels of a token to a thread.
template <int DT>
__global__ __launch_bounds__(256) void join_kernel(Product p) {
  const int64_t fours = p.sums_pitch / 4, all = p.M * fours;
  for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < all; i += gridDim.x * int64_t(256)) {
    const int64_t m = i / fours, n = i % fours * 4;
    i32x4 sum = {};
    for (int v = 0; v < p.splits; ++v)
      sum += *reinterpret_cast<const i32x4*>(p.sums + (v * p.M + m) * p.sums_pitch + n);
    const int left = static_cast<int>(min(p.N - n, int64_t(4)));
    const float xs = p.xs[m];
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = static_cast<float>(sum[e]) * xs * p.ws[n + min(e, left - 1)];
    store_four<DT>(p.y, m * p.N + n, left, f);
  }
}

// Tiles of BM rows that p.M rows need at most: every expert ends in at most one
// tile that is not full.
template <bool GROUPED>
int64_t row_tiles(const Product& p, int64_t BM) {
  if constexpr (GROUPED) return p.M / BM + (p.M < p.experts ? p.M : p.experts);
  return (p.M + BM - 1) / BM;
}

// Workgroups of `threads` for the tiles, a multiple of the dies; 0 if a grid
// cannot have so many.
template <bool GROUPED>
uint32_t tile_groups(const Product& p, int BM, int BN, int threads) {
  const int64_t all = row_tiles<GROUPED>(p, BM) * ((p.N + BN - 1) / BN);
  const int64_t groups = (all + kDies - 1) / kDies * kDies;
  return groups * threads < (int64_t(1) << 32) ? static_cast<uint32_t>(groups) : 0;
}

template <bool GROUPED, Share SHARE>
void launch_share(const Product& p, int32_t y_dtype, uint32_t groups, hipStream_t st) {
  with_dtype(y_dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    if constexpr (SHARE == kQuarters)
      hipLaunchKernelGGL((stream_kernel<DT, GROUPED, 2, 2, 1, 2, 2, 4, true>), dim3(groups), dim3(256), 0, st, p);
    else
      hipLaunchKernelGGL((tile_kernel<DT, GROUPED, SHARE>), dim3(groups), dim3(kTileThreads), 0, st, p);
  });
}

// Tiles of 256 x 256.  A last turn of the compute units that is half full at most is
// computed in halves of 128 tokens, in a second launch (8192 x 11008 x 4096 has 1376
// tiles, five turns of 256 and 96: 342 us whole, 331 so, 340 in quarters), and one
// that is a quarter full at most in quarters, by the kernel for smaller tiles (4352 x
// 4096 x 4096 with 272: 92 us in halves, 81 so; 576 tiles of eight experts' 4096 x
// 4096: 162 and 154).  For experts each launch that finds nothing to do costs 1.7 us.
template <bool GROUPED>
nf4_status launch_tiles(const Product& p, int32_t y_dtype, hipStream_t st) {
  const uint32_t groups = tile_groups<GROUPED>(p, kTile, kTile, kTileThreads);
  if (groups == 0) return NF4_EUNSUPPORTED;
  // how many tiles experts' rows make only the GPU knows: the launches find out
  const int64_t all = row_tiles<GROUPED>(p, kTile) * ((p.N + kTile - 1) / kTile);
  const uint32_t whole = whole_tiles(static_cast<uint32_t>(all), p.cus);
  if (GROUPED || whole > 0) launch_share<GROUPED, kWhole>(p, y_dtype, groups, st);
  const uint32_t rest = static_cast<uint32_t>(all) - whole, turn = (p.cus + kDies - 1) / kDies * kDies;
  const bool quarters = in_quarters(rest, p.cus);
  if (GROUPED || (rest > 0 && !quarters)) launch_share<GROUPED, kHalves>(p, y_dtype, turn, st);
  if (GROUPED || (rest > 0 && quarters)) launch_share<GROUPED, kQuarters>(p, y_dtype, turn, st);
  return launch_status();
}

template <bool GROUPED, int WM, int WN, int WK, int TM, int TN, int STAGES>
nf4_status launch_stream(const Product& p, int32_t y_dtype, hipStream_t st) {
  constexpr int kThreads = 64 * WM * WN * WK;
  const uint32_t groups = tile_groups<GROUPED>(p, 32 * WM * TM, 32 * WN * TN, kThreads);
  if (groups == 0) return NF4_EUNSUPPORTED;
  with_dtype(y_dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    hipLaunchKernelGGL((stream_kernel<DT, GROUPED, WM, WN, WK, TM, TN, STAGES>),
                       dim3(groups, static_cast<uint32_t>(p.splits)), dim3(kThreads), 0, st, p);
    if (p.splits > 1) {
      const int64_t blocks = (p.M * (p.sums_pitch / 4) + 255) / 256;
      hipLaunchKernelGGL((join_kernel<DT>), dim3(static_cast<uint32_t>(blocks < 4096 ? blocks : 4096)), dim3(256),
                         0, st, p);
    }
  });
  return launch_status();
}

// The longest rows: a wave's weights and codes take 176 of its 256 registers.  Past them
// tiles do better: with 24 units 16 x 4096 x 12288 takes 17.4 us against 14.7, with 28 x
// 14336 27.7 against 16.0 (at 11264 13.3 against 14.6), 16 x 4 tokens of 64 experts of
// 1024 x 14336 236 against 124.
constexpr int64_t kRowMaxUnits = 22;
constexpr int64_t kRowMaxPitch = kRowMaxUnits * kRowWaves * 64;

// The variant for rows of `pitch` bytes: units of 64 that a wave holds.
int64_t row_units(int64_t pitch) {
  const int64_t units = (pitch / 64 + kRowWaves - 1) / kRowWaves;
  return units <= 4 ? 4 : units <= 8 ? 8 : kRowMaxUnits;
}

template <bool GROUPED>
nf4_status launch_rows(const Product& p, int32_t y_dtype, hipStream_t st) {
  const int64_t tiles = (p.N + 15) / 16, rows = row_tiles<GROUPED>(p, 16);
  // two workgroups fit a compute unit
  const int64_t most = 2 * device_cus(), share = (most + rows - 1) / rows;
  const dim3 grid(static_cast<uint32_t>(tiles < share ? tiles : share), static_cast<uint32_t>(rows));
  const int64_t units = row_units(p.pitch);
  with_dtype(y_dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    if (units == 4)
      hipLaunchKernelGGL((row_kernel<DT, GROUPED, 4>), grid, dim3(kRowThreads), 0, st, p);
    else if (units == 8)
      hipLaunchKernelGGL((row_kernel<DT, GROUPED, 8>), grid, dim3(kRowThreads), 0, st, p);
    else
      hipLaunchKernelGGL((row_kernel<DT, GROUPED, kRowMaxUnits>), grid, dim3(kRowThreads), 0, st, p);
  });
  return launch_status();
}

// Rows whose codes and weights leave room for two workgroups on a compute unit: eight
// units of 64 bytes a wave.
constexpr int64_t kShortPitch = 8 * 64 * kRowWaves;

// The longest rows fill the registers that 16 waves a compute unit leave to one: with
// 12 blocks 1 x 4096 x 12288 takes 16.8 us against 15.0 in tiles, with 14 x 14336 24.4
// against 15.7 (at 11264 11.5 against 14.3; codes given).
constexpr int64_t kDotTokens = 2, kDotBlocks = 11;

// Whether the product goes to the single tokens' kernel, which quantizes on the
// way where it is given values: 2 x 4096 x 4096 in 7.6 us against 9.2 in two launches,
// 2 x 4096 x 11008 in 16.7 against 17.5; four tokens would take 15.0 against 14.4 at
// 11008 x 4096 and 23.5 against 17.6 at 4096 x 11008.  (Past 4096 channels of more than
// 8192 values two tokens do no better than in tiles: 2 x 8192 x 11264 26.8 against 22.7,
// 2 x 11008 x 11008 without the codes 30.3 against 30.9.)
bool single(int64_t M, int64_t K) { return M <= kDotTokens && pitch_of(K) <= kDotBlocks * 1024; }

// The variant for rows of `pitch` bytes: blocks of 1024 that it holds.
int64_t dot_blocks(int64_t pitch) { return pitch <= 4 * 1024 ? 4 : pitch <= 8 * 1024 ? 8 : kDotBlocks; }

template <int XT, int DT, int MT>
void launch_dot_blocks(const Product& p, const void* x, int64_t K, hipStream_t st) {
  const int64_t tiles = (p.N + kDotRows - 1) / kDotRows, most = 2 * device_cus();
  const dim3 grid(static_cast<uint32_t>(tiles < most ? tiles : most));
  const int64_t blocks = dot_blocks(p.pitch);
  if (blocks == 4)
    hipLaunchKernelGGL((dot_kernel<XT, DT, MT, 4>), grid, dim3(kDotThreads), 0, st, p, x, static_cast<int>(K));
  else if (blocks == 8)
    hipLaunchKernelGGL((dot_kernel<XT, DT, MT, 8>), grid, dim3(kDotThreads), 0, st, p, x, static_cast<int>(K));
  else
    hipLaunchKernelGGL((dot_kernel<XT, DT, MT, kDotBlocks>), grid, dim3(kDotThreads), 0, st, p, x,
                       static_cast<int>(K));
}

// The tokens' codes (XT = kCodes) or the tokens at x.
template <int XT>
nf4_status launch_dot(const Product& p, const void* x, int64_t K, int32_t y_dtype, hipStream_t st) {
  with_dtype(y_dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    if (p.M == 1)
      launch_dot_blocks<XT, DT, 1>(p, x, K, st);
    else
      launch_dot_blocks<XT, DT, kDotTokens>(p, x, K, st);
  });
  return launch_status();
}

// The tiled kernels, and what their steps of 128 bytes of K take (us, measured at
// 4096 x 4096, 11008 x 4096, 4096 x 11008, 2048 x 2048 and 1024 x 11008 with 32 to
// 2048 rows): where few compute units have a tile, and for each of its tiles where
// all have one or more (the memory behind them is busier then).  Largest tiles load
// the least per product, but leave compute units idle and take the longest for
// themselves: 512 x 4096 x 4096 takes 35 / 35 / 20 / 17 / 23 / 47 us from the smallest
// tiles to the largest, 64 x 4096 x 4096 8.5 / 10 / 12 / 14 / 19 / 44, 1024 x 11008 x
// 4096 176 / 174 / 88 / 94 / 70 / 52.
struct Tiling {
  int BM, BN;        // tokens, channels
  float alone, each; // us a step
  float fixed;       // us a turn that no step hides
};
constexpr Tiling kTilings[] = {{32, 32, 0.16f, 0.125f, 0.0f}, {64, 32, 0.215f, 0.25f, 0.0f},
                               {64, 64, 0.28f, 0.255f, 0.0f}, {128, 64, 0.35f, 0.47f, 0.0f},
                               {128, 128, 0.55f, 0.69f, 0.0f}, {256, 256, 1.05f, 1.6f, 4.0f}};
constexpr int kLargest = 5;
constexpr float kLaunchUs = 3.0f, kJoinUs = 4.5f, kSumUs = 8.0f / 3e6f;  // a sum there and back
constexpr int kMaxSplits = 16;

struct Plan {
  int tiling, splits;
};

// The tiling with the least time by the figures above, with K split over
// workgroups where that leaves compute units without a tile and the workspace has
// room for the sums (128 x 1024 x 11008: 15.2 us in one piece, 12.9 in six; 88 x 999
// x 34756: 39 and 20 in seven), unless writing and reading the sums costs as much
// (65 x 2100 x 8192: 11 us in one piece, 21 in thirteen).  The model orders the tilings;
// it is no time of long weights from memory, which it does not know (1 x 8192 x 28672:
// 39 us by it, while its bytes take 48).  Rows
// sorted by expert: every expert with rows ends in a tile that is half full, and
// where there are tiles for all compute units the weights' stream counts, which
// tiles of 32 channels hold up (1024 rows over 64 experts of 1024 x 2048: 31.8 us
// against 25.8).
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
    if (GROUPED && t.BN == 32 && tiles > cus) continue;
    const int most = GROUPED || i == kLargest ? 1 : kMaxSplits;
    for (int splits = 1; splits <= most; ++splits) {
      if (splits > 1 && (tiles * splits > cus || p.M * p.sums_pitch * 4 * splits > static_cast<int64_t>(room) ||
                         steps < 4 * splits))
        break;
      const double full = tiles * splits / cus, part = full - std::floor(full);
      double turns = std::ceil(full);
      if (i == kLargest && part > 0 && part <= 0.5) turns -= full > 1 && part <= 0.25 ? 0.6 : 0.3;  // in pieces
      const double more = t.each > t.alone ? t.each - t.alone : 0.0;
      const double step = full > 1 || turns < 1 ? turns * t.each : t.alone + more * full;
      const double us = kLaunchUs + turns * t.fixed + std::ceil(steps / splits) * step + (splits > 1 ? kJoinUs + p.M * p.sums_pitch * splits * kSumUs : 0.0);
      if (us < least * (splits > 1 ? 0.85 : 1.0)) {
        least = us;
        best = {i, splits};
      }
    }
  }
  return best;
}

Product dense(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws, void* y, int64_t M, int64_t N,
              int64_t K) {
  Product p = {};
  p.xq = xq, p.xs = xs, p.wq = wq, p.ws = ws, p.y = y;
  p.M = M, p.N = N, p.pitch = pitch_of(K), p.x_rows = M;
  p.top_k = p.experts = p.splits = 1;
  p.sums_pitch = (N + 3) / 4 * 4;
  p.cus = static_cast<uint32_t>(device_cus());
  return p;
}

// Whether the row kernel takes the product: it reads weights once for every 16 rows.
// Dense: 16 x 4096 x 4096 in 6.7 us, 8.4 in tiles; more rows where every workgroup that
// the card holds at a time (two to a compute unit, one where rows are long) has one
// tile of 16 x 16 at most, whose start is shorter than a larger tile's: 32 x 4096 x
// 4096 in 8.3 us against 9.3, 64 x 1024 x 4096 in 4.2 against 6.4, 32 x 2048 x 11008
// in 10.3 against 12.4, 512 x 256 x 4096 in 5.6 against 6.3; 48 x 4096 x 4096 would
// take 11.4 against 8.5, 17 x 4096 x 11008 23.5 against 15.2.  By expert: with 64
// experts of 4096 x 2048 two rows each on average take 96 us against 107, four 103
// against 111, six 114 against 110, sixteen 157 against 111 (any with more than 16 is
// read twice); with fewer tiles than compute units its shorter start counts to ten rows
// (16 experts of 256 x 512: 4.5 us against 5.0).
//
// Long rows leave one workgroup to a compute unit, with nothing beside it while it
// starts or turns to its next tile.  Up to 16 rows of a dense product: one tile each is
// as good as before (16 x 4096 x 6144 in 9.3 us against 10.4, x 11264 in 13.3 against
// 14.6; x 4160 in 8.4 against 8.9), a second turn is not (16 x 4608 x 4160 13.8 against
// 9.0, 16 x 8192 x 7168 18.4 against 13.6, x 11264 24.0 against 19.4), and more turns
// pay from 8192 on (16 x 11008 x 7168 21.4 against 20.9, x 8192 23.1 against 23.9, x
// 11264 28.1 against 31.0; to 16384 channels 39.5 against 34.4).  By expert: tiles do
// better (two tokens of eight experts of 4096 x 6144: 20.7 us against 11.9, 16 x 4 of
// 64 of 1024 x 4160 65 against 38, x 8192 31 against 22 for 4 x 4), except past 8192
// where the tiles here are about as many as the compute units (four rows of an expert
// of 1024 x 11264 9.6 against 11.1, 64 x 4 of 64 of 64 15.3 against 17.5; 16 of 16
// experts of 512 26.7 against 17.4), and with many of them and rows of 8192 bytes,
// which suit the tiles the least (32 x 4 of 64 of 1024 90 against 104, 16 x 4 of 2048
// 165 against 152; at 9216 97 against 97 and 176 against 150).
template <bool GROUPED>
bool few(const Product& p) {
  if (p.pitch <= 0 || p.pitch > kRowMaxPitch || row_tiles<GROUPED>(p, 16) > 65535) return false;
  const int64_t cus = device_cus(), tiles = row_tiles<GROUPED>(p, 16) * ((p.N + 15) / 16);
  const bool is_short = p.pitch <= kShortPitch;
  if (GROUPED) {
    const int64_t rows = p.M / p.experts;
    if (!is_short && !(p.pitch > 2 * kShortPitch && 4 * tiles <= 5 * cus) &&
        !(p.pitch == 2 * kShortPitch && tiles > 16 * cus))
      return false;
    return rows <= 4 || (rows <= 10 && p.experts * ((p.N + 63) / 64) <= cus);
  }
  if (tiles <= (is_short ? 2 : 1) * cus) return true;
  return p.M <= 16 && (is_short || (p.pitch >= 2 * kShortPitch && tiles > 2 * cus));
}

// What a product goes to: the one- and two-token kernel, the few-row kernel, or tiles
// as planned.
constexpr int kToDot = -2, kToRows = -1;

template <bool GROUPED>
Plan choose(const Product& p, size_t room) {
  if (!GROUPED && single(p.M, p.pitch)) return {kToDot, 1};
  if (few<GROUPED>(p)) return {kToRows, 1};
  return plan<GROUPED>(p, room);
}

template <bool GROUPED>
nf4_status launch(Product p, int32_t y_dtype, void* workspace, size_t room, hipStream_t st) {
  const Plan plan_ = choose<GROUPED>(p, workspace ? room : 0);
  if constexpr (!GROUPED)
    if (plan_.tiling == kToDot) return launch_dot<kCodes>(p, nullptr, 0, y_dtype, st);
  if (plan_.tiling == kToRows) return launch_rows<GROUPED>(p, y_dtype, st);
  p.splits = plan_.splits;
  p.sums = static_cast<int32_t*>(workspace);
  switch (plan_.tiling) {
    case 0: return launch_stream<GROUPED, 1, 1, 4, 1, 1, 8>(p, y_dtype, st);
    case 1: return launch_stream<GROUPED, 2, 1, 2, 1, 1, 8>(p, y_dtype, st);
    case 2: return launch_stream<GROUPED, 2, 2, 1, 1, 1, 4>(p, y_dtype, st);
    case 3: return launch_stream<GROUPED, 2, 2, 1, 2, 1, 4>(p, y_dtype, st);
    case 4: return launch_stream<GROUPED, 2, 2, 1, 2, 2, 4>(p, y_dtype, st);
    default: return launch_tiles<GROUPED>(p, y_dtype, st);
  }
}

// What the products check alike (the activations apart).
nf4_status check_product(const int8_t* wq, const float* ws, int64_t N, int64_t K, const void* y,
                         int32_t y_dtype) {
  if (!y || !ws || (K > 0 && !wq)) return NF4_EINVAL;
  if (!aligned(wq, 16) || !aligned(ws, 4) || !aligned(y, dtype_bytes(y_dtype))) return NF4_EINVAL;
  if (N > kMaxDim || K > kMaxK) return NF4_EUNSUPPORTED;
  return NF4_OK;
}

size_t scales_bytes(int64_t M) { return static_cast<size_t>(M * 4 + 255) / 256 * 256; }
size_t codes_bytes(int64_t M, int64_t K) { return static_cast<size_t>(M * pitch_of(K) + 255) / 256 * 256; }

}  // namespace

extern "C" {

nf4_status nf4_probe_int8_plan(int64_t M, int64_t N, int64_t K, int32_t experts, size_t room, int32_t* plan,
                               int32_t* detail) {
  if (!plan || !detail || M < 1 || N < 1 || K < 0 || experts < 0) return NF4_EINVAL;
  if (M > kMaxDim || N > kMaxDim || K > kMaxK || experts > kMaxExperts) return NF4_EUNSUPPORTED;
  Product p = dense(nullptr, nullptr, nullptr, nullptr, nullptr, M, N, K);
  if (experts > 0) p.experts = experts;
  const Plan best = experts > 0 ? choose<true>(p, 0) : choose<false>(p, room);
  *plan = best.tiling;
  if (best.tiling == kToDot) {
    *detail = static_cast<int32_t>(dot_blocks(p.pitch));
  } else if (best.tiling == kToRows) {
    *detail = static_cast<int32_t>(row_units(p.pitch));
  } else if (best.tiling < kLargest || experts > 0) {
    *detail = best.splits;
  } else {
    const uint32_t all = static_cast<uint32_t>(row_tiles<false>(p, kTile) * ((N + kTile - 1) / kTile));
    const uint32_t whole = whole_tiles(all, p.cus), rest = all - whole;
    *detail = (whole > 0 ? 1 : 0) + (rest == 0 ? 0 : in_quarters(rest, p.cus) ? 4 : 2);
  }
  return NF4_OK;
}

size_t int8_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxK) return 0;
  const Product p = dense(nullptr, nullptr, nullptr, nullptr, nullptr, M, N, K);
  const Plan best = choose<false>(p, static_cast<size_t>(1) << 62);
  return best.splits > 1 ? static_cast<size_t>(M * p.sums_pitch * 4 * best.splits) : 0;
}

nf4_status int8_gemm(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                     int64_t M, int64_t N, int64_t K, void* y, int32_t y_dtype, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || !known_dtype(y_dtype) || !aligned(workspace, 256))
    return NF4_EINVAL;
  if (M == 0 || N == 0) return NF4_OK;
  if (!xs || (K > 0 && !xq) || !aligned(xq, 16) || !aligned(xs, 4)) return NF4_EINVAL;
  if (const nf4_status st = check_product(wq, ws, N, K, y, y_dtype)) return st;
  if (M > kMaxDim) return NF4_EUNSUPPORTED;
  return launch<false>(dense(xq, xs, wq, ws, y, M, N, K), y_dtype, workspace, workspace_bytes,
                       reinterpret_cast<hipStream_t>(stream));
}

size_t int8_linear_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxK) return 0;
  if (single(M, K)) return 0;
  return codes_bytes(M, K) + scales_bytes(M) + int8_gemm_workspace_size(M, N, K);
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
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (single(M, K)) {
    const Product p = dense(nullptr, nullptr, wq, ws, y, M, N, K);
    nf4_status result = NF4_OK;
    with_dtype(x_dtype, [&](auto a) { result = launch_dot<decltype(a)::value>(p, x, K, y_dtype, st); });
    return result;
  }
  // the codes and scales have to have room; the rest is for the sums of a split, which
  // a workspace made for another shape may not hold (a smaller M may split more)
  const size_t used = codes_bytes(M, K) + scales_bytes(M);
  if (!workspace || workspace_bytes < used) return NF4_EINVAL;
  int8_t* xq = static_cast<int8_t*>(workspace);
  float* xs = reinterpret_cast<float*>(xq + codes_bytes(M, K));
  quantize_launch(x, x_dtype, M, K, xq, xs, st);
  return launch<false>(dense(xq, xs, wq, ws, y, M, N, K), y_dtype, xq + used, workspace_bytes - used, st);
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
  Product p = dense(xq, xs, wq, ws, y, rows, N, K);
  p.order = order, p.offsets = offsets, p.x_rows = x_rows;
  p.top_k = order ? top_k : 1, p.experts = experts;
  return launch<true>(p, y_dtype, nullptr, 0, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
