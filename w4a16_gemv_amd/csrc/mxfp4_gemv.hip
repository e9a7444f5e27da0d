// mxfp4_gemv.hip -- activations as they are times 4-bit microscaled weights: up to
// 16 rows (mxfp4_gemv), and the expert layer of a few tokens (mxfp4_moe_mlp).
//
// v_mfma_f32_16x16x32_bf16 with the weights as A: lane i + 16 g holds A[i][8 g .. + 7],
// B likewise with i the column, and D[4 g .. + 3][i].  Every value of the format is a
// bf16 number, so the weights are converted on the way (two codes and their scale an
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

// Eight activations to the parts' eight bf16 numbers each.
template <int DT>
__device__ __forceinline__ void split_piece(const Piece<DT>& p, u32x4 (&out)[parts_of(DT)]) {
  if constexpr (DT == INT8_BF16) {
    out[0] = p.v[0];
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float a[3], b[3];
      split(element<DT>(p, i), a);
      split(element<DT>(p, i + 1), b);
#pragma unroll
      for (int k = 0; k < parts_of(DT); ++k) out[k][i / 2] = upper_halves(a[k], b[k]);
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

struct Loaded {
  i32x4 codes;
  uint32_t scales;
};

__device__ __forceinline__ Loaded load_unit(const Channels& c, int unit, bool in) {
  return {__builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(c.codes, in ? c.code_at + 64 * unit : kNever, 0, 0)),
          __builtin_amdgcn_raw_buffer_load_b32(c.scales, in ? c.scale_at + 128 * unit : kNever, 0, 0)};
}

// The lane's block of a unit: 32 codes to lane i + 16 g, as four operands.
__device__ __forceinline__ void operands(const Loaded& l, bf16x8 (&a)[4]) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int from = 4 * (4 * (lane & 15) + g);  // a lane's number times 4
  const float s = scale_value(l.scales >> (8 * g) & 255);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int w = l.codes[e];
    a[e] = weights8(static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(from, w)), s);
  }
}

// The rows that a wave's products are made with: `count` (16 at most) of them, rows of
// `width` values of type DT (or, for kSplit + parts, that many rows of bf16 numbers each,
// `width` numbers long, zeros past the data).
constexpr int kSplit = 8;
__device__ __host__ constexpr int source_parts(int dt) { return dt >= kSplit ? dt - kSplit : parts_of(dt); }

// A lane's share of a unit: lane c + 16 r has elements 8 c .. + 7 of rows r, r + 4, ...
template <int DT, int RU>
struct Share {
  static constexpr int kParts = source_parts(DT);
  u32x4 v[RU][DT >= kSplit ? kParts : DT == INT8_FP32 ? 2 : 1];
};

// LDS of a wave: rows of a unit at a pitch of 272 bytes (so that a chunk of 16 rows lies
// in different banks), the parts one after the other.
constexpr int kLdsRow = 2 * kUnit + 16;

template <int DT, int RU>
__device__ __forceinline__ void stage(const Share<DT, RU>& x, uint8_t* lds, int count) {
  constexpr int kParts = source_parts(DT);
  const int lane = threadIdx.x & 63;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int j = 0; j < RU; ++j) {
    if (4 * j >= count) break;
    u32x4 part[kParts];
    if constexpr (DT >= kSplit) {
#pragma unroll
      for (int k = 0; k < kParts; ++k) part[k] = x.v[j][k];
    } else {
      Piece<DT> p;
      p.v[0] = x.v[j][0];
      if constexpr (DT == INT8_FP32) p.v[1] = x.v[j][1];
      split_piece<DT>(p, part);
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      *reinterpret_cast<u32x4*>(lds + (k * 4 * RU + 4 * j + (lane >> 4)) * kLdsRow + (lane & 15) * 16) = part[k];
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Part k's operand e of the lane's column.
template <int RU>
__device__ __forceinline__ bf16x8 staged(const uint8_t* lds, int k, int e, int column) {
  const int g = (threadIdx.x & 63) >> 4;
  return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(lds + (k * 4 * RU + column) * kLdsRow + 64 * g + 16 * e));
}

// Loads a unit's share of the rows row(0), row(1) ... (pointers; asked for below `count`
// only).
template <int DT, int RU, class Row>
__device__ __forceinline__ Share<DT, RU> load_share(int unit, bool in, int64_t width, int count, Row&& row) {
  Share<DT, RU> x;
  const int lane = threadIdx.x & 63;
  const int64_t at = int64_t(kUnit) * unit + 8 * (lane & 15);
#pragma unroll
  for (int j = 0; j < RU; ++j) {
    constexpr int kWords = sizeof(x.v[0]) / 16;
#pragma unroll
    for (int k = 0; k < kWords; ++k) x.v[j][k] = u32x4{0, 0, 0, 0};
    if (!in || 4 * j >= count) continue;
    const char* r = row(min(4 * j + (lane >> 4), count - 1));
    if constexpr (DT >= kSplit) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) x.v[j][k] = *reinterpret_cast<const u32x4*>(r + 2 * (k * width + at));
    } else {
      Piece<DT> p = {};
      if (int64_t(kUnit) * (unit + 1) <= width)
        p = whole_piece<DT>(r, at);
      else if (at < width)
        p = load_piece<DT>(r, at, width);
#pragma unroll
      for (int k = 0; k < kWords; ++k) x.v[j][k] = p.v[k];
    }
  }
  return x;
}

// acc[c] += the products of CT tiles of channels with the rows over the units first ..
// last - 1, DEPTH units in flight.
template <int DT, int RU, int CT, int DEPTH, class Row>
__device__ __forceinline__ void run_units(const Channels (&ch)[CT], int first, int last, int64_t width, int count,
                                          uint8_t* lds, Row&& row, f32x4 (&acc)[CT]) {
  constexpr int kParts = source_parts(DT);
  const int column = min(static_cast<int>(threadIdx.x & 15), count - 1);
  Loaded w[DEPTH][CT];
  Share<DT, RU> x[DEPTH];
  auto load = [&](int d, int unit) {
    const bool in = unit < last;
#pragma unroll
    for (int c = 0; c < CT; ++c) w[d][c] = load_unit(ch[c], unit, in);
    x[d] = load_share<DT, RU>(unit, in, width, count, row);
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(d, first + d);
  for (int u = first; u < last; u += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (u + d >= last) break;
      stage<DT, RU>(x[d], lds, count);
      bf16x8 a[CT][4];
#pragma unroll
      for (int c = 0; c < CT; ++c) operands(w[d][c], a[c]);
#pragma unroll
      for (int k = 0; k < kParts; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bf16x8 b = staged<RU>(lds, k, e, column);
#pragma unroll
          for (int c = 0; c < CT; ++c) acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[c][e], b, acc[c], 0, 0, 0);
        }
      __builtin_amdgcn_sched_barrier(0);
      load(d, u + d + DEPTH);
    }
  }
}

// The units of a wave: pairs (whole lines), as even over the waves as they go.
__device__ __forceinline__ void share_of(int units, int wave, int& first, int& last) {
  const int each = 2 * ((units + 2 * kWaves - 1) / (2 * kWaves));
  first = min(units, wave * each);
  last = min(units, first + each);
}

// ---------------------------------------------------------------------------
// Up to 16 rows.  A workgroup goes through the channels 16 at a time; its eight waves
// share K.  The weights go from memory through registers to the matrix cores, the rows
// through registers and the wave's own piece of LDS, several units of both in flight.  The
// waves' sums meet in LDS and are added in the waves' order.
// ---------------------------------------------------------------------------
struct Gemv {
  const void* x;
  const uint8_t* wq;
  const uint8_t* ws;
  void* y;
  int64_t M, N, K, pitch, steps;
};

template <int XT, int RU>
constexpr int stage_bytes() {
  return source_parts(XT) * 4 * RU * kLdsRow;
}

template <int XT, int DT, int RU>
__global__ __launch_bounds__(kThreads, 4) void mx_gemv_kernel(Gemv p) {
  __shared__ __attribute__((aligned(16))) uint8_t s_x[kWaves][stage_bytes<XT, RU>()];
  __shared__ f32x4 s_sum[2][kWaves][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t tiles = static_cast<uint32_t>((p.N + 15) / 16);
  const int units = static_cast<int>(p.pitch / 64), count = static_cast<int>(p.M);
  int first, last;
  share_of(units, wave, first, last);
  auto row = [&](int r) { return static_cast<const char*>(p.x) + r * p.K * dtype_bytes(XT); };
  int turn = 0;
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++turn) {
    const int64_t n0 = int64_t(16) * tile;
    const Channels ch[1] = {channels(p.wq, p.ws, n0, p.N - n0, p.pitch, p.steps)};
    f32x4 acc[1] = {};
    run_units<XT, RU, 1, 4>(ch, first, last, p.K, count, s_x[wave], row, acc);
    s_sum[turn & 1][wave][lane] = acc[0];
    __syncthreads();
    // one wave a turn adds up; its buffer is written again two turns later, after
    // a barrier that this wave reaches when it is through
    if (wave != (turn & (kWaves - 1))) continue;
    f32x4 sum = s_sum[turn & 1][0][lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) sum += s_sum[turn & 1][v][lane];
    const int64_t n = n0 + 4 * (lane >> 4);
    const int left = static_cast<int>(min(p.N - n, int64_t(4)));
    if ((lane & 15) >= count || left <= 0) continue;
    const float f[4] = {sum[0], sum[1], sum[2], sum[3]};
    store_four<DT>(p.y, (lane & 15) * p.N + n, left, f);
  }
}

// ---------------------------------------------------------------------------
// The expert layer.  Both kernels first see from the ids which tokens go to which
// expert: a mask of tokens to each.  The experts that have any are numbered in their
// order, and their (expert, token) pairs too: these are the rows of what lies between the
// two products (h).
//
//  up:    a workgroup takes an expert's 16 channels (of the gate and of the others) and
//         its tokens; eight waves share H.  act(v) times the router's weight goes to h as
//         parts.
//  down:  a workgroup takes 16 channels of y; its waves share the experts' F, an expert
//         after the other, and add each's sums to those of the tokens that it has.
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
};

// What h is kept in: 16 bits of each number, or all of fp32.
__device__ __host__ constexpr int h_parts(int dt) { return dt == INT8_FP32 ? 3 : 2; }

struct Routing {
  uint32_t masks[kMaxExperts][2];  // of an expert's tokens
};

__device__ __forceinline__ int64_t id_of(const Mlp& p, int slot) {
  return p.id_bytes == 8 ? static_cast<const int64_t*>(p.ids)[slot] : static_cast<const int32_t*>(p.ids)[slot];
}

// Fills the masks; past it every wave may read them.
__device__ __forceinline__ void read_routing(const Mlp& p, Routing& r) {
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) r.masks[e][0] = r.masks[e][1] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < p.T * p.top_k; s += blockDim.x) {
    const int64_t e = id_of(p, s);
    const int t = s / p.top_k;
    if (e >= 0 && e < p.experts) atomicOr(&r.masks[e][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
}

__device__ __forceinline__ uint64_t mask_of(const Routing& r, int e) {
  return static_cast<uint64_t>(r.masks[e][1]) << 32 | r.masks[e][0];
}

// The n'th token of a mask (n below their number).
__device__ __forceinline__ int nth_token(uint64_t mask, int n) {
  for (int i = 0; i < n; ++i) mask &= mask - 1;
  return __builtin_ctzll(mask);
}

template <int DT, int RU>
__global__ __launch_bounds__(kThreads, 2) void mx_up_kernel(Mlp p) {
  __shared__ __attribute__((aligned(16))) uint8_t s_x[kWaves][stage_bytes<DT, RU>()];
  __shared__ f32x4 s_sum[kWaves][2][64];
  __shared__ Routing s_routing;
  read_routing(p, s_routing);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  // the blockIdx.y'th expert that has tokens, and the pairs before it
  int expert = -1, rows = 0;
  {
    int seen = 0;
    for (int base = 0; base < p.experts && expert < 0; base += 64) {
      const uint64_t mine = base + lane < p.experts ? mask_of(s_routing, base + lane) : 0;
      uint64_t live = __ballot(mine != 0);
      const int n = __builtin_popcountll(live), want = static_cast<int>(blockIdx.y) - seen;
      int pairs = __builtin_popcountll(mine);
      if (want < n) {
        for (int i = 0; i < want; ++i) live &= live - 1;
        const int at = __builtin_ctzll(live);
        expert = base + at;
        if (lane >= at) pairs = 0;
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) pairs += __shfl_xor(pairs, d);
      rows += pairs;
      seen += n;
    }
  }
  if (expert < 0) return;
  expert = __builtin_amdgcn_readfirstlane(expert);
  rows = __builtin_amdgcn_readfirstlane(rows);
  const uint64_t mask = mask_of(s_routing, expert);
  const int tokens = __builtin_amdgcn_readfirstlane(__builtin_popcountll(mask));

  const int64_t n0 = int64_t(16) * blockIdx.x, each = p.gated ? 2 * p.F : p.F, c0 = expert * each + n0;
  const Channels ch[2] = {channels(p.w1q, p.w1s, c0, p.F - n0, p.pitch1, p.steps1),
                          channels(p.w1q, p.w1s, p.gated ? c0 + p.F : c0, p.gated ? p.F - n0 : 0, p.pitch1, p.steps1)};
  int first, last;
  share_of(static_cast<int>(p.pitch1 / 64), wave, first, last);
  for (int t0 = 0; t0 < tokens; t0 += 16) {
    const int count = min(tokens - t0, 16);
    // the token of the lane's column, as a place among the expert's
    const int token = nth_token(mask, t0 + min(lane & 15, count - 1));
    auto row = [&](int r) {
      return static_cast<const char*>(p.x) + __shfl(token, r) * p.H * dtype_bytes(DT);
    };
    f32x4 acc[2] = {};
    run_units<DT, RU, 2, 2>(ch, first, last, p.H, count, s_x[wave], row, acc);
    __syncthreads();  // the sums before have been read
    s_sum[wave][0][lane] = acc[0];
    s_sum[wave][1][lane] = acc[1];
    __syncthreads();
    if (wave != 0) continue;
    f32x4 v[2] = {s_sum[0][0][lane], s_sum[0][1][lane]};
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      v[0] += s_sum[w][0][lane];
      v[1] += s_sum[w][1][lane];
    }
    if ((lane & 15) >= count) continue;
    float weight = 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
      const int s = token * p.top_k + j;
      if (id_of(p, s) == expert) weight += p.weights ? p.weights[s] : 1.0f;
    }
    constexpr int kParts = h_parts(DT);
    uint32_t out[kParts][2];
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      float part[2][3];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float gate = v[0][e + i], other = v[1][e + i];
        const float a = gate / (1.0f + expf(-gate));
        split((p.gated ? a * other : a) * weight, part[i]);
        // the last of the parts that are kept is rounded
        if constexpr (kParts == 2) part[i][1] = part[i][1] + part[i][2];
      }
#pragma unroll
      for (int k = 0; k < kParts; ++k)
        out[k][e / 2] = k + 1 < kParts ? upper_halves(part[0][k], part[1][k]) : pack_pair<NF4_BF16>(part[0][k], part[1][k]);
    }
    const int64_t n = n0 + 4 * (lane >> 4);
    uint16_t* to = p.h + (rows + t0 + (lane & 15)) * (kParts * p.h_width) + n;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      // (n is below h_width, which the channels' tiles fill; past F all is zero)
      const bool live = n < p.F;
      const uint2 two = {live ? out[k][0] : 0u, live ? out[k][1] : 0u};
      *reinterpret_cast<uint2*>(to + k * p.h_width) = two;
    }
  }
}

template <int DT, int RU, int TT>
__global__ __launch_bounds__(kThreads, 2) void mx_down_kernel(Mlp p) {
  constexpr int kParts = h_parts(DT), kFrom = kSplit + kParts;
  __shared__ __attribute__((aligned(16))) uint8_t s_h[kWaves][stage_bytes<kFrom, RU>()];
  __shared__ f32x4 s_sum[kWaves][TT][64];
  __shared__ Routing s_routing;
  __shared__ int s_list[kMaxExperts][2];  // the experts with tokens, and the pairs before each
  __shared__ int s_live;
  read_routing(p, s_routing);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (wave == 0) {
    int seen = 0, rows = 0;
    for (int base = 0; base < p.experts; base += 64) {
      const uint64_t mine = base + lane < p.experts ? mask_of(s_routing, base + lane) : 0;
      const uint64_t live = __ballot(mine != 0);
      const int pairs = __builtin_popcountll(mine);
      int in = pairs;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(in, d);
        if (lane >= d) in += o;
      }
      if (mine) {
        const int at = seen + __builtin_popcountll(live & ((uint64_t(1) << lane) - 1));
        s_list[at][0] = base + lane;
        s_list[at][1] = rows + in - pairs;
      }
      seen += __builtin_popcountll(live);
      rows += __shfl(in, 63);
    }
    if (lane == 0) s_live = seen;
  }
  __syncthreads();
  const int live = s_live, units = static_cast<int>(p.pitch2 / 64);
  const int64_t n0 = int64_t(16) * blockIdx.x;
  // the wave's units of all experts' (even numbers: whole lines)
  const int64_t all = int64_t(live) * units;
  const int64_t each = 2 * ((all + 2 * kWaves - 1) / (2 * kWaves));
  int64_t at = min(all, wave * each);
  const int64_t end = min(all, at + each);
  f32x4 total[TT] = {};
  while (at < end) {
    const int j = __builtin_amdgcn_readfirstlane(static_cast<int>(at / units));
    const int first = static_cast<int>(at - int64_t(j) * units);
    const int last = static_cast<int>(min(int64_t(units), end - int64_t(j) * units));
    at += last - first;
    const int expert = __builtin_amdgcn_readfirstlane(s_list[j][0]);
    const int rows = __builtin_amdgcn_readfirstlane(s_list[j][1]);
    const uint64_t mask = mask_of(s_routing, expert);
    const int tokens = __builtin_amdgcn_readfirstlane(__builtin_popcountll(mask));
    const Channels ch[1] = {channels(p.w2q, p.w2s, expert * p.H + n0, p.H - n0, p.pitch2, p.steps2)};
    for (int t0 = 0; t0 < tokens; t0 += 16) {
      const int count = min(tokens - t0, 16);
      auto row = [&](int r) {
        return reinterpret_cast<const char*>(p.h + static_cast<int64_t>(rows + t0 + r) * (kParts * p.h_width));
      };
      f32x4 acc[1] = {};
      run_units<kFrom, RU, 1, 4>(ch, first, last, p.h_width, count, s_h[wave], row, acc);
      // to the tokens' columns; the others keep theirs (not by adding zeros: a channel
      // whose weights are NaN leaves the tokens of other experts alone)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int token = 16 * t + (lane & 15);
        const int column = __builtin_popcountll(mask & ((uint64_t(1) << token) - 1)) - t0;
        const bool has = (mask >> token & 1) && column >= 0 && column < 16;
        const int from = (has ? column : 0) + (lane & 48);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = acc[0][e];
          const float o = __shfl(v, from);
          if (has) total[t][e] += o;
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) s_sum[wave][t][lane] = total[t];
  __syncthreads();
  if (wave >= TT) return;
  f32x4 sum = s_sum[0][wave][lane];
#pragma unroll
  for (int v = 1; v < kWaves; ++v) sum += s_sum[v][wave][lane];
  const int token = 16 * wave + (lane & 15);
  const int64_t n = n0 + 4 * (lane >> 4);
  const int left = static_cast<int>(min(p.H - n, int64_t(4)));
  if (token >= p.T || left <= 0) return;
  const float f[4] = {sum[0], sum[1], sum[2], sum[3]};
  store_four<DT>(p.y, token * p.H + n, left, f);
}

// Runs f with the loads of a unit's rows that `rows` rows (16 at most) take.
template <class F>
void with_loads(int64_t rows, F&& f) {
  if (rows <= 4)
    f(std::integral_constant<int, 1>{});
  else if (rows <= 8)
    f(std::integral_constant<int, 2>{});
  else
    f(std::integral_constant<int, 4>{});
}

int64_t h_width(int64_t F) { return (F + kUnit - 1) / kUnit * kUnit; }

bool known_mlp(int64_t T, int32_t top_k, int64_t F, int32_t dtype) {
  return T >= 0 && T <= kMaxTokens && top_k >= 1 && top_k <= kMaxTopK && F >= 0 && F <= kMaxK && known_dtype(dtype);
}

}  // namespace

extern "C" {

nf4_status mxfp4_gemv(const void* x, int32_t x_dtype, const uint8_t* wq, const uint8_t* ws, int64_t M,
                      int64_t N, int64_t K, void* y, int32_t y_dtype, void* stream) {
  if (M < 0 || M > 16 || N < 0 || K < 0 || !known_dtype(x_dtype) || !known_dtype(y_dtype)) return NF4_EINVAL;
  if (M == 0 || N == 0) return NF4_OK;
  if (!y || (K > 0 && (!x || !wq || !ws))) return NF4_EINVAL;
  if (!aligned(x, dtype_bytes(x_dtype)) || !aligned(wq, 16) || !aligned(ws, 16) || !aligned(y, dtype_bytes(y_dtype)))
    return NF4_EINVAL;
  if (N > kMaxDim || K > kMaxK) return NF4_EUNSUPPORTED;
  const Gemv p = {x, wq, ws, y, M, N, K, pitch_of(K), steps_of(K)};
  const int64_t tiles = (N + 15) / 16, most = 2 * device_cus();
  const dim3 grid(static_cast<uint32_t>(tiles < most ? tiles : most));
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  with_dtype(x_dtype, [&](auto a) {
    with_dtype(y_dtype, [&](auto d) {
      with_loads(M, [&](auto r) {
        hipLaunchKernelGGL((mx_gemv_kernel<decltype(a)::value, decltype(d)::value, decltype(r)::value>), grid,
                           dim3(kThreads), 0, st, p);
      });
    });
  });
  return launch_status();
}

size_t mxfp4_moe_mlp_workspace_size(int64_t T, int32_t top_k, int64_t F, int32_t dtype) {
  if (!known_mlp(T, top_k, F, dtype)) return 0;
  return static_cast<size_t>(T * top_k * h_parts(dtype) * h_width(F) * 2 + 255) / 256 * 256;
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
  if (!known_mlp(T, top_k, F, dtype) || H > kMaxK || experts > kMaxExperts || experts * H > kMaxDim ||
      experts * F * (gated ? 2 : 1) > kMaxDim)
    return NF4_EUNSUPPORTED;
  const size_t need = mxfp4_moe_mlp_workspace_size(T, top_k, F, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return NF4_EINVAL;
  Mlp p = {};
  p.x = x, p.w1q = w1q, p.w1s = w1s, p.w2q = w2q, p.w2s = w2s, p.ids = ids, p.weights = weights, p.y = y;
  p.h = static_cast<uint16_t*>(workspace);
  p.H = H, p.F = F, p.h_width = h_width(F);
  p.pitch1 = pitch_of(H), p.steps1 = steps_of(H), p.pitch2 = pitch_of(F), p.steps2 = steps_of(F);
  p.T = static_cast<int>(T), p.top_k = top_k, p.experts = F > 0 ? experts : 0, p.id_bytes = id_bytes, p.gated = gated;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int64_t slots = T * top_k, live = experts < slots ? experts : slots;
  with_dtype(dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    with_loads(T, [&](auto r) {
      constexpr int RU = decltype(r)::value;
      if (p.experts > 0)
        hipLaunchKernelGGL((mx_up_kernel<DT, RU>), dim3(static_cast<uint32_t>(p.h_width / 16), static_cast<uint32_t>(live)),
                           dim3(kThreads), 0, st, p);
      const dim3 grid(static_cast<uint32_t>((H + 15) / 16));
      if (T <= 16)
        hipLaunchKernelGGL((mx_down_kernel<DT, RU, 1>), grid, dim3(kThreads), 0, st, p);
      else if constexpr (RU == 4)
        hipLaunchKernelGGL((mx_down_kernel<DT, RU, 4>), grid, dim3(kThreads), 0, st, p);
    });
  });
  return launch_status();
}

}  // extern "C"
