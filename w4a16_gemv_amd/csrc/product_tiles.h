// product_tiles.h -- what the int8 and the 4-bit products share: where a workgroup's
// tile lies, loads from memory straight to LDS, and the last stores (private to
// libnf4).  P is the product's description, with M, N, x_rows, order, offsets, top_k
// and experts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8.h"
#include "nf4_device.h"
#include "row_io.h"

namespace tiledev {

using namespace nf4dev;
using namespace rowio;

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxExperts = 1024;

// Where a tile of rows lies: rows [first, end) of y, of expert `expert`
// (end <= first: no tile).
struct RowTile {
  int64_t first, end;
  int expert;
};

// The tile'th tile of BM rows over all experts, each of which starts a new
// tile: 64 experts at a time, the lanes count theirs' tiles and sum them up.
template <int BM, class P>
__device__ __forceinline__ RowTile find_tile(const P& p, int64_t tile) {
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
template <bool GROUPED, class P>
__device__ __forceinline__ int64_t source_row(const P& p, int64_t i) {
  if constexpr (!GROUPED) return i;
  const int64_t s = p.order ? (p.order[i] < 0 ? -1 : p.order[i] / p.top_k) : i;
  return s < p.x_rows ? s : -1;
}

// The bits of a row's outputs that stay: none of a row without a source.
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
template <int BM, class P>
__device__ __forceinline__ uint32_t count_tiles(const P& p) {
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

template <int DT>
__device__ __forceinline__ void store_one(void* y, int64_t i, float v) {
  if constexpr (DT == INT8_FP32)
    static_cast<float*>(y)[i] = v;
  else
    static_cast<uint16_t*>(y)[i] = to_half_bits<DT>(v);
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

// Loads of 16 bytes a lane from memory to LDS, lane l's to byte 16 l from `to` on
// (one address per wave), and of 4 bytes.  The builtins for these would do, but for the
// waits: the compiler puts one for all of them before a loop's first LDS read, every
// time round.  Nothing lands in a register, and the kernel does all the waiting.  m0
// holds the LDS address.  It stands among the clobbers, so that the compiler carries no
// value of its own in it across a load; the warning put off here says that it does not
// save m0 around the statement either, which nothing asks for.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_load(uint32_t to, i32x4 range, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(at), "s"(range)
               : "m0", "memory");
}
__device__ __forceinline__ void lds_load(uint32_t to, const int8_t* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "m0", "memory");
}
__device__ __forceinline__ void lds_load_dword(uint32_t to, const uint8_t* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "m0", "memory");
}
#pragma clang diagnostic pop

// Tiles of BM rows that p.M rows need at most: every expert ends in at most one
// tile that is not full.
template <bool GROUPED, class P>
int64_t row_tiles(const P& p, int64_t BM) {
  if constexpr (GROUPED) return p.M / BM + (p.M < p.experts ? p.M : p.experts);
  return (p.M + BM - 1) / BM;
}

// Workgroups of `threads` for the tiles, a multiple of the dies; 0 if a grid
// cannot have so many.
template <bool GROUPED, class P>
uint32_t tile_groups(const P& p, int BM, int BN, int threads) {
  const int64_t all = row_tiles<GROUPED>(p, BM) * ((p.N + BN - 1) / BN);
  const int64_t groups = (all + kDies - 1) / kDies * kDies;
  return groups * threads < (int64_t(1) << 32) ? static_cast<uint32_t>(groups) : 0;
}

}  // namespace tiledev
