// moe.hip -- routing around expert products: slots sorted by expert, rows moved
// into that order and back with the router's weights, and the gradients.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "int8_product.h"
#include "moe.h"
#include "nf4_device.h"
#include "row_io.h"

namespace {

using namespace nf4dev;
using namespace rowio;

// ---------------------------------------------------------------------------
// Sort.  A stable counting sort: the row of a slot is the number of slots with
// a smaller expert, plus those of its expert before it.  A workgroup of 16
// waves takes a tile of 1024 STEPS slots, wave w the 64 STEPS from 64 STEPS w on, 64
// at a time: the lanes of a wave find those with their own expert by one ballot per bit
// of the id, which gives the rank among the 64; counters per wave and expert
// in LDS carry it on.  After the tile, a sum over the waves and one over the
// experts turn the counters into rows.
//
// Up to kSortOne slots one workgroup does it all in one launch.  Beyond, a first
// kernel writes each workgroup's counts per expert to the workspace and a
// second one adds those of the workgroups before it to its own.  Latency bounds both,
// that of the tiles and of the sum over all workgroups' counts, which each of them
// takes for itself: 64 slots over 64 experts take 3.3 us, 32764 take 11.1 in a captured
// graph (4.8 and 8.2 traced apart), 131072 17.9, 524288 38.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortOne = 4 * kSortThreads;
constexpr int kMaxSortGroups = 256;
constexpr int kMaxExperts = 1024;
constexpr int64_t kMaxSlots = int64_t(1) << 30;

struct SortShared {
  uint16_t count[kSortWaves][kMaxExperts];  // per wave and expert, later the rows before the wave's
  uint32_t base[kMaxExperts];               // row of the expert's next slot
  uint32_t wave_sum[kSortWaves];
  uint32_t total;
};

__device__ __forceinline__ int slot_expert(const void* ids, int id_bytes, int64_t i, int64_t n,
                                           int experts) {
  if (i >= n) return -1;
  const int64_t e = id_bytes == 8 ? static_cast<const int64_t*>(ids)[i]
                                  : static_cast<const int32_t*>(ids)[i];
  return e >= 0 && e < experts ? static_cast<int>(e) : -1;
}

// Ranks the tile's slots within (wave, expert) and leaves the counters in
// s.count.
template <int STEPS>
__device__ __forceinline__ void rank_tile(SortShared& s, const int (&e)[STEPS], int (&rank)[STEPS], int experts,
                                          int bits) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = lane; i < experts; i += 64) s.count[wave][i] = 0;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int t = 0; t < STEPS; ++t) {
    uint64_t same = __ballot(e[t] >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((e[t] >> b) & 1);
      same &= (e[t] >> b) & 1 ? set : ~set;
    }
    rank[t] = 0;
    int before = 0, mine = 0;
    if (e[t] >= 0) {
      before = s.count[wave][e[t]];
      mine = __popcll(same & ((uint64_t(1) << lane) - 1));
      rank[t] = before + mine;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (e[t] >= 0 && mine == 0) s.count[wave][e[t]] = static_cast<uint16_t>(before + __popcll(same));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

__device__ __forceinline__ uint32_t wave_inclusive(uint32_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = static_cast<uint32_t>(__shfl_up(static_cast<int>(v), d));
    if (lane >= d) v += o;
  }
  return v;
}

// Thread i < experts gives expert i's count; returns the sum of those before it
// and leaves the sum of all in s.total.
__device__ __forceinline__ uint32_t scan_experts(SortShared& s, uint32_t v) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t in = wave_inclusive(v);
  if (lane == 63) s.wave_sum[wave] = in;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    before += w < wave ? s.wave_sum[w] : 0u;
    all += s.wave_sum[w];
  }
  if (threadIdx.x == 0) s.total = all;
  __syncthreads();
  return before + in - v;
}

// s.count[w][e] becomes the number of the tile's slots of expert e in the waves
// before w; returns the tile's count of expert threadIdx.x.
__device__ __forceinline__ uint32_t scan_waves(SortShared& s, int experts) {
  uint32_t sum = 0;
  const int e = threadIdx.x;
  if (e < experts)
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = s.count[w][e];
      s.count[w][e] = static_cast<uint16_t>(sum);
      sum += c;
    }
  return sum;
}

struct SortArgs {
  const void* ids;
  int id_bytes;
  int64_t n;
  int experts, bits;
  int32_t *offsets, *order, *pos;
  uint32_t* counts;    // [groups][experts] of the workspace
  int64_t per_group;   // slots of a workgroup, a multiple of the tile
};

template <int STEPS>
__device__ __forceinline__ void load_tile(const SortArgs& a, int64_t tile, int (&e)[STEPS]) {
  const int64_t first = tile + (threadIdx.x >> 6) * (64 * STEPS) + (threadIdx.x & 63);
#pragma unroll
  for (int t = 0; t < STEPS; ++t)
    e[t] = slot_expert(a.ids, a.id_bytes, first + 64 * t, a.n, a.experts);
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ uint32_t s_count[kMaxExperts];
  for (int i = threadIdx.x; i < a.experts; i += kSortThreads) s_count[i] = 0;
  __syncthreads();
  const int64_t begin = a.per_group * blockIdx.x;
  const int64_t end = min(a.n, begin + a.per_group);
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const int e = slot_expert(a.ids, a.id_bytes, i, a.n, a.experts);
    if (e >= 0) atomicAdd(&s_count[e], 1u);  // whole numbers: the order does not matter
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.experts; i += kSortThreads)
    a.counts[static_cast<int64_t>(blockIdx.x) * a.experts + i] = s_count[i];
}

// ONE: the only workgroup, of a single tile; its own counts are the totals.
template <bool ONE, int STEPS>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  __shared__ SortShared s;
  int e[STEPS], rank[STEPS];
  const int wave = threadIdx.x >> 6;
  const int64_t begin = ONE ? 0 : a.per_group * blockIdx.x;
  const int64_t end = ONE ? a.n : min(a.n, begin + a.per_group);
  if constexpr (!ONE) {
    uint32_t before = 0, all = 0;
    if (static_cast<int>(threadIdx.x) < a.experts)
      for (uint32_t g = 0; g < gridDim.x; ++g) {
        const uint32_t c = a.counts[static_cast<int64_t>(g) * a.experts + threadIdx.x];
        before += g < blockIdx.x ? c : 0u;
        all += c;
      }
    const uint32_t row = scan_experts(s, all);
    if (static_cast<int>(threadIdx.x) < a.experts) {
      s.base[threadIdx.x] = row + before;
      if (blockIdx.x == 0) a.offsets[threadIdx.x] = static_cast<int32_t>(row);
    }
  }
  for (int64_t tile = begin; tile < end || (ONE && tile == 0); tile += STEPS * kSortThreads) {
    load_tile(a, tile, e);
    rank_tile(s, e, rank, a.experts, a.bits);
    __syncthreads();
    const uint32_t tile_count = scan_waves(s, a.experts);
    if constexpr (ONE) {
      const uint32_t row = scan_experts(s, tile_count);
      if (static_cast<int>(threadIdx.x) < a.experts) {
        s.base[threadIdx.x] = row;
        a.offsets[threadIdx.x] = static_cast<int32_t>(row);
      }
    }
    __syncthreads();
    const int64_t first = tile + wave * (64 * STEPS) + (threadIdx.x & 63);
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      const int64_t i = first + 64 * t;
      if (i >= a.n) continue;
      int row = -1;
      if (e[t] >= 0) {
        row = static_cast<int>(s.base[e[t]] + s.count[wave][e[t]] + rank[t]);
        a.order[row] = static_cast<int32_t>(i);
      }
      a.pos[i] = row;
    }
    __syncthreads();
    if (!ONE && static_cast<int>(threadIdx.x) < a.experts) s.base[threadIdx.x] += tile_count;
    __syncthreads();
  }
  const uint32_t total = s.total;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.experts] = static_cast<int32_t>(total);
  for (int64_t i = total + static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; i < a.n;
       i += static_cast<int64_t>(gridDim.x) * kSortThreads)
    a.order[i] = -1;
}

// ---------------------------------------------------------------------------
// Rows.  2^width threads of a workgroup per token: all 256, or for short rows as
// many as there are pieces of eight (at most a wave, so that a token's sums stay
// within one).  Each row of the batch is read once and each sorted row read or
// written once; all three kernels are bound by memory: 8191 tokens of 4096 bf16
// with four slots, a tenth of them dropped, gather in 48-63 us (309 MB) and combine
// in 62 (5.0 TB/s), and 8192 with all slots give their gradients in 104-121 us
// (combine, 604 MB) and 64 (gather, 5.2 TB/s); a large copy reaches 4.9.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int64_t kMaxRowGroups = 1 << 20;  // a grid may not have 2^32 threads: past this, several turns

// Up to two pieces a lane a wave does better than the workgroup (8192 tokens with
// four slots combine rows of 64 in 4.9 us against 10.3, of 640 in 13.3 against 17.2,
// of 1024 in 16.6 against 19.0), with more it does not (gradients at 1536 54.7 against
// 43.4, at 2048 76 against 54).  With two pieces a lane that takes as many waves as the
// card holds at once: 4096 tokens with two slots combine rows of 1024 in 8.0 us against
// 8.5 (gradients 12.8 against 15.2), but where the tokens' waves leave a compute unit
// one workgroup at most, a workgroup each is faster: 1024 tokens in 5.4 us against 4.3
// (8.5 against 6.1), 257 of 1001 fp32 in 6.2 against 3.7 (8.9 against 6.6), 64 in 3.2
// against 2.5.  (At 2048 it depends: 6.3 and 5.6 at 1024 bf16, gradients 15.5 and 17.2
// at 1001 fp32.)
int row_width(int64_t T, int64_t H) {
  if (H > 16 * 64 || (H > 8 * 64 && T <= 4 * device_cus())) return 8;
  int width = 3;
  while (width < 6 && (8 << width) < H) ++width;
  return width;
}

uint32_t row_groups(int64_t T, int width) {
  const int64_t n = (T + (kRowThreads >> width) - 1) / (kRowThreads >> width);
  return static_cast<uint32_t>(n < kMaxRowGroups ? n : kMaxRowGroups);
}

struct RowArgs {
  const int32_t* pos;
  int64_t T;
  int top_k;
  int64_t rows, H;
  int width;
};

// WIDE: width 8, where the token is the workgroup's and its slots are read as
// scalars.
template <bool WIDE>
struct Rows : RowArgs {
  __device__ __forceinline__ explicit Rows(const RowArgs& a) : RowArgs(a) {
    if (WIDE) width = 8;
  }
  __device__ __forceinline__ int64_t first() const {
    return WIDE ? blockIdx.x : int64_t(blockIdx.x) * (kRowThreads >> width) + (threadIdx.x >> width);
  }
  __device__ __forceinline__ int64_t turn() const { return int64_t(gridDim.x) * (kRowThreads >> width); }
  __device__ __forceinline__ int64_t piece() const { return 8 * (threadIdx.x & ((1 << width) - 1)); }
  __device__ __forceinline__ int64_t stride() const { return 8 << width; }
  // f(true, at) for the thread's whole pieces of a row, f(false, at) for the row's
  // last, shorter one: a test in every load would part the loads
  template <class F>
  __device__ __forceinline__ void pieces(F&& f) const {
    for (int64_t at = piece(); at + 8 <= H; at += stride()) f(std::true_type{}, at);
    const int64_t last = H & ~int64_t(7);
    if (last < H && ((last ^ piece()) & (stride() - 1)) == 0) f(std::false_type{}, last);
  }
  // the sorted row of slot j of token t, -1 if it has none
  __device__ __forceinline__ int64_t row(int64_t t, int j) const {
    const int32_t p = pos[t * top_k + j];
    return p >= 0 && p < rows ? p : -1;
  }
};

template <int DT, bool STREAM, class WHOLE>
__device__ __forceinline__ Piece<DT> get(WHOLE, const void* p, int64_t row_bytes, int64_t row, int64_t at, int64_t H) {
  const char* r = static_cast<const char*>(p) + row * row_bytes;
  if constexpr (WHOLE::value)
    return whole_piece<DT, STREAM>(r, at);
  else
    return load_piece<DT>(r, at, H);
}

template <int DT, class WHOLE>
__device__ __forceinline__ void put(WHOLE, void* p, int64_t row_bytes, int64_t row, int64_t at, int64_t H,
                                    const Piece<DT>& v) {
  char* r = static_cast<char*>(p) + row * row_bytes;
  if constexpr (WHOLE::value)
    store_whole_piece<DT>(r, at, v);
  else
    store_piece<DT>(r, at, H, v);
}

template <int DT, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void gather_kernel(RowArgs args, const void* __restrict__ x,
                                                             void* __restrict__ xs) {
  const Rows<WIDE> a(args);
  const int64_t bytes = a.H * dtype_bytes(DT);
  for (int64_t t = a.first(); t < a.T; t += a.turn())
    a.pieces([&](auto whole, int64_t at) {
      const Piece<DT> p = get<DT, false>(whole, x, bytes, t, at, a.H);
      for (int j = 0; j < a.top_k; ++j) {
        const int64_t r = a.row(t, j);
        if (r >= 0) put<DT>(whole, xs, bytes, r, at, a.H, p);
      }
    });
}

// The sorted rows are read past the caches: 62 us for 8191 tokens of 4096 with four
// slots, 87 through them.  (Rows that gather writes gain nothing from that.)
template <int DT, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(RowArgs args, const void* __restrict__ ys,
                                                              const float* __restrict__ weights,
                                                              void* __restrict__ y) {
  constexpr int kSlots = 4;  // whose rows are asked for together
  const Rows<WIDE> a(args);
  const int64_t bytes = a.H * dtype_bytes(DT);
  for (int64_t t = a.first(); t < a.T; t += a.turn())
    a.pieces([&](auto whole, int64_t at) {
      float acc[8] = {};
      for (int j0 = 0; j0 < a.top_k; j0 += kSlots) {
        Piece<DT> p[kSlots];
        float w[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          const int64_t r = j0 + j < a.top_k ? a.row(t, j0 + j) : -1;
          p[j] = Piece<DT>{};
          w[j] = 0.0f;
          if (r < 0) continue;  // adds 0 * 0
          w[j] = weights ? weights[t * a.top_k + j0 + j] : 1.0f;
          p[j] = get<DT, true>(whole, ys, bytes, r, at, a.H);
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[j], element<DT>(p[j], i), acc[i]);
      }
      put<DT>(whole, y, bytes, t, at, a.H, make_piece<DT>(acc));
    });
}

// Four slots at a time: their sums over the row run side by side, each a chain of
// FMAs per thread and then a tree over the threads in a fixed order.
template <int DT, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void combine_grad_kernel(RowArgs args, const void* __restrict__ dy,
                                                                   const void* __restrict__ ys,
                                                                   const float* __restrict__ weights,
                                                                   void* __restrict__ dys,
                                                                   float* __restrict__ dweights) {
  constexpr int kSlots = 4, kWaves = kRowThreads / 64;
  __shared__ float s_sum[kWaves][kSlots];
  const Rows<WIDE> a(args);
  const int64_t bytes = a.H * dtype_bytes(DT);
  // every thread takes as many turns: there is a barrier in them
  const int64_t turns = (a.T + a.turn() - 1) / a.turn();
  for (int64_t i = 0; i < turns; ++i) {
    const int64_t t = a.first() + i * a.turn();
    const bool live = t < a.T;
    for (int j0 = 0; j0 < a.top_k; j0 += kSlots) {
      float dot[kSlots] = {};
      if (live)
        a.pieces([&](auto whole, int64_t at) {
          const Piece<DT> g = get<DT, false>(whole, dy, bytes, t, at, a.H);
          Piece<DT> p[kSlots];
          int64_t r[kSlots];
#pragma unroll
          for (int j = 0; j < kSlots; ++j) {
            r[j] = j0 + j < a.top_k ? a.row(t, j0 + j) : -1;
            p[j] = Piece<DT>{};
            if (r[j] >= 0 && dweights) p[j] = get<DT, true>(whole, ys, bytes, r[j], at, a.H);
          }
#pragma unroll
          for (int j = 0; j < kSlots; ++j) {
            if (r[j] < 0) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) dot[j] = fmaf(element<DT>(p[j], e), element<DT>(g, e), dot[j]);
            if (dys) {
              const float w = weights ? weights[t * a.top_k + j0 + j] : 1.0f;
              float f[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] = w * element<DT>(g, e);
              put<DT>(whole, dys, bytes, r[j], at, a.H, make_piece<DT>(f));
            }
          }
        });
      if (!dweights) continue;
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        for (int d = (a.width < 6 ? 1 << a.width : 64) / 2; d >= 1; d >>= 1) dot[j] += __shfl_xor(dot[j], d);
      if (a.width > 6) {  // the token's waves
        if ((threadIdx.x & 63) == 0)
#pragma unroll
          for (int j = 0; j < kSlots; ++j) s_sum[threadIdx.x >> 6][j] = dot[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          dot[j] = s_sum[0][j];
#pragma unroll
          for (int v = 1; v < kWaves; ++v) dot[j] += s_sum[v][j];
        }
        __syncthreads();
      }
      if (live && a.piece() == 0)
#pragma unroll
        for (int j = 0; j < kSlots; ++j)  // a slot without a row has added nothing
          if (j0 + j < a.top_k) dweights[t * a.top_k + j0 + j] = dot[j];
    }
  }
}

// Steps of a workgroup's tile.  One workgroup: no more than the slots fill (64 slots in
// 3.2 us, with four steps 4.7).  Several: two for few slots, which more workgroups
// then share (8192 in 7.5 us against 9.1, 32764 in 10.7 against 11.1), four for many,
// whose workgroups would be too many to add up (131072 in 16.8 against 21.1; each pair
// from one run).
int sort_steps(int64_t n) {
  if (n <= kSortOne) return n <= kSortThreads ? 1 : n <= 2 * kSortThreads ? 2 : 4;
  return n <= 32768 ? 2 : 4;
}

int64_t sort_groups(int64_t n, int64_t* per_group) {
  const int64_t tile = int64_t(sort_steps(n)) * kSortThreads, tiles = (n + tile - 1) / tile;
  const int64_t per = (tiles + kMaxSortGroups - 1) / kMaxSortGroups;
  *per_group = per * tile;
  return (tiles + per - 1) / per;
}

bool slots_fit(int64_t T, int32_t top_k) { return T <= kMaxSlots / top_k; }

// What gather, combine and combine_grad check alike.
nf4_status check_rows(int32_t dtype, const int32_t* pos, int64_t T, int32_t top_k, int64_t rows,
                      int64_t H) {
  if (T < 0 || top_k < 1 || rows < 0 || H < 0 || !known_dtype(dtype)) return NF4_EINVAL;
  if (T > 0 && (!pos || !aligned(pos, 4))) return NF4_EINVAL;
  if (!slots_fit(T, top_k) || rows > int8dev::kMaxDim || H > int8dev::kMaxDim)
    return NF4_EUNSUPPORTED;
  return NF4_OK;
}

}  // namespace

extern "C" {

size_t moe_sort_workspace_size(int64_t T, int32_t top_k, int32_t experts) {
  if (T <= 0 || top_k < 1 || experts < 1 || experts > kMaxExperts || !slots_fit(T, top_k)) return 0;
  if (T * top_k <= kSortOne) return 0;
  int64_t per = 0;
  return static_cast<size_t>(sort_groups(T * top_k, &per)) * experts * sizeof(uint32_t);
}

nf4_status moe_sort(const void* ids, int32_t id_bytes, int64_t T, int32_t top_k, int32_t experts,
                    int32_t* offsets, int32_t* order, int32_t* pos, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (T < 0 || top_k < 1 || experts < 0 || (id_bytes != 4 && id_bytes != 8)) return NF4_EINVAL;
  if (!offsets || !aligned(offsets, 4)) return NF4_EINVAL;
  if (T > 0 && (!ids || !order || !pos)) return NF4_EINVAL;
  if (!aligned(ids, id_bytes) || !aligned(order, 4) || !aligned(pos, 4) || !aligned(workspace, 256))
    return NF4_EINVAL;
  if (experts > kMaxExperts || !slots_fit(T, top_k)) return NF4_EUNSUPPORTED;
  const size_t need = moe_sort_workspace_size(T, top_k, experts);
  if (need > 0 && (!workspace || workspace_bytes < need)) return NF4_EINVAL;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  SortArgs a = {ids, id_bytes, T * top_k, experts, 0, offsets, order, pos, nullptr, 0};
  while ((1 << a.bits) < experts) ++a.bits;
  if (a.n <= kSortOne) {
    switch (sort_steps(a.n)) {
      case 1: hipLaunchKernelGGL((sort_place_kernel<true, 1>), dim3(1), dim3(kSortThreads), 0, st, a); break;
      case 2: hipLaunchKernelGGL((sort_place_kernel<true, 2>), dim3(1), dim3(kSortThreads), 0, st, a); break;
      default: hipLaunchKernelGGL((sort_place_kernel<true, 4>), dim3(1), dim3(kSortThreads), 0, st, a);
    }
    return launch_status();
  }
  const uint32_t groups = static_cast<uint32_t>(sort_groups(a.n, &a.per_group));
  a.counts = static_cast<uint32_t*>(workspace);
  hipLaunchKernelGGL(sort_count_kernel, dim3(groups), dim3(kSortThreads), 0, st, a);
  if (sort_steps(a.n) == 2)
    hipLaunchKernelGGL((sort_place_kernel<false, 2>), dim3(groups), dim3(kSortThreads), 0, st, a);
  else
    hipLaunchKernelGGL((sort_place_kernel<false, 4>), dim3(groups), dim3(kSortThreads), 0, st, a);
  return launch_status();
}

nf4_status moe_gather(const void* x, int32_t dtype, const int32_t* pos, int64_t T, int32_t top_k,
                      int64_t rows, int64_t H, void* xs, void* stream) {
  if (const nf4_status st = check_rows(dtype, pos, T, top_k, rows, H)) return st;
  if (T == 0 || rows == 0 || H == 0) return NF4_OK;
  if (!x || !xs || !aligned(x, dtype_bytes(dtype)) || !aligned(xs, dtype_bytes(dtype)))
    return NF4_EINVAL;
  const RowArgs a = {pos, T, top_k, rows, H, row_width(T, H)};
  with_dtype(dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    const dim3 grid(row_groups(T, a.width));
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (a.width == 8)
      hipLaunchKernelGGL((gather_kernel<DT, true>), grid, dim3(kRowThreads), 0, st, a, x, xs);
    else
      hipLaunchKernelGGL((gather_kernel<DT, false>), grid, dim3(kRowThreads), 0, st, a, x, xs);
  });
  return launch_status();
}

nf4_status moe_combine(const void* ys, int32_t dtype, const float* weights, const int32_t* pos,
                       int64_t T, int32_t top_k, int64_t rows, int64_t H, void* y, void* stream) {
  if (const nf4_status st = check_rows(dtype, pos, T, top_k, rows, H)) return st;
  if (T == 0 || H == 0) return NF4_OK;
  if ((rows > 0 && !ys) || !y || !aligned(ys, dtype_bytes(dtype)) ||
      !aligned(y, dtype_bytes(dtype)) || !aligned(weights, 4))
    return NF4_EINVAL;
  const RowArgs a = {pos, T, top_k, rows, H, row_width(T, H)};
  with_dtype(dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    const dim3 grid(row_groups(T, a.width));
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (a.width == 8)
      hipLaunchKernelGGL((combine_kernel<DT, true>), grid, dim3(kRowThreads), 0, st, a, ys, weights, y);
    else
      hipLaunchKernelGGL((combine_kernel<DT, false>), grid, dim3(kRowThreads), 0, st, a, ys, weights, y);
  });
  return launch_status();
}

nf4_status moe_combine_grad(const void* dy, const void* ys, int32_t dtype, const float* weights,
                            const int32_t* pos, int64_t T, int32_t top_k, int64_t rows, int64_t H,
                            void* dys, float* dweights, void* stream) {
  if (const nf4_status st = check_rows(dtype, pos, T, top_k, rows, H)) return st;
  if (T == 0 || (!dys && !dweights)) return NF4_OK;
  const int b = dtype_bytes(dtype);
  if ((H > 0 && !dy) || (H > 0 && rows > 0 && dweights && !ys)) return NF4_EINVAL;
  if (!aligned(dy, b) || !aligned(ys, b) || !aligned(dys, b) || !aligned(weights, 4) ||
      !aligned(dweights, 4))
    return NF4_EINVAL;
  const RowArgs a = {pos, T, top_k, rows, H, row_width(T, H)};
  with_dtype(dtype, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    const dim3 grid(row_groups(T, a.width));
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (a.width == 8)
      hipLaunchKernelGGL((combine_grad_kernel<DT, true>), grid, dim3(kRowThreads), 0, st, a, dy, ys, weights, dys, dweights);
    else
      hipLaunchKernelGGL((combine_grad_kernel<DT, false>), grid, dim3(kRowThreads), 0, st, a, dy, ys, weights, dys, dweights);
  });
  return launch_status();
}

}  // extern "C"
